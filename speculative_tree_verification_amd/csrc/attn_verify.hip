// attn_verify.hip -- attention of a packed tree's nodes over the paged cache:
// the plain fp32 kernel (any head_dim up to 256, any types), the join of the
// parts, and the choice of the kernel. The kernels on matrix instructions are in
// attn_mfma.hip (bf16) and attn_f32.hip.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = 2^(scale log2(e) q_i . k_j - m_i)
// over the cache's positions and node i's ancestors, in one pass with a running
// maximum m_i and sum; parts of the cache (attn_common.hpp) are joined by
//   o = sum_k 2^(m_k - m) o_k / sum_k 2^(m_k - m) l_k,  m = max_k m_k.
//
// Plain kernel: a work-group takes kRows rows (node, query head) of one key
// head and one part; its waves take 64 keys each in turn. Scores: a lane per
// key, the rows' q from LDS (the same for all lanes). Values: lanes over the
// head_dim, weights from LDS. Bound by the vector ALU and the LDS broadcasts (4 D
// operations per row and key): 4 trees of 63 nodes over 2200 positions, 32 heads of
// 128, 721 us where attn_f32.hip takes 106; 32 bf16 trees over 300 to 4099 of them,
// 16 heads of 256, 6.6 ms.
#include "attn_common.hpp"

namespace tsv {

namespace {

constexpr int kRows = 8;

template <typename TC>
__device__ __forceinline__ float elem(const TC* p, size_t i) {
    if constexpr (sizeof(TC) == 1)
        return e4m3_ld((const uint8_t*)p + i);
    else
        return Elem<TC>::ld(p, i);
}

// One wave's 64 keys: scores, running maximum, weights, products with v.
// `key`: this lane's row in kp / vp (elements), -1: none; ks, vs: its scales.
template <typename TC, int DV>
__device__ __forceinline__ void plain_tile(const AttnArgs& a, const TC* kp, const TC* vp, long long key, float ks, float vs,
                                           const uint32_t* s_anc, int words, int tree_key, const int* s_node,
                                           const float (*s_q)[256], float (*s_p)[kWave], long long* s_off, int n,
                                           float* m, float* l, float (*o)[DV]) {
    const int lane = threadIdx.x & (kWave - 1), D = a.D;
    float s[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) s[r] = 0.f;
    if (key >= 0) {
        for (int d = 0; d < D; ++d) {
            const float kv = elem<TC>(kp, (size_t)key * D + d);
#pragma unroll
            for (int r = 0; r < kRows; ++r) s[r] = fmaf(s_q[r][d], kv, s[r]);
        }
    }
    s_off[lane] = key;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        bool seen = key >= 0;
        if (s_anc && seen) seen = s_anc[s_node[r] * words + tree_key / 32] >> (tree_key % 32) & 1;
        const float sc = seen ? s[r] * ks * a.scale_log2 : -INFINITY;
        float top = sc;
#pragma unroll
        for (int x = 1; x < kWave; x <<= 1) top = fmaxf(top, __shfl_xor(top, x, kWave));
        // fmaxf passes over a NaN, which the weights then carry
        const float mn = fmaxf(m[r], top), base = mn == -INFINITY ? 0.f : mn;
        const float p = seen ? exp2f(sc - base) : 0.f, al = exp2f(m[r] - base);
        float sum = p;
#pragma unroll
        for (int x = 1; x < kWave; x <<= 1) sum += __shfl_xor(sum, x, kWave);
        l[r] = l[r] * al + sum;
        m[r] = mn;
#pragma unroll
        for (int i = 0; i < DV; ++i) o[r][i] *= al;
        s_p[r][lane] = p * vs;
    }
    wave_sync();
    for (int j = 0; j < n; ++j) {
        const long long at = s_off[j];
        if (at < 0) continue;
#pragma unroll
        for (int i = 0; i < DV; ++i) {
            const int d = lane + i * kWave;
            if (d >= D) continue;
            const float v = elem<TC>(vp, (size_t)at * D + d);
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                // a key that row r does not see has weight 0, also where its value is not finite
                const float p = s_p[r][j];
                o[r][i] = p == 0.f ? o[r][i] : fmaf(p, v, o[r][i]);
            }
        }
    }
    wave_sync();
}

template <typename TIO, typename TC, int DV>
__global__ __launch_bounds__(256) void attn_plain_kernel(AttnArgs a, AttnPlan plan, AttnWorkspace ws, int row_blocks) {
    __shared__ __attribute__((aligned(8))) int s_red[6];
    __shared__ Part s_part;
    __shared__ float s_q[kRows][256], s_p[4][kRows][kWave], s_o[kRows][256], s_ml[4][kRows][2];
    __shared__ long long s_off[4][kWave];
    __shared__ int s_par[1024], s_node[kRows];
    __shared__ uint32_t s_anc[kRows * 32];
    const int tid = threadIdx.x, lane = tid & (kWave - 1), w = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int reader = blockIdx.x % plan.readers, hk = reader / row_blocks, rb = reader % row_blocks;
    const Part pt = find_part<256>(a.cache_len, a.batch, a.room, plan, blockIdx.x / plan.readers, false, s_red, &s_part);
    if (!pt.ok) return;
    const int b = pt.item, T = a.T, H = a.H, D = a.D, g = H / a.Hk, R = T * g, row0 = rb * kRows;
    const bool last = pt.k == pt.n - 1;
    int st = pt.bad_len ? kStBadCache : 0;
    const int first = row0 / g, nodes = min(R - 1, row0 + kRows - 1) / g - first + 1, words = (T + 31) / 32;
    if (last) st |= tree_words<256>(a.parent + (size_t)b * T, T, first, nodes, words, s_par, s_anc);
    for (int i = tid; i < kRows * D; i += 256) {
        const int r = row0 + i / D;
        s_q[i / D][i % D] = r < R ? Elem<TIO>::ld((const TIO*)a.q, (((size_t)b * T + r / g) * H + hk * g + r % g) * D + i % D) : 0.f;
    }
    if (tid < kRows) s_node[tid] = min(R - 1, row0 + tid) / g - first;
    __syncthreads();
    float m[kRows], l[kRows], o[kRows][DV];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int i = 0; i < DV; ++i) o[r][i] = 0.f;
    }
    const int k0 = pt.k * pt.keys, k1 = last ? pt.len : min(pt.len, k0 + pt.keys);
    int bad = 0;
    for (int t0 = k0 + w * kWave; t0 < k1; t0 += 4 * kWave) {
        const int pos = t0 + lane;
        long long key = -1;
        float ks = 1.f, vs = 1.f;
        if (pos < k1) {
            const int page = page_of(pos, a.div), pg = a.page_table[(size_t)b * a.max_pages + page];
            if (pg < 0 || pg >= a.n_pages) {
                bad = 1;
            } else {
                key = ((long long)pg * a.Hk + hk) * a.page_size + (pos - page * a.page_size);
                if (a.k_scale) {
                    ks = a.k_scale[key];
                    vs = a.v_scale[key];
                }
            }
        }
        plain_tile<TC, DV>(a, (const TC*)a.k_cache, (const TC*)a.v_cache, key, ks, vs, nullptr, 0, 0, s_node, s_q, s_p[w],
                           s_off[w], min(kWave, k1 - t0), m, l, o);
    }
    if (last && !st) {
        for (int t0 = w * kWave; t0 < T; t0 += 4 * kWave) {
            const int j = t0 + lane;
            plain_tile<TIO, DV>(a, (const TIO*)a.k, (const TIO*)a.v, j < T ? ((long long)b * T + j) * a.Hk + hk : -1, 1.f, 1.f,
                                s_anc, words, min(j, T - 1), s_node, s_q, s_p[w], s_off[w], min(kWave, T - t0), m, l, o);
        }
    }
    st |= __syncthreads_or(bad) ? kStBadCache : 0;
    // the four waves' parts
#pragma unroll
    for (int r = 0; r < kRows; ++r)
        if (lane == 0) {
            s_ml[w][r][0] = m[r];
            s_ml[w][r][1] = l[r];
        }
    __syncthreads();
    float mt[kRows], lt[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        mt[r] = fmaxf(fmaxf(s_ml[0][r][0], s_ml[1][r][0]), fmaxf(s_ml[2][r][0], s_ml[3][r][0]));
        const float base = mt[r] == -INFINITY ? 0.f : mt[r];
        lt[r] = 0.f;
#pragma unroll
        for (int x = 0; x < 4; ++x) lt[r] += s_ml[x][r][1] * exp2f(s_ml[x][r][0] - base);
        const float al = exp2f(m[r] - base);
#pragma unroll
        for (int i = 0; i < DV; ++i) o[r][i] *= al;
    }
    for (int x = 0; x < 4; ++x) {
        if (w == x) {
#pragma unroll
            for (int r = 0; r < kRows; ++r)
#pragma unroll
                for (int i = 0; i < DV; ++i) {
                    const int d = lane + i * kWave;
                    s_o[r][d] = x == 0 ? o[r][i] : s_o[r][d] + o[r][i];
                }
        }
        __syncthreads();
    }
    const int part = blockIdx.x / plan.readers;
    if (reader == 0 && tid == 0) {
        if (pt.n > 1)
            ws.bits[part] = st;
        else if (a.status)
            a.status[b] = st;
    }
    if (pt.n == 1 && st) return;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        if (row0 + r >= R) break;
        const int node = (row0 + r) / g, head = hk * g + (row0 + r) % g;
        const size_t row = (size_t)node * H + head;
        if (pt.n > 1) {
            if (tid < D) ws.o[((size_t)part * T * H + row) * D + tid] = s_o[r][tid];
            if (tid < 2) ws.ml[((size_t)part * T * H + row) * 2 + tid] = tid ? lt[r] : mt[r];
        } else if (tid < D) {
            Elem<TIO>::st((TIO*)a.o, ((size_t)b * T * H + row) * D + tid, s_o[r][tid] / lt[r]);
        }
    }
}

// Lanes take 4 elements of a row each, LPR lanes a row.
//   RW 0  few rows (one new token over a long cache: up to 130 parts): each has a
//         work-group, whose waves split its parts (38 -> 7 us)
//   RW 1  each has a wave, which reads PW = 64 / LPR parts at once, four times
//         that before it adds; the parts' maxima and sums are a lane's each, 64 at
//         a time, with a running maximum over them
//   RW 4  many rows: few parts each, and the work per row counts. LPR lanes read
//         the row's parts by themselves, four at once, for RW rows one after
//         another (the search for the item's parts costs as much as a row). 64512
//         rows of 1 to 6 parts: 16 us, and 34 us read as by RW 1
template <typename TIO, int LPR, int RW>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a, AttnPlan plan, AttnWorkspace ws, int blocks) {
    constexpr int PW = kWave / LPR;
    constexpr bool SHARED = RW == 0;
    __shared__ __attribute__((aligned(8))) int s_red[6];
    __shared__ Part s_part;
    __shared__ __attribute__((aligned(16))) float s_o[4][LPR * 4];
    __shared__ float s_ml[4][2];
    const int tid = threadIdx.x, lane = tid & (kWave - 1), w = __builtin_amdgcn_readfirstlane(tid / kWave);
    const Part pt = find_part<256>(a.cache_len, a.batch, a.room, plan, blockIdx.x / blocks, true, s_red, &s_part);
    if (pt.n < 2) return;
    const int rows = a.T * a.H, D = a.D, n = pt.n, rb = blockIdx.x % blocks;
    int bits = 0;
    for (int k = tid; k < n; k += 256) bits |= ws.bits[pt.base + k];
    if (__syncthreads_or(bits)) {
        int all = 0;
        for (int bit = 1; bit <= kStBadCache; bit <<= 1) all |= __syncthreads_or(bits & bit) ? bit : 0;
        if (rb == 0 && tid == 0 && a.status) a.status[pt.item] = all;
        return;
    }
    if (rb == 0 && tid == 0 && a.status) a.status[pt.item] = 0;
    const int d = lane % LPR * 4, sub = lane / LPR;
    const bool whole = D % 4 == 0 && (uintptr_t)a.o % (4 * sizeof(TIO)) == 0;  // pieces of four, aligned
    auto piece = [&](const float* p) { return d >= D ? make_float4(0.f, 0.f, 0.f, 0.f) : whole ? ld4<true>(p, 4) : ld4<false>(p, D - d); };
    auto finish = [&](int row, float4 o, float l) {
        const float f[4] = {o.x / l, o.y / l, o.z / l, o.w / l};
        TIO* to = (TIO*)a.o + ((size_t)pt.item * rows + row) * D + d;
        if (whole && d < D) {
            if constexpr (sizeof(TIO) == 4)
                *(float4*)to = make_float4(f[0], f[1], f[2], f[3]);
            else
                *(uint2*)to = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (d + e < D) Elem<TIO>::st(to, e, f[e]);
        }
    };
    if (RW > 1) {
        for (int i = 0; i < RW; ++i) {
            const int row = ((rb * 4 + w) * RW + i) * PW + sub;
            if (row >= rows) return;
            const float* ml = ws.ml + ((size_t)pt.base * rows + row) * 2;
            const float* po = ws.o + ((size_t)pt.base * rows + row) * D + d;
            float m = -INFINITY, l = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k0 = 0; k0 < n; k0 += 4) {
                float mk[4], lk[4];
                float4 v[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    mk[u] = -INFINITY;
                    lk[u] = 0.f;
                    v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (k0 + u >= n) continue;
                    mk[u] = ml[(size_t)(k0 + u) * rows * 2];
                    lk[u] = ml[(size_t)(k0 + u) * rows * 2 + 1];
                    v[u] = piece(po + (size_t)(k0 + u) * rows * D);
                }
                const float mn = fmaxf(fmaxf(fmaxf(mk[0], mk[1]), fmaxf(mk[2], mk[3])), m);
                const float base = mn == -INFINITY ? 0.f : mn, old = exp2f(m - base);
                l *= old;
                o = make_float4(o.x * old, o.y * old, o.z * old, o.w * old);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float f = exp2f(mk[u] - base);
                    l = fmaf(f, lk[u], l);
                    o.x = fmaf(f, v[u].x, o.x);
                    o.y = fmaf(f, v[u].y, o.y);
                    o.z = fmaf(f, v[u].z, o.z);
                    o.w = fmaf(f, v[u].w, o.w);
                }
                m = mn;
            }
            finish(row, o, l);
        }
        return;
    }
    const int per = SHARED ? (n + 3) / 4 : n, first = SHARED ? w * per : 0, end = min(n, first + per);
    for (int i = 0; i < (SHARED ? 1 : RW); ++i) {
        const int row = SHARED ? rb : (rb * 4 + w) * RW + i;
        if (row >= rows) return;  // the same for all threads where they share
        const float* ml = ws.ml + ((size_t)pt.base * rows + row) * 2;
        const float* po = ws.o + ((size_t)pt.base * rows + row) * D + d;
        float m = -INFINITY, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c0 = first; c0 < end; c0 += kWave) {
            const int cnt = min(kWave, end - c0);
            float mk = -INFINITY, lk = 0.f;
            if (lane < cnt) {
                mk = ml[(size_t)(c0 + lane) * rows * 2];
                lk = ml[(size_t)(c0 + lane) * rows * 2 + 1];
            }
            float top = mk;
#pragma unroll
            for (int x = 1; x < kWave; x <<= 1) top = fmaxf(top, __shfl_xor(top, x, kWave));
            const float mn = fmaxf(m, top), base = mn == -INFINITY ? 0.f : mn, old = exp2f(m - base);
            const float al = exp2f(mk - base);
            float sum = al * lk;
#pragma unroll
            for (int x = 1; x < kWave; x <<= 1) sum += __shfl_xor(sum, x, kWave);
            l = l * old + sum;
            o = make_float4(o.x * old, o.y * old, o.z * old, o.w * old);
            m = mn;
            for (int k0 = 0; k0 < cnt; k0 += 4 * PW) {
                float4 v[4];
                float f[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int k = k0 + u * PW + sub;
                    v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (k < cnt) v[u] = piece(po + (size_t)(c0 + k) * rows * D);
                    f[u] = __shfl(al, min(k, kWave - 1), kWave);
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (k0 + u * PW + sub >= cnt) continue;
                    o.x = fmaf(f[u], v[u].x, o.x);
                    o.y = fmaf(f[u], v[u].y, o.y);
                    o.z = fmaf(f[u], v[u].z, o.z);
                    o.w = fmaf(f[u], v[u].w, o.w);
                }
            }
        }
#pragma unroll
        for (int x = LPR; x < kWave; x <<= 1) {
            o.x += __shfl_xor(o.x, x, kWave);
            o.y += __shfl_xor(o.y, x, kWave);
            o.z += __shfl_xor(o.z, x, kWave);
            o.w += __shfl_xor(o.w, x, kWave);
        }
        if (SHARED) {
            if (sub == 0) *(float4*)&s_o[w][d] = o;
            if (lane == 0) {
                s_ml[w][0] = m;
                s_ml[w][1] = l;
            }
            __syncthreads();
            if (w != 0) return;
            const float mt = fmaxf(fmaxf(s_ml[0][0], s_ml[1][0]), fmaxf(s_ml[2][0], s_ml[3][0]));
            const float base = mt == -INFINITY ? 0.f : mt;
            l = 0.f;
            o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float4 t = *(const float4*)&s_o[x][d];
                const float f = exp2f(s_ml[x][0] - base);
                l = fmaf(f, s_ml[x][1], l);
                o.x = fmaf(f, t.x, o.x);
                o.y = fmaf(f, t.y, o.y);
                o.z = fmaf(f, t.z, o.z);
                o.w = fmaf(f, t.w, o.w);
            }
        }
        if (sub == 0) finish(row, o, l);
    }
}

template <typename TIO, typename TC>
void launch_plain(const AttnArgs& a, const AttnPlan& p, const AttnWorkspace& ws, int row_blocks, hipStream_t stream) {
    const dim3 grid((unsigned)((long long)p.parts * p.readers));
    if (a.D <= 64)
        hipLaunchKernelGGL((attn_plain_kernel<TIO, TC, 1>), grid, dim3(256), 0, stream, a, p, ws, row_blocks);
    else if (a.D <= 128)
        hipLaunchKernelGGL((attn_plain_kernel<TIO, TC, 2>), grid, dim3(256), 0, stream, a, p, ws, row_blocks);
    else
        hipLaunchKernelGGL((attn_plain_kernel<TIO, TC, 4>), grid, dim3(256), 0, stream, a, p, ws, row_blocks);
}

template <typename TIO, int LPR>
void launch_join_lpr(const AttnArgs& a, const AttnPlan& p, const AttnWorkspace& ws, hipStream_t stream) {
    const int rows = a.T * a.H;
    const long long all = (long long)a.batch * rows;
    const int rw = all <= 1024 ? 0 : all <= 16384 ? 1 : 4;
    const int per = rw == 4 ? 16 * (kWave / LPR) : rw == 1 ? 4 : 1;  // rows of a work-group
    const int blocks = (rows + per - 1) / per;
    const dim3 grid((unsigned)((long long)a.batch * blocks));
    if (rw == 0)
        hipLaunchKernelGGL((attn_join_kernel<TIO, LPR, 0>), grid, dim3(256), 0, stream, a, p, ws, blocks);
    else if (rw == 1)
        hipLaunchKernelGGL((attn_join_kernel<TIO, LPR, 1>), grid, dim3(256), 0, stream, a, p, ws, blocks);
    else
        hipLaunchKernelGGL((attn_join_kernel<TIO, LPR, 4>), grid, dim3(256), 0, stream, a, p, ws, blocks);
}

template <typename TIO>
void launch_join(const AttnArgs& a, const AttnPlan& p, const AttnWorkspace& ws, hipStream_t stream) {
    if (a.D <= 64)
        launch_join_lpr<TIO, 16>(a, p, ws, stream);
    else if (a.D <= 128)
        launch_join_lpr<TIO, 32>(a, p, ws, stream);
    else
        launch_join_lpr<TIO, 64>(a, p, ws, stream);
}

// Whether the matrix kernels take the shape: 32-bit row numbers into the pool, and
// 16-byte rows of 64 or 128 elements (their alignment is looked at per call)
bool matrix_shape(const tsv_attn_shape* s) {
    return (s->head_dim == 64 || s->head_dim == 128) && !(s->flags & TSV_FLAG_FORCE_GENERIC) &&
           (long long)s->n_pages * s->n_kv_heads * s->page_size < (1LL << 32);
}

// Rows of a work-group: 16 (attn_rows_kernel, attn_f32_kernel), 64 (both tile
// kernels), 128 (attn_tiles_kernel) or 8 (plain). Of bf16 trees, 128 rows cost less
// per row (caches of 2200 positions, 8 key heads: 16 items of 252 rows 68 us against
// 83, 32 items of 92 rows 82 against 102), but not if that leaves a fifth more rows
// empty (48 items of 180 rows 194 against 171), and not where few items have to fill
// the GPU, whose time is latency (1 item of 252 rows 27 against 21, 4 items 38
// against 35; 8 items 53 against 55).
int block_rows_of(const tsv_attn_shape* s, bool matrix) {
    if (!matrix) return kRows;
    const int R = s->n_nodes * (s->n_heads / s->n_kv_heads);
    if (R <= 16) return 16;
    if (s->in_dtype == TSV_F32) return 64;
    const int r64 = (R + 63) / 64 * 64, r128 = (R + 127) / 128 * 128;
    return r128 * 5 > r64 * 6 || (long long)s->batch * s->n_kv_heads <= 64 ? 64 : 128;
}

// Work-groups wanted, for x of them that would run without any split (an item's
// last part is half empty on average, so about want + x / 2 parts are whole).
//   tiles  two fit a compute unit: whole rounds of 512, so that no round is nearly
//          empty, with want at least x (32 trees of 63 nodes, x = 512: 153 us for
//          512, 133 for 768, 138 for 1024, and the join rises with want). From
//          1024 on the items fill the GPU, and only the longest are cut.
//   rows   few parts while they fill one round, for the join's sake (a cache of
//          65533, x = 8: 58 us for 512, 62 for 1024), small ones where many
//          items of different lengths share the GPU (64 items, x = 512: 122 us for
//          1024, 118 for 2048)
int want_of(bool matrix, int block_rows, long long x) {
    if (!matrix) return 1024;
    if (block_rows == 16) return x <= 128 ? 512 : x >= 512 ? 2048 : (int)(4 * x);
    return x >= 1024 ? 1024 : (int)((3 * x / 2 + 511) / 512 * 512 - x / 2);
}

AttnPlan plan_of(const tsv_attn_shape* s, bool matrix, int* block_rows, int* row_blocks) {
    *block_rows = block_rows_of(s, matrix);
    *row_blocks = (int)(((long long)s->n_nodes * (s->n_heads / s->n_kv_heads) + *block_rows - 1) / *block_rows);
    const int readers = s->n_kv_heads * *row_blocks;
    AttnPlan p = attn_plan(s->batch, (long long)s->max_pages * s->page_size, readers, kAttnMinKeys,
                           want_of(matrix, *block_rows, (long long)s->batch * readers));
    // the tile kernel's work-groups are few and long, so that none should start late
    // (32 trees of 63 nodes: 124 us, 137 in the items' order)
    p.sorted = p.split && matrix && *block_rows > 16 && s->batch > 1 && s->batch <= kWave;
    return p;
}

}  // namespace

// both kernels' needs: which of them runs depends on the pointers too
uint64_t attn_verify_workspace_bytes(const tsv_attn_shape* s) {
    uint64_t most = 0;
    for (int matrix = 0; matrix <= (int)matrix_shape(s); ++matrix) {
        int br, rb;
        const uint64_t n = attn_workspace_bytes(plan_of(s, matrix, &br, &rb), s->n_nodes, s->n_heads, s->head_dim);
        if (n > most) most = n;
    }
    return most;
}

long long attn_verify_blocks(const tsv_attn_shape* s) {
    long long most = (long long)s->batch * (((long long)s->n_nodes * s->n_heads + 15) / 16);  // the join
    for (int matrix = 0; matrix <= (int)matrix_shape(s); ++matrix) {
        int br, rb;
        const AttnPlan p = plan_of(s, matrix, &br, &rb);
        const long long n = (long long)p.parts * p.readers + 8 * rb;  // (the tile kernel rounds its units up to eight)
        if (n > most) most = n;
    }
    return most;
}

hipError_t launch_attn_verify(const AttnArgs& a, const tsv_attn_shape* s, void* workspace, hipStream_t stream) {
    const uintptr_t all = (uintptr_t)a.q | (uintptr_t)a.k | (uintptr_t)a.v | (uintptr_t)a.o | (uintptr_t)a.k_cache | (uintptr_t)a.v_cache;
    const bool matrix = matrix_shape(s) && all % 16 == 0;
    int block_rows, row_blocks;
    const AttnPlan p = plan_of(s, matrix, &block_rows, &row_blocks);
    const AttnWorkspace ws = attn_workspace(workspace, p, a.T, a.H, a.D);
    const bool bf16 = s->in_dtype == TSV_BF16, e4m3 = s->cache_dtype == TSV_E4M3;
    if (matrix && !bf16)
        launch_attn_f32(a, e4m3, p, ws, block_rows, row_blocks, stream);
    else if (matrix)
        launch_attn_mfma(a, e4m3, p, ws, block_rows, row_blocks, stream);
    else if (bf16 && e4m3)
        launch_plain<uint16_t, uint8_t>(a, p, ws, row_blocks, stream);
    else if (bf16)
        launch_plain<uint16_t, uint16_t>(a, p, ws, row_blocks, stream);
    else if (e4m3)
        launch_plain<float, uint8_t>(a, p, ws, row_blocks, stream);
    else
        launch_plain<float, float>(a, p, ws, row_blocks, stream);
    if (p.split) {
        if (bf16)
            launch_join<uint16_t>(a, p, ws, stream);
        else
            launch_join<float>(a, p, ws, stream);
    }
    return hipGetLastError();
}

}  // namespace tsv
