// attn_prefill.hip -- attention of packed rows over the paged cache: the plain fp32
// kernel (any head_dim up to 256, any types), the join of the parts, and the choice of
// the kernel.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = 2^(scale log2(e) q_i . k_j - m_i)
// over the positions j <= cache_len + i that row i sees, in one pass with a running maximum
// m_i and sum; parts of the keys (attn_chunk.hpp) are joined by
//   o = sum_k 2^(m_k - m) o_k / sum_k 2^(m_k - m) l_k,  m = max_k m_k.
//
// Plain kernel: a work-group takes kRows rows (token, query head) of one key head; its
// waves take 64 keys each in turn. Scores: a lane per key, the rows' q from LDS (the same
// for all lanes). Values: lanes over the head_dim, weights from LDS. Bound by the vector
// ALU and the LDS broadcasts (4 D operations per row and key): 512
// tokens, 32 query and 8 key heads of 80, 123 us (11 TFLOP/s), 16 and 4 heads of 256 201 us; 32
// single tokens over 2200 positions each, heads of 80, 283 us.
#include "attn_chunk.hpp"

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

template <typename TIO, typename TC, int DV>
__global__ __launch_bounds__(256) void chunk_plain_kernel(ChunkArgs a, ChunkPlan plan, ChunkWorkspace ws) {
    __shared__ float s_q[kRows][256], s_p[4][kRows][kWave], s_o[kRows][256], s_ml[4][kRows][2];
    __shared__ long long s_off[4][kWave];
    const int tid = threadIdx.x, lane = tid & (kWave - 1), w = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int hk = blockIdx.x % a.Hk;
    const ChunkUnit u = find_unit<false>(a, plan, blockIdx.x / a.Hk);
    if (blockIdx.x == 0 && w == 0) chunk_status(a, plan, u.bad);
    if (!u.ok) return;
    if (chunk_check<256>(a, u, hk, ws)) return;
    const ChunkKeys kk = chunk_keys(a, plan, u);
    const int D = a.D, g = plan.g, R = u.n * g, row0 = u.block * kRows;
    for (int i = tid; i < kRows * D; i += 256) {
        const int r = row0 + i / D;
        s_q[i / D][i % D] = r < R ? Elem<TIO>::ld((const TIO*)a.q, (((size_t)u.start + r / g) * a.H + hk * g + r % g) * D + i % D) : 0.f;
    }
    __syncthreads();
    float m[kRows], l[kRows], o[kRows][DV];
    int own[kRows];  // the rows' positions
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        own[r] = u.old + min(row0 + r, R - 1) / g;
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int i = 0; i < DV; ++i) o[r][i] = 0.f;
    }
    const TC* kp = (const TC*)a.k_cache;
    const TC* vp = (const TC*)a.v_cache;
    for (int t0 = kk.k0 + w * kWave; t0 < kk.k1; t0 += 4 * kWave) {
        const int v = t0 + lane, n = min(kWave, kk.k1 - t0);
        long long key = -1;
        int pos = 0;
        float ks = 1.f, vs = 1.f;
        if (v < kk.k1) {
            pos = chunk_pos(kk, v);
            const int page = page_of(pos, a.div);
            key = ((long long)a.page_table[(size_t)u.seq * a.max_pages + page] * a.Hk + hk) * a.page_size + (pos - page * a.page_size);
            if (a.k_scale) {
                ks = a.k_scale[key];
                vs = a.v_scale[key];
            }
        }
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
        s_off[w][lane] = key;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const bool seen = key >= 0 && pos <= own[r] && (own[r] - pos < a.window || pos < a.sinks);
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
            s_p[w][r][lane] = p * vs;
            if (!seen) s_p[w][r][lane] = 0.f;  // (a scale that is not finite)
        }
        wave_sync();
        for (int j = 0; j < n; ++j) {
            const long long at = s_off[w][j];
#pragma unroll
            for (int i = 0; i < DV; ++i) {
                const int d = lane + i * kWave;
                if (d >= D) continue;
                const float x = elem<TC>(vp, (size_t)at * D + d);
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    // a key that row r does not see has weight 0, also where its value is not finite
                    const float p = s_p[w][r][j];
                    o[r][i] = p == 0.f ? o[r][i] : fmaf(p, x, o[r][i]);
                }
            }
        }
        wave_sync();
    }
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
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        if (row0 + r >= R) break;
        if (u.parts > 1) {
            const size_t at = ((size_t)u.slot * a.Hk + hk) * kRows + r;
            if (tid < D) ws.o[at * D + tid] = s_o[r][tid];
            if (tid < 2) ws.ml[at * 2 + tid] = tid ? lt[r] : mt[r];
        } else if (tid < D) {
            const int row = row0 + r;
            Elem<TIO>::st((TIO*)a.o, (((size_t)u.start + row / g) * a.H + hk * g + row % g) * D + tid, s_o[r][tid] / lt[r]);
        }
    }
}

// Lanes take 4 elements of a row each, LPR lanes a row. A work-group has `per` rows of a
// block; where it has more groups of lanes than rows, several share a row's parts. Few blocks
// have many parts, and their rows work-groups of their own (64 tokens over 30000 positions,
// 2048 rows of 32 parts each: 53 us with 32 rows a work-group, 15 with 2); but a work-group's
// search for its block costs as much as some rows, so there are some 2000 of them.
template <typename TIO, int LPR>
__global__ __launch_bounds__(256) void chunk_join_kernel(ChunkArgs a, ChunkPlan plan, ChunkWorkspace ws, int per, int groups) {
    constexpr int kAt = 256 / LPR, kLoads = 8;
    __shared__ __attribute__((aligned(16))) float s_o[kAt][LPR * 4];
    __shared__ float s_ml[kAt][2];
    const int tid = threadIdx.x, unit = blockIdx.x / groups, hk = unit % a.Hk, grp = tid / LPR, d = tid % LPR * 4;
    const ChunkUnit u = find_unit<true>(a, plan, unit / a.Hk);
    if (!u.ok || ws.bad[(size_t)u.slot * a.Hk + hk]) return;
    const int D = a.D, g = plan.g, row0 = u.block * plan.rows, rows = min(u.n * g - row0, plan.rows);
    int share = 1;  // groups of a row
    while (2 * share * min(per, rows) <= kAt) share *= 2;
    const int first = blockIdx.x % groups * per;
    const bool whole = D % 4 == 0 && (uintptr_t)a.o % (4 * sizeof(TIO)) == 0;  // pieces of four, aligned
    auto piece = [&](const float* p) { return d >= D ? make_float4(0.f, 0.f, 0.f, 0.f) : whole ? ld4<true>(p, 4) : ld4<false>(p, D - d); };
    for (int r0 = first; r0 < min(rows, first + per); r0 += kAt / share) {
        const int r = min(r0 + grp / share, rows - 1);
        float m = -INFINITY, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k0 = grp % share; k0 < u.parts; k0 += kLoads * share) {
            float mk[kLoads], lk[kLoads];
            float4 v[kLoads];
            float mn = m;
#pragma unroll
            for (int x = 0; x < kLoads; ++x) {
                mk[x] = -INFINITY;
                lk[x] = 0.f;
                v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (k0 + x * share >= u.parts) continue;
                const size_t at = ((size_t)(u.slot + k0 + x * share) * a.Hk + hk) * plan.rows + r;
                mk[x] = ws.ml[at * 2];
                lk[x] = ws.ml[at * 2 + 1];
                v[x] = piece(ws.o + at * D + d);
            }
#pragma unroll
            for (int x = 0; x < kLoads; ++x) mn = fmaxf(mn, mk[x]);
            const float base = mn == -INFINITY ? 0.f : mn, old = exp2f(m - base);
            l *= old;
            o = make_float4(o.x * old, o.y * old, o.z * old, o.w * old);
#pragma unroll
            for (int x = 0; x < kLoads; ++x) {
                const float f = exp2f(mk[x] - base);
                l = fmaf(f, lk[x], l);
                o.x = fmaf(f, v[x].x, o.x);
                o.y = fmaf(f, v[x].y, o.y);
                o.z = fmaf(f, v[x].z, o.z);
                o.w = fmaf(f, v[x].w, o.w);
            }
            m = mn;
        }
        if (share > 1) {  // (one turn of this loop)
            *(float4*)&s_o[grp][d] = o;
            if (d == 0) {
                s_ml[grp][0] = m;
                s_ml[grp][1] = l;
            }
            __syncthreads();
            float mt = -INFINITY;
            for (int x = 0; x < share; ++x) mt = fmaxf(mt, s_ml[grp / share * share + x][0]);
            l = 0.f;
            o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int x = 0; x < share; ++x) {
                const int from = grp / share * share + x;
                const float f = exp2f(s_ml[from][0] - (mt == -INFINITY ? 0.f : mt));
                const float4 v = *(const float4*)&s_o[from][d];
                l = fmaf(f, s_ml[from][1], l);
                o.x = fmaf(f, v.x, o.x);
                o.y = fmaf(f, v.y, o.y);
                o.z = fmaf(f, v.z, o.z);
                o.w = fmaf(f, v.w, o.w);
            }
        }
        if (d >= D || grp % share || r0 + grp / share >= min(rows, first + per)) continue;
        const int row = row0 + r, token = page_of(row, plan.by_g);
        TIO* to = (TIO*)a.o + (((size_t)u.start + token) * a.H + hk * g + (row - token * g)) * D + d;
        const float f[4] = {o.x / l, o.y / l, o.z / l, o.w / l};
        if (whole) {
            if constexpr (sizeof(TIO) == 4)
                *(float4*)to = make_float4(f[0], f[1], f[2], f[3]);
            else
                *(uint2*)to = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (d + e < D) Elem<TIO>::st(to, e, f[e]);
        }
    }
}

template <typename TIO, typename TC>
void launch_plain(const ChunkArgs& a, const ChunkPlan& p, const ChunkWorkspace& ws, dim3 grid, hipStream_t stream) {
    if (a.D <= 64)
        hipLaunchKernelGGL((chunk_plain_kernel<TIO, TC, 1>), grid, dim3(256), 0, stream, a, p, ws);
    else if (a.D <= 128)
        hipLaunchKernelGGL((chunk_plain_kernel<TIO, TC, 2>), grid, dim3(256), 0, stream, a, p, ws);
    else
        hipLaunchKernelGGL((chunk_plain_kernel<TIO, TC, 4>), grid, dim3(256), 0, stream, a, p, ws);
}

// Work-groups of the join, for the blocks that may be cut
struct Join {
    int per, groups;  // rows of a work-group, work-groups of a block
    long long blocks;  // work-groups
};
Join join_of(const ChunkPlan& p, long long T, int H, int Hk, int batch) {
    const long long blocks = chunk_blocks(p, T, H / Hk, batch), units = (blocks < p.want / Hk ? blocks : p.want / Hk) * Hk;
    Join j;
    for (j.per = 1; j.per < 32 && units * ((p.rows + j.per - 1) / j.per) > 2048;) j.per *= 2;
    j.groups = (p.rows + j.per - 1) / j.per;
    j.blocks = units * j.groups;
    return j;
}

template <typename TIO>
void launch_join(const ChunkArgs& a, const ChunkPlan& p, const ChunkWorkspace& ws, hipStream_t stream) {
    const Join j = join_of(p, a.T, a.H, a.Hk, a.batch);
    const dim3 grid((unsigned)j.blocks);
    if (a.D <= 64)
        hipLaunchKernelGGL((chunk_join_kernel<TIO, 16>), grid, dim3(256), 0, stream, a, p, ws, j.per, j.groups);
    else if (a.D <= 128)
        hipLaunchKernelGGL((chunk_join_kernel<TIO, 32>), grid, dim3(256), 0, stream, a, p, ws, j.per, j.groups);
    else
        hipLaunchKernelGGL((chunk_join_kernel<TIO, 64>), grid, dim3(256), 0, stream, a, p, ws, j.per, j.groups);
}

// Whether the matrix kernels take the shape: 32-bit row numbers into the pool, and
// 16-byte rows of 64 or 128 elements (their alignment is looked at per call)
bool matrix_shape(const tsv_attn_shape* s) {
    return (s->head_dim == 64 || s->head_dim == 128) && !(s->flags & TSV_FLAG_FORCE_GENERIC) &&
           (long long)s->n_pages * s->n_kv_heads * s->page_size < (1LL << 32);
}

// Rows of a block, by those that the sequences (empty ones among them) have of a key head on
// average, since the host does not know their lengths:
//   bf16   16 (chunk_rows_kernel) up to 16, as single tokens do, otherwise 128
//          (chunk_tiles_kernel). 8 single tokens over 1000 positions 15.9 us, 22.8 in blocks of
//          128; 32 chains of 5 tokens, 20 rows, over 4096 114 us, 125 in blocks of 16
//   fp32   16 up to 32 rows, otherwise 64. 32 single tokens over 4096 positions 201 us, 235 in
//          blocks of 64; 32 chains of 8 tokens 255 and 319, of 16 tokens 438 in blocks of 16, 331
//   plain  8
// So a long chunk beside many single tokens goes in blocks of 16 (512 tokens behind 30000
// positions and 256 behind 1000: 1268 us, 487 as two calls; beside 64 of them 335 and 346).
// Work-groups wanted, for x of them that would run without any cut:
//   tiles  one round of two a compute unit (a chunk of 509 over 33258 positions: 312 us, 362
//          for half as many, 325 for twice)
//   rows   few parts while they fill one round, small ones where many items of different
//          lengths share the GPU (us for half as many, as here, and twice: 1 token over 65532
//          positions 62, 64, 68; 8 over 4000 34, 34, 38; 32 over 2200 62, 65, 69; 64 over 17 to
//          8190 in e4m3 118, 115, 122)
// No block is cut that has no more than 512 keys, nor where a window bounds every block and
// blocks fill the GPU (64 tokens, windows of 1021: 50.6 us, 65.2 cut, most of it a second launch
// that finds little to join; 4096 tokens in a window of 1024 84 and 88). A window that is longer
// than most caches bounds little: 63 tokens behind 100 positions and one behind 65000 take 682 us
// in a window of 65536, 114 without one.
ChunkPlan plan_of(const tsv_attn_shape* s, bool matrix, int window, int sinks) {
    ChunkPlan p;
    const int g = s->n_heads / s->n_kv_heads;
    const long long T = s->n_nodes, rows = T * g, items = s->batch < T ? s->batch : T, x = items * s->n_kv_heads;
    const bool f32 = s->in_dtype == TSV_F32;
    p.rows = !matrix ? kRows : rows <= (f32 ? 32LL : 16LL) * s->batch ? 16 : f32 ? 64 : 128;
    p.want = !matrix ? 1024 : p.rows > 16 || x <= 128 ? 512 : x >= 512 ? 2048 : (int)(4 * x);
    p.min_keys = 256;
    for (p.shift = 0; 1 << p.shift < p.rows;) ++p.shift;
    p.g = g;
    p.by_g = page_div(g);
    p.tokens = (p.rows + g - 2) / g + 1;
    p.share = (float)s->n_kv_heads / (float)p.want * (1.f + 0x1p-20f);
    const long long blocks = rows / p.rows > items ? rows / p.rows : items;
    long long longest = (long long)s->max_pages * s->page_size;
    if (window > 0 && longest > (long long)window + sinks + p.rows) longest = (long long)window + sinks + p.rows;
    p.split = longest > 2 * p.min_keys && s->n_kv_heads <= p.want && !(window > 0 && blocks * s->n_kv_heads >= 512);
    // long work-groups should not start last (their order costs each a search of a microsecond: 16
    // mixed e4m3 chunks 295 us, 318 in the sequences' order)
    p.sorted = p.rows > 16 && s->batch > 1 && s->batch <= kWave;
    return p;
}

}  // namespace

// both kernels' needs, without a window: which of them runs depends on the pointers too, and
// a window cuts no more
uint64_t attn_prefill_workspace_bytes(const tsv_attn_shape* s) {
    uint64_t most = 0;
    for (int matrix = 0; matrix <= (int)matrix_shape(s); ++matrix) {
        const uint64_t n = chunk_workspace_bytes(plan_of(s, matrix, 0, 0), s->n_kv_heads, s->head_dim);
        if (n > most) most = n;
    }
    return most;
}

long long attn_prefill_blocks(const tsv_attn_shape* s) {
    long long most = 0;
    for (int matrix = 0; matrix <= (int)matrix_shape(s); ++matrix) {
        const ChunkPlan p = plan_of(s, matrix, 0, 0);
        const long long units = chunk_units(p, s->n_nodes, s->n_heads / s->n_kv_heads, s->batch, s->n_kv_heads) * s->n_kv_heads;
        const long long join = join_of(p, s->n_nodes, s->n_heads, s->n_kv_heads, s->batch).blocks;
        if (units > most) most = units;
        if (join > most) most = join;
    }
    return most;
}

hipError_t launch_attn_prefill(const ChunkArgs& a, const tsv_attn_shape* s, void* workspace, hipStream_t stream) {
    const uintptr_t all = (uintptr_t)a.q | (uintptr_t)a.o | (uintptr_t)a.k_cache | (uintptr_t)a.v_cache;
    const bool matrix = matrix_shape(s) && all % 16 == 0;
    const ChunkPlan p = plan_of(s, matrix, a.window == 0x7fffffff ? 0 : a.window, a.sinks);
    const ChunkWorkspace ws = chunk_workspace(workspace, p, a.Hk, a.D);
    const long long units = chunk_units(p, a.T, a.H / a.Hk, a.batch, a.Hk) * a.Hk;
    const dim3 grid((unsigned)(units > 0 ? units : 1));
    const bool bf16 = s->in_dtype == TSV_BF16, e4m3 = s->cache_dtype == TSV_E4M3;
    if (matrix && !bf16)
        launch_chunk_f32(a, e4m3, p, ws, grid, stream);
    else if (matrix)
        launch_chunk_mfma(a, e4m3, p, ws, grid, stream);
    else if (bf16 && e4m3)
        launch_plain<uint16_t, uint8_t>(a, p, ws, grid, stream);
    else if (bf16)
        launch_plain<uint16_t, uint16_t>(a, p, ws, grid, stream);
    else if (e4m3)
        launch_plain<float, uint8_t>(a, p, ws, grid, stream);
    else
        launch_plain<float, float>(a, p, ws, grid, stream);
    if (p.split && a.T > 0) {
        if (bf16)
            launch_join<uint16_t>(a, p, ws, stream);
        else
            launch_join<float>(a, p, ws, stream);
    }
    return hipGetLastError();
}

}  // namespace tsv
