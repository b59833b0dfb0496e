// attn_f32.hip -- tree attention on fp32 matrix instructions (fp32 inputs,
// head_dim 64 or 128, cache in fp32 or e4m3).
//
// As in attn_mfma.hip the scores are formed transposed, S^T = K Q^T, on 16x16x4
// products: a lane holds the keys 4 g + r (g = l / 16) of one row l % 16, and the
// weights P are the next product's operand as they are, O^T = V^T P^T, if its
// step r takes key 4 g + r from lane group g. Which element of the head each k-slot
// of K Q^T stands for is free, so a lane reads K and Q as 16-byte pieces (d = 16 j +
// 4 g + e in step 4 j + e); so is which row of O^T stands for which d, and a 16-byte
// piece of V feeds four products (tile 4 h + c: d = 64 h + 4 i + c for its row i).
//
// 64 keys at a time are shared in LDS by four waves; WK 1: of 16 rows each, WK 4: of
// the same 16 rows, a quarter of the keys each, which meet at the end. Bound by the
// fp32 matrix rate and, for single tokens, the cache's bytes: 32 tokens over 2200
// positions each, 8 key heads of 128 (577 MB), 111 us (5.2 TB/s; 359 us in the
// plain kernel), 4 trees of 63 nodes over them 106 us (85 of 153 TFLOP/s, the matrix
// unit busy 72% of the cycles; 721 us).
#include <cfloat>

#include "attn_lanes.hpp"

namespace tsv {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

template <int D, bool E4M3, int WK>
__global__ __launch_bounds__(256, 2) void attn_f32_kernel(AttnArgs a, AttnPlan plan, AttnWorkspace ws, int row_blocks) {
    constexpr int M = 64 / WK, kS = D + 4, NX = 4 / WK;
    __shared__ __attribute__((aligned(8))) int s_red[6];
    __shared__ Part s_part;
    __shared__ __attribute__((aligned(16))) float s_K[kTileKeys * kS], s_V[kTileKeys * kS];  // s_K: then the waves' outputs
    __shared__ __attribute__((aligned(16))) float s_ks[kTileKeys], s_vs[kTileKeys], s_ml[4][16][2];
    __shared__ uint32_t s_row[2][kTileKeys];
    __shared__ uint32_t s_odd[32];  // nodes whose values are not all finite
    extern __shared__ uint32_t s_anc[];  // [nodes of the block][words of T bits]
    int* s_par = (int*)s_K;  // before the tiles (1024 nodes at most)
    const int tid = threadIdx.x, lane = tid & (kWave - 1), w = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int l16 = lane & 15, lg = lane >> 4, wr = w / WK, wk = w % WK;
    // units as in the bf16 tile kernel
    const int turn = blockIdx.x / 8, rb = turn % row_blocks, unit = turn / row_blocks * 8 + blockIdx.x % 8;
    const int hk = unit % a.Hk;
    Part pt = find_part<256>(a.cache_len, a.batch, a.room, plan, unit / a.Hk, false, s_red, &s_part);
    if (!pt.ok) return;
    pt = uniform(pt);
    const int part = pt.base + pt.k;
    const int b = pt.item, T = a.T, H = a.H, g = H / a.Hk, R = T * g, row0 = rb * M;
    const bool last = pt.k == pt.n - 1;
    int st = pt.bad_len ? kStBadCache : 0;
    const int first = row0 / g, last_node = min(R - 1, row0 + M - 1) / g, words = (T + 31) / 32;
    const int k0 = pt.k * pt.keys, k1 = last ? pt.len : min(pt.len, k0 + pt.keys);
    int page = 0;  // of this lane's key, in the first wave
    if (w == 0 && k1 > k0 && a.n_pages > 0) page = a.page_table[(size_t)b * a.max_pages + page_of(min(k0 + lane, k1 - 1), a.div)];
    if (last) st |= tree_words<256>(a.parent + (size_t)b * T, T, first, last_node - first + 1, words, s_par, s_anc);
    if (tid < 32) s_odd[tid] = 0;

    // this lane's row
    const int row = row0 + 16 * wr + l16, node = min(row, R - 1) / g;
    float4 q[D / 16];
    {
        const float* qp = (const float*)a.q + (((size_t)b * T + node) * H + hk * g + min(row, R - 1) % g) * D + 4 * lg;
        const float sign = a.scale_log2 < 0.f ? -1.f : 1.f;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            q[j] = gload((const float4*)(qp + 16 * j));
            q[j] = make_float4(sign * q[j].x, sign * q[j].y, sign * q[j].z, sign * q[j].w);
        }
    }
    const float c = score_factor(a);
    float base = -FLT_MAX, l = 0.f;  // as in the bf16 tile kernel
    f32x4 o[D / 16];
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[i] = f32x4{0.f, 0.f, 0.f, 0.f};

    // One tile of keys in LDS, `limit` of them. TREE: keys j0 + ... of the tree
    auto take = [&](auto tree, int limit, int j0) {
        constexpr bool TREE = decltype(tree)::value, SCALED = E4M3 && !TREE;
        f32x4 s[NX];
#pragma unroll
        for (int x = 0; x < NX; ++x) s[x] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
#pragma unroll
            for (int x = 0; x < NX; ++x) s[x] = mma4(*(const float4*)&s_K[(16 * (x + wk) + l16) * kS + 16 * j + 4 * lg], q[j], s[x]);
            if (j % 2) __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int x = 0; x < NX; ++x) {
            const int j = 16 * (x + wk) + 4 * lg;  // key of s[x][0]
            if (SCALED) s[x] *= *(const f32x4*)&s_ks[j];
            if (TREE) {
                const uint32_t bits = s_anc[(node - first) * words + min((j0 + j) / 32, words - 1)] >> ((j0 + j) % 32);
#pragma unroll
                for (int r = 0; r < 4; ++r) s[x][r] = j + r < limit && (bits >> r & 1) ? s[x][r] : -INFINITY;
            } else if (limit < kTileKeys) {
#pragma unroll
                for (int r = 0; r < 4; ++r) s[x][r] = j + r < limit ? s[x][r] : -INFINITY;
            }
        }
        float mx = max3(max3(s[0][0], s[0][1], s[0][2]), s[0][3], s[0][3]);
#pragma unroll
        for (int x = 1; x < NX; ++x) mx = max3(max3(mx, s[x][0], s[x][1]), s[x][2], s[x][3]);
        if (__ballot(fmaf(mx, c, -base) > kSlack)) {
            const float top = row_max(mx);  // a row moves by its own scores alone: its bits do not follow from its neighbours'
            const float to = fmaf(top, c, -base) > kSlack ? top * c : base, al = __builtin_amdgcn_exp2f(base - to);
            l *= al;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) o[i] *= al;
            base = to;
        }
#pragma unroll
        for (int x = 0; x < NX; ++x) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                s[x][r] = __builtin_amdgcn_exp2f(fmaf(s[x][r], c, -base));
                l += s[x][r];  // of this lane's keys; the lanes of a row meet at the end
            }
            if (SCALED) s[x] *= *(const f32x4*)&s_vs[16 * (x + wk) + 4 * lg];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
#pragma unroll
                for (int h = 0; h < D / 64; ++h) {
                    const float4 v = *(const float4*)&s_V[(16 * (x + wk) + 4 * lg + r) * kS + 64 * h + 4 * l16];
                    o[4 * h] = __builtin_amdgcn_mfma_f32_16x16x4f32(v.x, s[x][r], o[4 * h], 0, 0, 0);
                    o[4 * h + 1] = __builtin_amdgcn_mfma_f32_16x16x4f32(v.y, s[x][r], o[4 * h + 1], 0, 0, 0);
                    o[4 * h + 2] = __builtin_amdgcn_mfma_f32_16x16x4f32(v.z, s[x][r], o[4 * h + 2], 0, 0, 0);
                    o[4 * h + 3] = __builtin_amdgcn_mfma_f32_16x16x4f32(v.w, s[x][r], o[4 * h + 3], 0, 0, 0);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    // the tree's own keys, up to the block's last node; values that are not finite
    // enter as 0 and are added for the rows that see them
    auto take_tree = [&]() {
        if (!last || st) return;
        const size_t stride = (size_t)a.Hk * D;
        const float* kp = (const float*)a.k + ((size_t)b * T * a.Hk + hk) * D;
        const float* vp = (const float*)a.v + ((size_t)b * T * a.Hk + hk) * D;
        for (int j0 = 0; j0 <= last_node; j0 += kTileKeys) {
            lds_barrier();
            for (int i = tid; i < kTileKeys * (D / 4); i += 256) {
                const int key = i / (D / 4), d = i % (D / 4) * 4;
                float4 kf = make_float4(0.f, 0.f, 0.f, 0.f), vf = kf;
                if (j0 + key < T) {
                    kf = gload((const float4*)(kp + (size_t)(j0 + key) * stride + d));
                    vf = gload((const float4*)(vp + (size_t)(j0 + key) * stride + d));
                }
                if (nonfinite(vf.x) || nonfinite(vf.y) || nonfinite(vf.z) || nonfinite(vf.w)) {
                    atomicOr(&s_odd[(j0 + key) / 32], 1u << ((j0 + key) % 32));
                    vf = make_float4(nonfinite(vf.x) ? 0.f : vf.x, nonfinite(vf.y) ? 0.f : vf.y, nonfinite(vf.z) ? 0.f : vf.z,
                                     nonfinite(vf.w) ? 0.f : vf.w);
                }
                *(float4*)&s_K[key * kS + d] = kf;
                *(float4*)&s_V[key * kS + d] = vf;
            }
            lds_barrier();
            take(std::true_type(), T - j0, j0);
        }
        for (int x = 0; x < (wk == 0 ? words : 0); ++x) {
            if (!s_odd[x]) continue;
            for (int j = 0; j < 32; ++j) {
                if (!(s_odd[x] & s_anc[(node - first) * words + x] & (1u << j))) continue;
                const float* v = vp + (size_t)(32 * x + j) * stride + 16 * lg;
#pragma unroll
                for (int h = 0; h < D / 64; ++h)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float f = gload(v + 64 * h + 4 * r + e);
                            if (nonfinite(f)) o[4 * h + e][r] += f;
                        }
            }
        }
    };

    int bad = 0;
    if (k1 > k0 && a.n_pages > 0) {
        constexpr int EB = E4M3 ? 1 : 4;
        constexpr int L = kTileKeys * D * EB / 16 / 256;  // 16-byte loads of K, and of V, per thread
        constexpr int RR = 256 / (D * EB / 16);           // rows that one of them covers
        const int32_t* table = a.page_table + (size_t)b * a.max_pages;
        uint4 rk[L], rv[L];
        float rks = 1.f, rvs = 1.f;
        const int prow = tid / (D * EB / 16), pcol = tid % (D * EB / 16) * 16;
        // the first wave looks up pages and rows, for all
        auto key_of = [&](int t) { return min(t + lane, k1 - 1); };
        auto look_up = [&](int t) {
            if (w == 0) page = table[page_of(key_of(t), a.div)];
        };
        auto find_rows = [&](int t, int set) {
            if (w != 0) return;
            const bool fine = page_ok(a, page);
            bad |= !fine;
            s_row[set][lane] = cache_row(a, fine ? page : 0, hk, key_of(t));
        };
        auto request = [&](int set) {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const size_t at = (size_t)s_row[set][prow + i * RR] * (D * EB) + pcol;
                rk[i] = gload((const uint4*)((const char*)a.k_cache + at));
                rv[i] = gload((const uint4*)((const char*)a.v_cache + at));
            }
            if (E4M3 && w == 0) {
                rks = gload(a.k_scale + s_row[set][lane]);
                rvs = gload(a.v_scale + s_row[set][lane]);
            }
        };
        auto put = [&](float* to, uint4 u) {
            if (!E4M3) {
                *(uint4*)to = u;
                return;
            }
            const uint32_t wd[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *(float4*)(to + 4 * i) = make_float4(
                    __builtin_amdgcn_cvt_f32_fp8((int)wd[i], 0), __builtin_amdgcn_cvt_f32_fp8((int)wd[i], 1),
                    __builtin_amdgcn_cvt_f32_fp8((int)wd[i], 2), __builtin_amdgcn_cvt_f32_fp8((int)wd[i], 3));
        };
        find_rows(k0, 0);
        look_up(k0 + kTileKeys);
        __syncthreads();
        request(0);
        take_tree();
        int set = 0;
        for (int t = k0; t < k1; t += kTileKeys, set ^= 1) {
            lds_barrier();  // the last tile's reads are done
            if (t + kTileKeys > k1) {  // past the last key its row was read again: 0, for a value that is not finite
#pragma unroll
                for (int i = 0; i < L; ++i)
                    if (prow + i * RR >= k1 - t) rv[i] = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < L; ++i) {
                put(&s_K[(prow + i * RR) * kS + pcol / EB], rk[i]);
                put(&s_V[(prow + i * RR) * kS + pcol / EB], rv[i]);
            }
            if (E4M3 && w == 0) {
                s_ks[lane] = rks;
                s_vs[lane] = t + lane < k1 ? rvs : 0.f;
            }
            find_rows(t + kTileKeys, set ^ 1);
            lds_barrier();
            if (t + kTileKeys < k1) {
                look_up(t + 2 * kTileKeys);
                request(set ^ 1);
            }
            take(std::false_type(), min(kTileKeys, k1 - t), 0);
        }
    } else {
        bad = k1 > k0;  // positions without a page
        __syncthreads();
        take_tree();
    }
    st |= __syncthreads_or(bad) ? kStBadCache : 0;
    if (hk == 0 && rb == 0 && tid == 0) {
        if (pt.n > 1)
            ws.bits[part] = st;
        else if (a.status)
            a.status[b] = st;
    }
    if (pt.n == 1 && st) return;
    l = row_sum(l);
    if (WK == 4) {
        // (all waves are past the barrier above, so s_K is free)
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                *(float4*)&s_K[(16 * wk + l16) * kS + 64 * h + 16 * lg + 4 * r] =
                    make_float4(o[4 * h][r], o[4 * h + 1][r], o[4 * h + 2][r], o[4 * h + 3][r]);
        if (lg == 0) {
            s_ml[wk][l16][0] = base;
            s_ml[wk][l16][1] = l;
        }
        __syncthreads();
        for (int i = tid; i < R * (D / 4); i += 256) {
            const int r = i / (D / 4), d = i % (D / 4) * 4;
            const float m = fmaxf(fmaxf(s_ml[0][r][0], s_ml[1][r][0]), fmaxf(s_ml[2][r][0], s_ml[3][r][0]));
            float sum = 0.f;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float f = __builtin_amdgcn_exp2f(s_ml[x][r][0] - m);
                const float4 u = *(const float4*)&s_K[(16 * x + r) * kS + d];
                sum = fmaf(f, s_ml[x][r][1], sum);
                v = make_float4(fmaf(f, u.x, v.x), fmaf(f, u.y, v.y), fmaf(f, u.z, v.z), fmaf(f, u.w, v.w));
            }
            const size_t at = (size_t)(r / g) * H + hk * g + r % g;
            if (pt.n > 1) {
                *(float4*)(ws.o + ((size_t)part * T * H + at) * D + d) = v;
                if (d == 0) {
                    ws.ml[((size_t)part * T * H + at) * 2] = m;
                    ws.ml[((size_t)part * T * H + at) * 2 + 1] = sum;
                }
            } else {
                gstore((float4*)((float*)a.o + ((size_t)b * T * H + at) * D + d),
                       make_float4(v.x / sum, v.y / sum, v.z / sum, v.w / sum));
            }
        }
        return;
    }
    if (row >= R) return;
    const size_t at = (size_t)node * H + hk * g + row % g;
    const float by = pt.n > 1 ? 1.f : 1.f / l;
    float* to = (pt.n > 1 ? ws.o + ((size_t)part * T * H + at) * D : (float*)a.o + ((size_t)b * T * H + at) * D) + 16 * lg;
#pragma unroll
    for (int h = 0; h < D / 64; ++h)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            gstore((float4*)(to + 64 * h + 4 * r),
                   make_float4(o[4 * h][r] * by, o[4 * h + 1][r] * by, o[4 * h + 2][r] * by, o[4 * h + 3][r] * by));
    if (pt.n > 1 && lg == 0) {
        ws.ml[((size_t)part * T * H + at) * 2] = base;
        ws.ml[((size_t)part * T * H + at) * 2 + 1] = l;
    }
}

template <int D, bool E4M3>
void launch_d(const AttnArgs& a, const AttnPlan& p, const AttnWorkspace& ws, int block_rows, int row_blocks, hipStream_t stream) {
    const long long units = (long long)p.parts * a.Hk;
    const dim3 grid((unsigned)((units + 7) / 8 * 8 * row_blocks));
    const int g = a.H / a.Hk;
    const unsigned nodes = min(a.T, (block_rows + g - 2) / g + 1), lds = nodes * ((a.T + 31) / 32) * 4;
    if (block_rows == 16)
        hipLaunchKernelGGL((attn_f32_kernel<D, E4M3, 4>), grid, dim3(256), lds, stream, a, p, ws, row_blocks);
    else
        hipLaunchKernelGGL((attn_f32_kernel<D, E4M3, 1>), grid, dim3(256), lds, stream, a, p, ws, row_blocks);
}

}  // namespace

void launch_attn_f32(const AttnArgs& a, bool e4m3, const AttnPlan& p, const AttnWorkspace& ws, int block_rows, int row_blocks,
                     hipStream_t stream) {
    if (a.D == 64)
        e4m3 ? launch_d<64, true>(a, p, ws, block_rows, row_blocks, stream) : launch_d<64, false>(a, p, ws, block_rows, row_blocks, stream);
    else
        e4m3 ? launch_d<128, true>(a, p, ws, block_rows, row_blocks, stream) : launch_d<128, false>(a, p, ws, block_rows, row_blocks, stream);
}

}  // namespace tsv
