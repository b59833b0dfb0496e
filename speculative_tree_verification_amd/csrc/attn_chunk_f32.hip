// attn_chunk_f32.hip -- attention of packed rows over the paged cache on fp32 matrix
// instructions (fp32 inputs, head_dim 64 or 128, cache in fp32 or e4m3).
//
// As in attn_f32.hip the scores are formed transposed, S^T = K Q^T, on 16x16x4 products: a
// lane holds the keys 4 g + r (g = l / 16) of one row l % 16, and the weights P are the
// next product's operand as they are, O^T = V^T P^T, if its step r takes key 4 g + r from
// lane group g. Which element of the head each k-slot of K Q^T stands for is free, so a lane
// reads K and Q as 16-byte pieces (d = 16 j + 4 g + e in step 4 j + e); so is which row of
// O^T stands for which d, and a 16-byte piece of V feeds four products (tile 4 h + c: d = 64
// h + 4 i + c for its row i).
//
// 64 keys at a time are shared in LDS by four waves; WK 1: of 16 rows each, WK 4: of the
// same 16 rows, a quarter of the keys each, which meet at the end.
//
// Many rows are bound by the fp32 matrix unit, which waits for LDS and the softmax of its own
// step: 2 chunks of 500 tokens behind 1000 positions, 32 query and 8 key heads of 128, 218 us
// (94 TFLOP/s; a large fp32 product reaches 154; over an e4m3 cache 239 us); 3 prompts of 130 to 777 tokens in a window of
// 255, 24 and 3 heads of 64, 29.3 us, the unit busy in 35% of the cycles. Few rows are bound by
// the cache's bytes: 32 tokens over 2200 positions, 578 MB, 116 us (5.0 TB/s). In e4m3 those are
// 150 MB, but the products are the same: 84 us. Weights stay in fp32.
#include <cfloat>
#include <type_traits>

#include "attn_chunk.hpp"
#include "attn_lanes.hpp"

namespace tsv {
namespace {

template <int D, bool E4M3, int WK>
__global__ __launch_bounds__(256, 2) void chunk_f32_kernel(ChunkArgs a, ChunkPlan plan, ChunkWorkspace ws) {
    constexpr int M = 64 / WK, kS = D + 4, NX = 4 / WK;
    __shared__ __attribute__((aligned(16))) float s_K[kTileKeys * kS], s_V[kTileKeys * kS];  // s_K: then the waves' outputs
    __shared__ __attribute__((aligned(16))) float s_ks[kTileKeys], s_vs[kTileKeys], s_ml[4][16][2];
    __shared__ uint32_t s_row[2][kTileKeys];
    __shared__ uint32_t s_odd[2][2];  // keys of a tile that not all rows see, with values that are not finite
    const int tid = threadIdx.x, lane = tid & (kWave - 1), w = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int l16 = lane & 15, lg = lane >> 4, wr = w / WK, wk = w % WK;
    const int hk = blockIdx.x % a.Hk;
    const ChunkUnit u = find_unit<false>(a, plan, blockIdx.x / a.Hk);
    if (blockIdx.x == 0 && w == 0) chunk_status(a, plan, u.bad);
    if (!u.ok) return;
    const ChunkKeys kk = chunk_keys(a, plan, u);
    const int H = a.H, g = plan.g, R = u.n * g, row0 = u.block * M;
    const int32_t* table = a.page_table + (size_t)u.seq * a.max_pages;

    // this lane's row
    const int row = min(row0 + 16 * wr + l16, R - 1), token = page_of(row, plan.by_g), own = u.old + token;
    const size_t at = ((size_t)u.start + token) * H + hk * g + (row - token * g);  // in q and o
    const int own_min = u.old + page_of(row0, plan.by_g), own_max = u.old + page_of(min(R, row0 + M) - 1, plan.by_g);
    const bool active = row0 + 16 * wr < R;
    float4 q[D / 16];
    {
        const float* qp = (const float*)a.q + at * D + 4 * lg;
        const float sign = a.scale_log2 < 0.f ? -1.f : 1.f;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            q[j] = gload((const float4*)(qp + 16 * j));
            q[j] = make_float4(sign * q[j].x, sign * q[j].y, sign * q[j].z, sign * q[j].w);
        }
    }
    const float c = fmaxf(fabsf(a.scale_log2), 1.17549435e-38f);
    float base = -FLT_MAX, l = 0.f;  // as in the bf16 tile kernel
    f32x4 o[D / 16];
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    const ChunkSeen seen = chunk_seen(a, kk, own);
    auto sees = [&](int v) { return v < seen.hi && (v >= seen.lo || v < a.sinks); };  // virtual position v

    // One tile of keys in LDS, from virtual position t on, or the first `keys` of it
    auto take = [&](int t, bool whole, auto keys) {
        constexpr int NK = decltype(keys)::value / 16 < NX ? decltype(keys)::value / 16 : NX;  // products of 16 keys
        f32x4 s[NK];
#pragma unroll
        for (int x = 0; x < NK; ++x) s[x] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
#pragma unroll
            for (int x = 0; x < NK; ++x) s[x] = mma4(*(const float4*)&s_K[(16 * (x + wk) + l16) * kS + 16 * j + 4 * lg], q[j], s[x]);
            if (j % 2) __builtin_amdgcn_sched_barrier(0);
        }
        if (E4M3) {
#pragma unroll
            for (int x = 0; x < NK; ++x) s[x] *= *(const f32x4*)&s_ks[16 * (x + wk) + 4 * lg];
        }
        if (!whole) {
#pragma unroll
            for (int x = 0; x < NK; ++x)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int v = t + 16 * (x + wk) + 4 * lg + r;
                    s[x][r] = sees(v) ? s[x][r] : -INFINITY;
                }
        }
        float mx = max3(max3(s[0][0], s[0][1], s[0][2]), s[0][3], s[0][3]);
#pragma unroll
        for (int x = 1; x < NK; ++x) mx = max3(max3(mx, s[x][0], s[x][1]), s[x][2], s[x][3]);
        if (__ballot(fmaf(mx, c, -base) > kSlack)) {
            const float top = row_max(mx);  // a row moves by its own scores alone: its bits do not follow from its neighbours'
            const float to = fmaf(top, c, -base) > kSlack ? top * c : base, al = __builtin_amdgcn_exp2f(base - to);
            l *= al;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) o[i] *= al;
            base = to;
        }
#pragma unroll
        for (int x = 0; x < NK; ++x) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                s[x][r] = __builtin_amdgcn_exp2f(fmaf(s[x][r], c, -base));
                l += s[x][r];  // of this lane's keys; the lanes of a row meet at the end
            }
            if (E4M3) {
                const f32x4 vs = *(const f32x4*)&s_vs[16 * (x + wk) + 4 * lg];
#pragma unroll
                for (int r = 0; r < 4; ++r) s[x][r] = s[x][r] == 0.f ? 0.f : s[x][r] * vs[r];  // (a scale that is not finite is no masked row's)
            }
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
    // the values of a tile that are not finite, to the rows that see them, from the waves that
    // have their keys
    auto add_odd = [&](int t, const uint32_t* odd) {
#pragma unroll
        for (int half = 0; half < 2; ++half)
            for (uint32_t left = odd[half]; left; left &= left - 1) {
                const int key = 32 * half + __builtin_ctz(left), pos = chunk_pos(kk, t + key), page = page_of(pos, a.div);
                if (WK == 4 && key / 16 != wk) continue;
                const size_t row = ((size_t)table[page] * a.Hk + hk) * a.page_size + (pos - page * a.page_size);
                const bool here = sees(t + key);
#pragma unroll
                for (int i = 0; i < D / 4; ++i) {
                    const size_t d = row * D + 64 * (i / 16) + 16 * lg + i % 16;
                    const float f = E4M3 ? e4m3_ld((const uint8_t*)a.v_cache + d) : gload((const float*)a.v_cache + d);
                    if (here && nonfinite(f)) o[4 * (i / 16) + i % 4][i % 16 / 4] += f;
                    if (i % 4 == 3) __builtin_amdgcn_sched_barrier(0);
                }
            }
    };

    constexpr int EB = E4M3 ? 1 : 4;
    constexpr int L = kTileKeys * D * EB / 16 / 256;  // 16-byte loads of K, and of V, per thread
    constexpr int RR = 256 / (D * EB / 16);           // rows that one of them covers
    uint4 rk[L], rv[L];
    float rks = 1.f, rvs = 1.f;
    int page = 0;  // of this lane's key, in the first wave
    const int prow = tid / (D * EB / 16), pcol = tid % (D * EB / 16) * 16;
    // the first wave looks up pages and rows, for all
    auto pos_of = [&](int t) { return chunk_pos(kk, min(t + lane, kk.k1 - 1)); };
    auto look_up = [&](int t) {
        if (w == 0) page = table[page_of(pos_of(t), a.div)];
    };
    auto find_rows = [&](int t, int set) {
        if (w != 0) return;
        const int pos = pos_of(t);
        s_row[set][lane] = ((uint32_t)page * a.Hk + hk) * a.page_size + (pos - page_of(pos, a.div) * a.page_size);
    };
    auto request = [&](int set) {
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const size_t from = (size_t)s_row[set][prow + i * RR] * (D * EB) + pcol;
            rk[i] = gload((const uint4*)((const char*)a.k_cache + from));
            rv[i] = gload((const uint4*)((const char*)a.v_cache + from));
        }
        if (E4M3 && w == 0) {
            rks = gload(a.k_scale + s_row[set][lane]);
            rvs = gload(a.v_scale + s_row[set][lane]);
        }
    };
    auto floats = [&](uint4 x, float4 (&f)[E4M3 ? 4 : 1]) {
        const uint32_t wd[4] = {x.x, x.y, x.z, x.w};
        if (E4M3) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f[i % (E4M3 ? 4 : 1)] = make_float4(__builtin_amdgcn_cvt_f32_fp8((int)wd[i], 0), __builtin_amdgcn_cvt_f32_fp8((int)wd[i], 1),
                                                    __builtin_amdgcn_cvt_f32_fp8((int)wd[i], 2), __builtin_amdgcn_cvt_f32_fp8((int)wd[i], 3));
        } else {
            f[0] = make_float4(__uint_as_float(wd[0]), __uint_as_float(wd[1]), __uint_as_float(wd[2]), __uint_as_float(wd[3]));
        }
    };
    // the pages are checked while the queries and the first keys' pages are on their way (the
    // three windowed prompts above: 34.6 us, 35.1 with the check first)
    look_up(kk.k0);
    if (chunk_check<256>(a, u, hk, ws)) return;
    if (kk.k1 > kk.k0) {
        if (tid < 4) s_odd[tid / 2][tid % 2] = 0;
        find_rows(kk.k0, 0);
        look_up(kk.k0 + kTileKeys);
        __syncthreads();
        request(0);
        int set = 0;
        for (int t = kk.k0; t < kk.k1; t += kTileKeys, set ^= 1) {
            const int end = t + kTileKeys;
            const bool whole = end <= kk.k1 && (end <= kk.sinks || (t >= kk.sinks && chunk_pos(kk, end - 1) <= own_min && own_max - chunk_pos(kk, t) < a.window));
            lds_barrier();  // the last tile's reads are done
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const int key = prow + i * RR;
                float4 f[E4M3 ? 4 : 1];
                floats(rk[i], f);
#pragma unroll
                for (int e = 0; e < (E4M3 ? 4 : 1); ++e) *(float4*)&s_K[key * kS + pcol / EB + 4 * e] = f[e];
                floats(rv[i], f);
#pragma unroll
                for (int e = 0; e < (E4M3 ? 4 : 1); ++e) {
                    if (!whole) {
                        // past the last key its row was read again: 0 in its place; values that are not
                        // finite enter as 0 and are added for the rows that see them
                        if (t + key >= kk.k1) {
                            f[e] = make_float4(0.f, 0.f, 0.f, 0.f);
                        } else if (nonfinite(f[e].x) || nonfinite(f[e].y) || nonfinite(f[e].z) || nonfinite(f[e].w)) {
                            atomicOr(&s_odd[set][key / 32], 1u << (key % 32));
                            f[e] = make_float4(nonfinite(f[e].x) ? 0.f : f[e].x, nonfinite(f[e].y) ? 0.f : f[e].y,
                                               nonfinite(f[e].z) ? 0.f : f[e].z, nonfinite(f[e].w) ? 0.f : f[e].w);
                        }
                    }
                    *(float4*)&s_V[key * kS + pcol / EB + 4 * e] = f[e];
                }
            }
            if (E4M3 && w == 0) {
                s_ks[lane] = rks;
                s_vs[lane] = rvs;
            }
            find_rows(end, set ^ 1);
            lds_barrier();
            if (tid < 2) s_odd[set ^ 1][tid] = 0;
            if (end < kk.k1) {
                look_up(end + kTileKeys);
                request(set ^ 1);
            }
            if (!active) continue;
            // the last tile may have few keys (the windowed prompts above: 29.3 us, 30.2 without the
            // quarter, 32.4 with all products)
            if (NX > 2 && t + kTileKeys / 4 >= kk.k1)
                take(t, false, std::integral_constant<int, kTileKeys / 4>());
            else if (NX > 2 && t + kTileKeys / 2 >= kk.k1)
                take(t, false, std::integral_constant<int, kTileKeys / 2>());
            else
                take(t, whole, std::integral_constant<int, kTileKeys>());
            if (!whole) add_odd(t, s_odd[set]);
        }
    }
    l = row_sum(l);
    if (WK == 4) {
        __syncthreads();  // s_K is free
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
        for (int i = tid; i < min(M, R - row0) * (D / 4); i += 256) {
            const int r = i / (D / 4), d = i % (D / 4) * 4;
            const float m = fmaxf(fmaxf(s_ml[0][r][0], s_ml[1][r][0]), fmaxf(s_ml[2][r][0], s_ml[3][r][0]));
            float sum = 0.f;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float f = __builtin_amdgcn_exp2f(s_ml[x][r][0] - m);
                const float4 y = *(const float4*)&s_K[(16 * x + r) * kS + d];
                sum = fmaf(f, s_ml[x][r][1], sum);
                v = make_float4(fmaf(f, y.x, v.x), fmaf(f, y.y, v.y), fmaf(f, y.z, v.z), fmaf(f, y.w, v.w));
            }
            if (u.parts > 1) {
                const size_t slot = ((size_t)u.slot * a.Hk + hk) * M + r;
                *(float4*)(ws.o + slot * D + d) = v;
                if (d == 0) {
                    ws.ml[slot * 2] = m;
                    ws.ml[slot * 2 + 1] = sum;
                }
            } else {
                const int tk = page_of(row0 + r, plan.by_g);
                gstore((float4*)((float*)a.o + (((size_t)u.start + tk) * H + hk * g + (row0 + r - tk * g)) * D + d),
                       make_float4(v.x / sum, v.y / sum, v.z / sum, v.w / sum));
            }
        }
        return;
    }
    if (row0 + 16 * wr + l16 >= R) return;
    const size_t slot = ((size_t)u.slot * a.Hk + hk) * M + 16 * wr + l16;
    const float by = u.parts > 1 ? 1.f : 1.f / l;
    float* to = (u.parts > 1 ? ws.o + slot * D : (float*)a.o + at * D) + 16 * lg;
#pragma unroll
    for (int h = 0; h < D / 64; ++h)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            gstore((float4*)(to + 64 * h + 4 * r),
                   make_float4(o[4 * h][r] * by, o[4 * h + 1][r] * by, o[4 * h + 2][r] * by, o[4 * h + 3][r] * by));
    if (u.parts > 1 && lg == 0) {
        ws.ml[slot * 2] = base;
        ws.ml[slot * 2 + 1] = l;
    }
}

template <int D, bool E4M3>
void launch_d(const ChunkArgs& a, const ChunkPlan& p, const ChunkWorkspace& ws, dim3 grid, hipStream_t stream) {
    if (p.rows == 16)
        hipLaunchKernelGGL((chunk_f32_kernel<D, E4M3, 4>), grid, dim3(256), 0, stream, a, p, ws);
    else
        hipLaunchKernelGGL((chunk_f32_kernel<D, E4M3, 1>), grid, dim3(256), 0, stream, a, p, ws);
}

}  // namespace

void launch_chunk_f32(const ChunkArgs& a, bool e4m3, const ChunkPlan& p, const ChunkWorkspace& ws, dim3 grid, hipStream_t stream) {
    if (a.D == 64)
        e4m3 ? launch_d<64, true>(a, p, ws, grid, stream) : launch_d<64, false>(a, p, ws, grid, stream);
    else
        e4m3 ? launch_d<128, true>(a, p, ws, grid, stream) : launch_d<128, false>(a, p, ws, grid, stream);
}

}  // namespace tsv
