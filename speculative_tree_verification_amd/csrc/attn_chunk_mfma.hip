// attn_chunk_mfma.hip -- attention of packed rows over the paged cache on bf16 matrix
// instructions (head_dim 64 or 128, cache in bf16 or e4m3).
//
// The scores are formed transposed, S^T = K Q^T (32 keys x 32 rows a product): a lane then
// holds 16 keys of one row, the softmax statistics are a reduction in registers and over two
// lanes, the factor of a rescaling is one value per lane, and the weights are the next
// product's operand, O^T = V^T P^T, as they are. V^T comes from LDS through the transposing
// read, in the same order of keys.
#include <cfloat>

#include "attn_chunk.hpp"
#include "attn_lanes.hpp"
#include "mfma_util.hpp"

#define TSV_INLINE __attribute__((always_inline))

namespace tsv {
namespace {

constexpr int kSub = 32;  // keys of a step

// Most steps whose keys not all of a block's 128 rows see: up to 127 positions at the windows'
// start, behind the sinks' last step's others, and up to 127 at the end, each with what is
// left of its steps
constexpr int kOddSteps = 12;

__device__ __forceinline__ uint32_t chunk_row(const ChunkArgs& a, int page, int hk, int pos) {
    return ((uint32_t)page * a.Hk + hk) * a.page_size + (pos - page_of(pos, a.div) * a.page_size);
}

// ---------------------------------------------------------------- few rows
// Up to 16 rows share a key head: single tokens, or a few of them. Four waves take 32 keys
// each in turn and meet at the end; K goes from memory into the operand registers, V through
// LDS. The weights enter the product with V as two bf16 parts: free here, since the kernel
// is bound by the cache's bytes (32 query and 8 key heads of 128: one token over 65532
// positions, 268 MB, 65 us with the join, 4.1 TB/s, and 51 where the last call left most of it in
// the last-level cache; 64 tokens with windows of 1021, 251 MB, 50.7 us; 64 over e4m3 caches of 17
// to 8190 positions 116 us, 4.8 TB/s).
template <int ND, bool E4M3>
__global__ __launch_bounds__(256, 3) void chunk_rows_kernel(ChunkArgs a, ChunkPlan plan, ChunkWorkspace ws) {
    constexpr int D = ND * 32, M = 16, kVs = D + 16, kOs = D + 4;
    __shared__ __attribute__((aligned(16))) uint16_t s_V[4][kSub * kVs];  // then the waves' outputs
    __shared__ __attribute__((aligned(16))) float s_ks[4][kSub], s_vs[4][kSub], s_ml[4][M][2];
    __shared__ uint32_t s_row[4][2][kSub];
    static_assert(sizeof(s_V) >= 4 * M * kOs * sizeof(float), "outputs take the place of V");
    const int tid = threadIdx.x, lane = tid & (kWave - 1), w = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int l16 = lane & 15, lg = lane >> 4;
    const int hk = blockIdx.x % a.Hk;
    const ChunkUnit u = find_unit<false>(a, plan, blockIdx.x / a.Hk);
    if (blockIdx.x == 0 && w == 0) chunk_status(a, plan, u.bad);
    if (!u.ok) return;
    const ChunkKeys kk = chunk_keys(a, plan, u);
    const int H = a.H, g = plan.g, R = u.n * g, row0 = u.block * M;
    const int32_t* table = a.page_table + (size_t)u.seq * a.max_pages;

    // this lane's row: k-slot e of step 2 j + h is d = 64 j + 16 lg + 8 h + e
    const int row = min(row0 + l16, R - 1), token = page_of(row, plan.by_g), own = u.old + token;
    const int own_min = u.old + page_of(row0, plan.by_g), own_max = u.old + page_of(min(R, row0 + M) - 1, plan.by_g);
    bf16x8 q[ND];
    {
        const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;
        const uint16_t* qp = (const uint16_t*)a.q + (((size_t)u.start + token) * H + hk * g + (row - token * g)) * D + 16 * lg;
#pragma unroll
        for (int i = 0; i < ND; ++i) {
            const uint4 v = gload((const uint4*)(qp + 64 * (i / 2) + 8 * (i % 2)));
            q[i] = as_operand(make_uint4(v.x ^ flip, v.y ^ flip, v.z ^ flip, v.w ^ flip));
        }
    }
    const float c = fmaxf(fabsf(a.scale_log2), 1.17549435e-38f);

    float base = -FLT_MAX, l = 0.f;  // the row's maximum, c times its largest score, as it is rounded
    f32x4 o[D / 16];
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[i] = f32x4{0.f, 0.f, 0.f, 0.f};

    constexpr int EB = E4M3 ? 1 : 2;          // bytes of an element
    constexpr int KL = E4M3 ? ND / 2 : ND;    // 16-byte loads of a key's lane
    constexpr int VL = kSub * D * EB / 16 / kWave;  // of V per lane
    constexpr int VR = kWave / (D * EB / 16);       // rows of V a load covers
    const char* kc = (const char*)a.k_cache;
    const char* vc = (const char*)a.v_cache;
    uint4 rk[2][KL], rv[VL];
    float rks = 1.f, rvs = 1.f;
    int page = 0;  // of this lane's key (lane % 32) of the step after the one being requested
    auto pos_of = [&](int t) TSV_INLINE { return chunk_pos(kk, min(t + (lane & 31), kk.k1 - 1)); };
    auto look_up = [&](int t) TSV_INLINE { page = table[page_of(pos_of(t), a.div)]; };
    auto request_rows = [&](int t, int set) TSV_INLINE {  // row of each key, to all lanes
        const uint32_t r = chunk_row(a, page, hk, pos_of(t));
        if (lane < kSub) s_row[w][set][lane] = r;
        if (E4M3) {
            rks = gload(a.k_scale + r);
            rvs = gload(a.v_scale + r);
        }
        wave_sync();
    };
    auto request_K = [&](int set) TSV_INLINE {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const char* p = kc + (size_t)s_row[w][set][16 * t + l16] * (D * EB) + lg * (E4M3 ? 16 : 32);
#pragma unroll
            for (int i = 0; i < KL; ++i) rk[t][i] = gload((const uint4*)(p + (E4M3 ? 64 * i : 128 * (i / 2) + 16 * (i % 2))));
        }
    };
    auto request_V = [&](int set) TSV_INLINE {
#pragma unroll
        for (int i = 0; i < VL; ++i) {
            const int key = i * VR + lane / (D * EB / 16), col = lane % (D * EB / 16) * 16;
            rv[i] = gload((const uint4*)(vc + (size_t)s_row[w][set][key] * (D * EB) + col));
        }
    };
    int t = kk.k0 + w * kSub, set = 0;
    // the pages are checked while the first step's are on their way
    const bool work = t < kk.k1;
    if (work) look_up(t);
    if (chunk_check<256>(a, u, hk, ws)) return;
    if (work) {
        request_rows(t, 0);
        request_K(0);
        request_V(0);
        look_up(t + 4 * kSub);
    }
    for (; t < kk.k1; t += 4 * kSub, set ^= 1) {
        const bool more = t + 4 * kSub < kk.k1;
        if (E4M3) {
            if (lane < kSub) {
                s_ks[w][lane] = rks;
                s_vs[w][lane] = rvs;
            }
            wave_sync();
        }
        f32x4 s[2], vs[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            s[x] = f32x4{0.f, 0.f, 0.f, 0.f};
            if (E4M3) {
#pragma unroll
                for (int i = 0; i < KL; ++i) {
                    s[x] = mma(as_operand(e4m3_to_bf16(make_uint2(rk[x][i].x, rk[x][i].y))), q[2 * i], s[x]);
                    s[x] = mma(as_operand(e4m3_to_bf16(make_uint2(rk[x][i].z, rk[x][i].w))), q[2 * i + 1], s[x]);
                }
                s[x] *= *(const f32x4*)&s_ks[w][16 * x + 4 * lg];
                vs[x] = *(const f32x4*)&s_vs[w][16 * x + 4 * lg];
            } else {
#pragma unroll
                for (int i = 0; i < KL; ++i) s[x] = mma(as_operand(rk[x][i]), q[i], s[x]);
            }
        }
        if (more) {
            request_rows(t + 4 * kSub, set ^ 1);
            request_K(set ^ 1);
        }
        // V into LDS, its registers free for the next step. Where not all rows see all keys, an
        // element that is not finite enters as 0, and the rows that see it add it afterwards;
        // past the last key its row was read again: 0 in its place
        const int end = t + kSub;
        const bool whole = end <= kk.k1 && (end <= kk.sinks || (t >= kk.sinks && chunk_pos(kk, end - 1) <= own_min && own_max - chunk_pos(kk, t) < a.window));
        uint32_t strange = 0;
#pragma unroll
        for (int i = 0; i < VL; ++i) {
            const int key = i * VR + lane / (D * EB / 16), col = lane % (D * EB / 16) * (16 / EB);
            uint4 x[2] = {rv[i], rv[i]};
            if (E4M3) {
                x[0] = e4m3_to_bf16(make_uint2(rv[i].x, rv[i].y));
                x[1] = e4m3_to_bf16(make_uint2(rv[i].z, rv[i].w));
            }
#pragma unroll
            for (int h = 0; h < (E4M3 ? 2 : 1); ++h) {
                if (!whole) {
                    if (t + key >= kk.k1) {
                        x[h] = make_uint4(0, 0, 0, 0);
                    } else if (nonfinite_bits(x[h]) & 0x80008000u) {
                        strange |= 1u << key;
                        x[h] = only_finite(x[h]);
                    }
                }
                *(uint4*)&s_V[w][key * kVs + col + 8 * h] = x[h];
            }
        }
        if (more) {
            request_V(set ^ 1);
            look_up(t + 8 * kSub);
        }
        if (!whole) {
            asm volatile("");
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int v = t + 16 * (e / 4) + 4 * lg + e % 4, pos = chunk_pos(kk, v);
                if (!(v < kk.k1 && pos <= own && (own - pos < a.window || pos < a.sinks))) s[e / 4][e % 4] = -INFINITY;
            }
        }
        wave_sync();
        // softmax and product
        const float top = max3(max3(s[0][0], s[0][1], s[0][2]), max3(s[0][3], s[1][0], s[1][1]), max3(s[1][1], s[1][2], s[1][3]));
        const float to = fmaxf(base, row_max(top) * c);
        if (__ballot(to > base)) {  // some row's maximum moved (the factor of the others is 1)
            const float al = __builtin_amdgcn_exp2f(base - to);
            base = to;
            l *= al;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) o[i] *= al;
        }
        float p[8], sum = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            p[e] = __builtin_amdgcn_exp2f(fmaf(s[e / 4][e % 4], c, -base));
            sum += p[e];
        }
        l += sum;  // of this lane's keys; the four lanes of a row meet at the end
        if (E4M3) {
#pragma unroll
            for (int e = 0; e < 8; ++e) p[e] = p[e] == 0.f ? 0.f : p[e] * vs[e / 4][e % 4];  // (a scale that is not finite is no masked row's)
        }
        // The upper 16 bits of a weight, and what is left with 2^-23 of it: both parts are
        // positive, so that an infinite value times them is one infinity (0 times it, or a part of
        // the other sign, makes a NaN)
        uint32_t hi[4], lo[4];
        constexpr float kUp = 1.f + 0x1p-23f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            hi[e] = __builtin_amdgcn_perm(__float_as_uint(p[2 * e + 1]), __float_as_uint(p[2 * e]), 0x07060302u);
            lo[e] = pack_bf16x2(fmaf(p[2 * e], kUp, -__uint_as_float(hi[e] << 16)), fmaf(p[2 * e + 1], kUp, -__uint_as_float(hi[e] & 0xffff0000u)));
        }
        const bf16x8 pf = as_operand(make_uint4(hi[0], hi[1], hi[2], hi[3])), pl = as_operand(make_uint4(lo[0], lo[1], lo[2], lo[3]));
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            const bf16x8 v = read_columns(&s_V[w][16 * i], kVs, lane);
            o[i] = mma(v, pf, o[i]);
            o[i] = mma(v, pl, o[i]);
        }
        if (!whole && __ballot(strange != 0)) {
#pragma unroll
            for (int x = 1; x < kWave; x <<= 1) strange |= __shfl_xor(strange, x, kWave);
            for (; strange; strange &= strange - 1) {
                const int pos = chunk_pos(kk, t + __builtin_ctz(strange));
                const size_t at = (size_t)chunk_row(a, table[page_of(pos, a.div)], hk, pos) * D;
                const bool seen = pos <= own && (own - pos < a.window || pos < a.sinks);
#pragma unroll
                for (int e = 0; e < D / 4; ++e) {
                    const size_t d = at + e / 4 * 16 + 4 * lg + e % 4;
                    const uint16_t b = !E4M3 ? gload((const uint16_t*)a.v_cache + d) : (gload((const uint8_t*)a.v_cache + d) & 0x7f) == 0x7f ? 0x7fc0 : 0;
                    if (seen && (b & 0x7f80) == 0x7f80) o[e / 4][e % 4] += bf16_bits_to_f32(b);
                    if (e % 4 == 3) __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
        wave_sync();
    }
    l = row_sum(l);

    // the four waves
    if (lg == 0) {
        s_ml[w][l16][0] = base;
        s_ml[w][l16][1] = l;
    }
    __syncthreads();
    float mt = -FLT_MAX, lt = 0.f;
#pragma unroll
    for (int x = 0; x < 4; ++x) mt = fmaxf(mt, s_ml[x][l16][0]);
#pragma unroll
    for (int x = 0; x < 4; ++x) lt += s_ml[x][l16][1] * __builtin_amdgcn_exp2f(s_ml[x][l16][0] - mt);
    {
        const float al = __builtin_amdgcn_exp2f(base - mt);
        float* so = (float*)s_V + (w * M + l16) * kOs + 4 * lg;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) *(f32x4*)(so + 16 * i) = o[i] * al;
    }
    // a row's m and l for all threads
    __shared__ float s_m[M], s_l[M];
    if (tid < M) {
        s_m[tid] = mt;
        s_l[tid] = lt;
    }
    __syncthreads();
    for (int i = tid; i < min(M, R - row0) * (D / 4); i += 256) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int x = 0; x < 4; ++x) v += *(const f32x4*)((const float*)s_V + (x * M + r) * kOs + d);
        if (u.parts > 1) {
            const size_t at = ((size_t)u.slot * a.Hk + hk) * M + r;
            *(f32x4*)(ws.o + at * D + d) = v;
            if (d == 0) {
                ws.ml[at * 2] = s_m[r];
                ws.ml[at * 2 + 1] = s_l[r];
            }
        } else {
            const float lr = s_l[r];
            const int tk = page_of(row0 + r, plan.by_g);
            gstore((uint2*)((uint16_t*)a.o + (((size_t)u.start + tk) * H + hk * g + (row0 + r - tk * g)) * D + d),
                   make_uint2(pack_bf16x2(v[0] / lr, v[1] / lr), pack_bf16x2(v[2] / lr, v[3] / lr)));
        }
    }
}

// ---------------------------------------------------------------- tiles
// Four waves of 32 rows.
//
// A step takes 32 keys. Its products are not its own softmax's: while the weights of step s
// are formed, the matrix unit has the scores of step s + 1 and the product of step s - 1
// with V, so that neither waits for the other. Keys and values are in rings of four steps
// in LDS, filled two steps at a time (one barrier), from registers that were requested
// two steps before; the values follow the keys by two steps.
//
// The weights are rounded to bf16 once, relative to a maximum that they pass by a factor of
// 2^kSlack at most, and the sum is formed before: a second part, as above, would be half of the
// matrix products again. Each weight is off by e_j, 2^-8 of itself at most, and an output by sum w_j
// e_j v_j / sum w_j: 0.0021 to 0.0024 of its size on average, of which its own rounding is 0.0017. (The
// sum of the rounded weights would make it sum w_j e_j (v_j - o) / sum w_j: less where one key has most
// of the weight, but up to twice as much where values differ in sign.)
//
// Bound by three units that two waves a SIMD keep busy in turn, none of them to the end, and by
// the clock that the card's power leaves them (2.0 GHz): 4096 tokens, 32 query and 8 key heads of
// 128, 155 us, 889 TFLOP/s, the matrix unit busy in 41% of the cycles, the vector unit issuing in
// 42%, and LDS, from which each wave reads all of a step's keys and values for its 32 rows, active
// in 34% (18.3 MB read and 4.5 written a compute unit: 54% at 128 bytes a cycle); 509
// tokens behind 32749 positions 294 us, 938 TFLOP/s. At an earlier step (177 and 319 us) slower
// were 64 rows a wave, with operands read for twice the rows but one wave a SIMD (207 and 344),
// and all scores of a step before the product with V (182 and 321). D 64 forms as many weights
// for half of the products: 104 us for 4096 tokens (660 TFLOP/s). e4m3 steps pay for their
// conversion: 16 chunks of 1 to 701 tokens behind 0 to 4099 positions 286 us, 750 TFLOP/s; the
// LDS bank conflicts of the converted pieces (9% of its cycles) cost nothing (306 us, 309 without).
template <int ND, bool E4M3>
__global__ __launch_bounds__(256, ND == 2 ? 3 : 2) void chunk_tiles_kernel(ChunkArgs a, ChunkPlan plan, ChunkWorkspace ws) {
    constexpr int D = ND * 32, M = 128, NK = D / 16, NO = D / 32;
    constexpr int kKs = D + 8, kVs = D + 32;
    __shared__ __attribute__((aligned(16))) uint16_t s_K[4][kSub * kKs], s_V[4][kSub * kVs];
    __shared__ __attribute__((aligned(16))) float s_ks[8][kSub], s_vs[8][kSub];
    __shared__ uint32_t s_row[8][2 * kSub];
    __shared__ uint32_t s_odd[kOddSteps];  // of the steps that not all rows see: keys with values that are not finite
    const int tid = threadIdx.x, lane = tid & (kWave - 1), w = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int lr = lane & 31, lg = lane >> 5;
    const int hk = blockIdx.x % a.Hk;
    const ChunkUnit u = find_unit<false>(a, plan, blockIdx.x / a.Hk);
    if (blockIdx.x == 0 && w == 0) chunk_status(a, plan, u.bad);
    if (!u.ok) return;
    const ChunkKeys kk = chunk_keys(a, plan, u);
    const int H = a.H, g = plan.g, R = u.n * g, row0 = u.block * M;
    const int32_t* table = a.page_table + (size_t)u.seq * a.max_pages;
    const int n = (kk.k1 - kk.k0 + kSub - 1) / kSub;  // steps
    const bool active = row0 + 32 * w < R;

    // this lane's rows: their positions and queries (with the sign of the scores' factor)
    const int row = min(row0 + 32 * w + lr, R - 1), token = page_of(row, plan.by_g), own = u.old + token;
    const size_t at = ((size_t)u.start + token) * H + hk * g + (row - token * g);  // in q and o
    bf16x8 q[NK];
    const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;
#pragma unroll
    for (int i = 0; i < NK; ++i) {
        const uint4 v = gload((const uint4*)((const uint16_t*)a.q + at * D + 8 * lg + 16 * i));
        q[i] = as_operand(make_uint4(v.x ^ flip, v.y ^ flip, v.z ^ flip, v.w ^ flip));
    }
    const int own_min = u.old + page_of(row0, plan.by_g), own_max = u.old + page_of(min(R, row0 + M) - 1, plan.by_g);
    const float c = fmaxf(fabsf(a.scale_log2), 1.17549435e-38f);  // (0 becomes the smallest normal: a masked score of -inf stays one)

    // The steps whose keys every row of the block sees: those of the sinks, and [whole0, whole1)
    const int sink_steps = min(n, max(0, (kk.sinks - kk.k0) / kSub));
    int whole0, whole1;
    {
        const long long from = max((long long)kk.sinks, (long long)own_max - a.window - kk.lo + kk.sinks + 1) - kk.k0;
        const int to = min(kk.k1, own_min - kk.lo + kk.sinks + 1) - kk.k0;
        whole0 = (int)max((long long)sink_steps, (from + kSub - 1) / kSub);
        whole1 = max(whole0, max(0, to) / kSub);
    }
    auto full = [&](int s) TSV_INLINE { return s < sink_steps || (s >= whole0 && s < whole1); };
    // the others in turn, [sink_steps, whole0) and from whole1 on
    auto odd_of = [&](int s) TSV_INLINE { return min(s < whole0 ? s - sink_steps : s - whole1 + whole0 - sink_steps, kOddSteps - 1); };

    // ---- keys and values on their way. Group m: steps 2 m - 1 and 2 m (m = 0: step 0 alone).
    constexpr int EB = E4M3 ? 1 : 2;
    constexpr int RR = 256 / (D * EB / 16);  // rows that a load of all threads covers
    constexpr int L = 2 * kSub / RR;         // loads of a group's keys, and of its values
    static_assert(L * RR == 2 * kSub, "whole loads");
    const int prow = tid / (D * EB / 16), pcol = tid % (D * EB / 16) * 16;
    struct Keys {
        uint4 u[L];
        float ks, vs;
    } rk;
    uint4 rv[L];
    const char* k_from = (const char*)a.k_cache + pcol;
    const char* v_from = (const char*)a.v_cache + pcol;
    int page;
    auto virt = [&](int m, int i) TSV_INLINE { return min(max(kk.k0, kk.k0 + kSub * (2 * m - 1) + i), kk.k1 - 1); };  // key i of group m
    // wave w looks up the pages and rows of group m + w, for all
    auto look_up = [&](int m) TSV_INLINE { page = table[page_of(chunk_pos(kk, virt(m + w, lane)), a.div)]; };
    auto find_rows = [&](int m) TSV_INLINE { s_row[(m + w) & 7][lane] = chunk_row(a, page, hk, chunk_pos(kk, virt(m + w, lane))); };
    auto request_K = [&](int m, Keys& rk) TSV_INLINE {
#pragma unroll
        for (int i = 0; i < L; ++i) rk.u[i] = gload((const uint4*)(k_from + (size_t)s_row[m & 7][prow + i * RR] * (D * EB)));
        if (E4M3 && w == 0) {
            rk.ks = gload(a.k_scale + s_row[m & 7][lane]);
            rk.vs = gload(a.v_scale + s_row[m & 7][lane]);
        }
    };
    auto request_V = [&](int m) TSV_INLINE {
#pragma unroll
        for (int i = 0; i < L; ++i) rv[i] = gload((const uint4*)(v_from + (size_t)s_row[m & 7][prow + i * RR] * (D * EB)));
    };
    // `first`: 2 m - 1 modulo 4, the ring's place of a group's first step
    auto store_K = [&](int m, int first, const Keys& rk) TSV_INLINE {
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const int key = prow + i * RR, col = pcol / EB;
            uint16_t* to = &s_K[(first + (RR > kSub ? key : i * RR) / kSub) & 3][(RR > kSub ? key % kSub : prow + i * RR % kSub) * kKs + col];
            if (E4M3) {
                *(uint4*)to = e4m3_to_bf16(make_uint2(rk.u[i].x, rk.u[i].y));
                *(uint4*)(to + 8) = e4m3_to_bf16(make_uint2(rk.u[i].z, rk.u[i].w));
            } else {
                *(uint4*)to = rk.u[i];
            }
        }
        if (E4M3 && w == 0) {
            // a value row's scale that is not finite: as its elements (below). Past the last key its
            // row was read again: a key there has no position, and is none of those
            const int s = 2 * m - 1 + lane / kSub, k = kSub * (2 * m - 1) + lane;
            float vs = rk.vs;
            if (nonfinite(vs) && !full(s)) {
                if (k >= 0 && k < kk.k1 - kk.k0) atomicOr(&s_odd[odd_of(s)], 1u << (lane % kSub));
                vs = 0.f;
            }
            s_ks[s & 7][lane % kSub] = rk.ks;
            s_vs[s & 7][lane % kSub] = vs;
        }
    };
    auto store_V = [&](int m, int first) TSV_INLINE {
        const bool plain = m > 0 && full(2 * m - 1) && full(2 * m);
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const int key = prow + i * RR, col = pcol / EB;
            uint16_t* to = &s_V[(first + (RR > kSub ? key : i * RR) / kSub) & 3][(RR > kSub ? key % kSub : prow + i * RR % kSub) * kVs + col];
            uint4 x[2] = {rv[i], rv[i]};
            if (E4M3) {
                x[0] = e4m3_to_bf16(make_uint2(rv[i].x, rv[i].y));
                x[1] = e4m3_to_bf16(make_uint2(rv[i].z, rv[i].w));
            }
#pragma unroll
            for (int h = 0; h < (E4M3 ? 2 : 1); ++h) {
                if (!plain) {
                    // past the last key its row was read again: 0 in its place. A value that is not
                    // finite may reach the rows that see it only, but a product would carry it to
                    // all of them, at weight 0: it enters as 0, and those rows add it afterwards
                    const int k = kSub * (2 * m - 1) + key;
                    if (k < 0 || k >= kk.k1 - kk.k0) {
                        x[h] = make_uint4(0, 0, 0, 0);
                    } else if ((nonfinite_bits(x[h]) & 0x80008000u) && !full(k / kSub)) {
                        atomicOr(&s_odd[odd_of(k / kSub)], 1u << (k % kSub));
                        x[h] = only_finite(x[h]);
                    }
                }
                *(uint4*)(to + 8 * h) = x[h];
            }
        }
    };

    // the pages are checked while the queries and the first steps' pages are on their way (with
    // two groups of keys at once below, and masks of two compares: 4096 tokens in a window of 1024
    // 92.5 us, 100.4 before)
    look_up(0);
    if (chunk_check<256>(a, u, hk, ws)) return;

    const ChunkSeen seen = chunk_seen(a, kk, own);
    float base = -FLT_MAX, l = 0.f;
    f32x16 o[NO], sa, sb;
    bf16x8 pa[2] = {}, pb[2];
#pragma unroll
    for (int i = 0; i < NO; ++i) o[i] = f32x16{};
    auto scores = [&](f32x16& to) TSV_INLINE {  // of step 0
        to = f32x16{};
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            const bf16x8 kf = *(const bf16x8*)&s_K[0][lr * kKs + 16 * i + 8 * lg];
            to = mma(kf, q[i], to);
        }
    };
    auto product = [&](int s, const bf16x8 (&p)[2]) TSV_INLINE {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int i = 0; i < NO; ++i) {
                const bf16x8 vf = read_columns32(&s_V[s & 3][16 * x * kVs + 32 * i], kVs, lane);
                o[i] = mma(vf, p[x], o[i]);
            }
        }
    };
    // Step s: its weights, the scores of the next and the product of the one before. The
    // weights are 2^(c score - base); base is a maximum that moves, and all sums with it,
    // only when a score passes it by kSlack.
    float al = 1.f;
    bool moved = false;
    auto rescale = [&]() TSV_INLINE {
        if (!moved) return;
#pragma unroll
        for (int i = 0; i < NO; ++i) o[i] *= al;
    };
    auto step = [&](int s, int slot, f32x16& t, f32x16& sn, const bf16x8 (&p)[2], bf16x8 (&pn)[2]) TSV_INLINE {
        if (E4M3) {
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                const f32x4 ks = *(const f32x4*)&s_ks[s & 7][2 * e + 4 * lg];
#pragma unroll
                for (int i = 0; i < 4; ++i) t[e + i] *= ks[i];
            }
        }
        if (!full(s)) {
            asm volatile("");  // (or the compiler does this for every step)
            const int from = kk.k0 + kSub * s + 4 * lg;
#pragma unroll
            for (int e = 0; e < 16; ++e) t[e] = e / 4 * 8 + e % 4 < seen.hi - from ? t[e] : -INFINITY;
            if (s < whole0) {  // the windows' start
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int v = from + e / 4 * 8 + e % 4;
                    t[e] = v >= seen.lo || v < a.sinks ? t[e] : -INFINITY;
                }
            }
        }
        float mx = max3(t[0], t[1], t[2]), my = max3(t[3], t[4], t[5]);
#pragma unroll
        for (int e = 6; e < 14; e += 4) {
            mx = max3(mx, t[e], t[e + 1]);
            my = max3(my, t[e + 2], t[e + 3]);
        }
        mx = max3(max3(mx, my, my), t[14], t[15]);
        rescale();  // of the step before: the sums have its predecessor's product now
        moved = __ballot(fmaf(mx, c, -base) > kSlack) != 0;
        if (moved) {
            const float top = row_max<32>(mx);
            const float to = fmaf(top, c, -base) > kSlack ? top * c : base;
            al = __builtin_amdgcn_exp2f(base - to);
            l *= al;
            base = to;
        }
        // Slots of a product each, of the scores and with V in turn, with their share of the
        // weights beside them; operands come from LDS two slots ahead, three, four and six
        // being no faster (fences: the compiler would read all of K and V into registers first).
        // The wave goes first meanwhile (4096 tokens, at an earlier step: 177 us, 183 without)
        __builtin_amdgcn_s_setprio(1);
        constexpr int SLOTS = NK + 2 * NO, EVERY = SLOTS / 8;
        static_assert(NK == 2 * NO && SLOTS % 8 == 0, "as many slots of each, whole slots of a pair of weights");
        auto operand = [&](int j) TSV_INLINE {
            const int i = j / 2;
            return j % 2 == 0 ? *(const bf16x8*)&s_K[(slot + 1) & 3][lr * kKs + 16 * i + 8 * lg]
                          : read_columns32(&s_V[(slot + 3) & 3][16 * (i / NO) * kVs + 32 * (i % NO)], kVs, lane);
        };
        uint32_t b[8];
        float x[3][2];
        auto exponentials = [&](int y) TSV_INLINE {
            x[y % 3][0] = __builtin_amdgcn_exp2f(x[y % 3][0]);
            x[y % 3][1] = __builtin_amdgcn_exp2f(x[y % 3][1]);
        };
        auto weights = [&](int y) TSV_INLINE {
            float x0 = x[y % 3][0], x1 = x[y % 3][1];
            l += x0;  // of this lane's keys; the lanes of a row meet at the end
            l += x1;
            if (E4M3) {
                const float2 vs = *(const float2*)&s_vs[s & 7][y / 2 * 8 + 4 * lg + 2 * y % 4];
                x0 *= vs.x;
                x1 *= vs.y;
            }
            b[y] = pack_bf16x2(x0, x1);
            asm volatile("" : "+v"(b[y]), "+v"(l));  // (the compiler would move the weights behind all products)
        };
        constexpr int AHEAD = 2;
        bf16x8 f[AHEAD + 1];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) f[j] = operand(j);
        sn = f32x16{};
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
            if (j + AHEAD < SLOTS) f[(j + AHEAD) % (AHEAD + 1)] = operand(j + AHEAD);
            if (j % 2 == 0)
                sn = mma(f[j % (AHEAD + 1)], q[j / 2], sn);
            else
                o[j / 2 % NO] = mma(f[j % (AHEAD + 1)], p[j / 2 / NO], o[j / 2 % NO]);
            // pair y of weights: its arguments, a slot later its exponentials, and another one later
            // the rest, so that no instruction waits for the one before it (168 us, all in one slot 172)
            if (j % EVERY == 0) {
                const int y = j / EVERY;
                x[y % 3][0] = fmaf(t[2 * y], c, -base);
                x[y % 3][1] = fmaf(t[2 * y + 1], c, -base);
            }
            if (j >= 1 && (j - 1) % EVERY == 0) exponentials((j - 1) / EVERY);
            if (j >= 2 && (j - 2) % EVERY == 0) weights((j - 2) / EVERY);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (EVERY == 1) exponentials(7);
        if (EVERY == 1) weights(6);
        weights(7);
        __builtin_amdgcn_s_setprio(0);
        pn[0] = as_operand(make_uint4(b[0], b[1], b[2], b[3]));
        pn[1] = as_operand(make_uint4(b[4], b[5], b[6], b[7]));
    };
    // the elements of a key's value that are not finite, to the rows that see it
    auto add_odd = [&](int i) TSV_INLINE {
        const int v = kk.k0 + i, pos = chunk_pos(kk, v);
        if (v >= kk.k1) return;  // no key of this part: its page is not one that was checked
        const uint32_t at = chunk_row(a, table[page_of(pos, a.div)], hk, pos);
        const bool sees = v < seen.hi && (v >= seen.lo || v < a.sinks), scaled = !E4M3 || !nonfinite(gload(a.v_scale + at));
#pragma unroll
        for (int e = 0; e < NO * 16; ++e) {
            const size_t d = (size_t)at * D + e / 16 * 32 + e % 16 / 4 * 8 + 4 * lg + e % 4;
            const uint16_t b = !E4M3 ? gload((const uint16_t*)a.v_cache + d) : !scaled || (gload((const uint8_t*)a.v_cache + d) & 0x7f) == 0x7f ? 0x7fc0 : 0;
            if (sees && (b & 0x7f80) == 0x7f80) o[e / 16][e % 16] += bf16_bits_to_f32(b);
            if (e % 4 == 3) __builtin_amdgcn_sched_barrier(0);
        }
    };

    if (n > 0) {
        if (tid < kOddSteps) s_odd[tid] = 0;
        find_rows(0);
        look_up(4);
        lds_barrier();
        // in the rings: groups 0 and 1 of the keys, 0 of the values
        Keys r0;
        request_K(0, r0);
        request_K(1, rk);
        request_V(0);
        store_K(0, 3, r0);
        store_K(1, 1, rk);
        store_V(0, 3);
        // on their way: group 2 of the keys, 1 of the values
        request_V(1);
        request_K(2, rk);
        lds_barrier();
        if (active) scores(sa);
        for (int s = 0; s < n; s += 4) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // Until the next barrier the waves read the keys of steps s + 1 and s + 2 and the values
                // of s - 1 and s, and write the keys of s + 3 and s + 4 and the values of s + 1 and s + 2
                // (h = 1: two steps on)
                const int J = s / 2 + h, slot = 2 * h;
                if (h == 1 && s + 2 >= n) break;
                lds_barrier();
                store_K(J + 2, slot + 3, rk);
                store_V(J + 1, slot + 1);
                request_V(J + 2);
                request_K(J + 3, rk);
                if (h == 0 && s % 8 == 0) {
                    find_rows(J + 4);
                    look_up(J + 8);
                }
                if (!active) continue;
                step(s + slot, slot, sa, sb, pa, pb);
                if (s + slot + 1 >= n) {  // an odd number of steps
                    pa[0] = pb[0];
                    pa[1] = pb[1];
                    break;
                }
                step(s + slot + 1, slot + 1, sb, sa, pb, pa);
            }
        }
        lds_barrier();
        if (active) {
            rescale();
            product(n - 1, pa);
            for (int i = 0; i < kOddSteps; ++i) {
                const int s = i < whole0 - sink_steps ? sink_steps + i : whole1 + i - (whole0 - sink_steps);
                for (uint32_t odd = s_odd[i]; odd; odd &= odd - 1) add_odd(kSub * s + __builtin_ctz(odd));
            }
        }
    }
    const float sum = row_sum<32>(l);
    if (row0 + 32 * w + lr >= R) return;
    if (u.parts > 1) {
        const size_t slot = ((size_t)u.slot * a.Hk + hk) * M + 32 * w + lr;
        float* to = ws.o + slot * D + 4 * lg;
#pragma unroll
        for (int e = 0; e < D / 2; e += 4) {
            const f32x16& v = o[e / 16];
            *(f32x4*)(to + 2 * e) = f32x4{v[e % 16], v[e % 16 + 1], v[e % 16 + 2], v[e % 16 + 3]};
        }
        if (lg == 0) {
            ws.ml[slot * 2] = base;
            ws.ml[slot * 2 + 1] = sum;
        }
    } else {
        const float inv = 1.f / sum;
        // a lane has four elements of each eight; two lanes exchange them so that each has eight
        // neighbours to store
        uint16_t* to = (uint16_t*)a.o + at * D + 8 * lg;
#pragma unroll
        for (int e = 0; e < D / 2; e += 8) {
            const f32x16& v = o[e / 16];
            uint32_t b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = pack_bf16x2(v[e % 16 + 2 * i] * inv, v[e % 16 + 2 * i + 1] * inv);
            const auto x = __builtin_amdgcn_permlane32_swap(b[0], b[2], false, false), y = __builtin_amdgcn_permlane32_swap(b[1], b[3], false, false);
            gstore((uint4*)(to + 2 * e), make_uint4(x[0], y[0], x[1], y[1]));
        }
    }
}

template <int ND, bool E4M3>
void launch_nd(const ChunkArgs& a, const ChunkPlan& p, const ChunkWorkspace& ws, dim3 grid, hipStream_t stream) {
    if (p.rows == 16)
        hipLaunchKernelGGL((chunk_rows_kernel<ND, E4M3>), grid, dim3(256), 0, stream, a, p, ws);
    else
        hipLaunchKernelGGL((chunk_tiles_kernel<ND, E4M3>), grid, dim3(256), 0, stream, a, p, ws);
}

}  // namespace

void launch_chunk_mfma(const ChunkArgs& a, bool e4m3, const ChunkPlan& p, const ChunkWorkspace& ws, dim3 grid, hipStream_t stream) {
    if (a.D == 64)
        e4m3 ? launch_nd<2, true>(a, p, ws, grid, stream) : launch_nd<2, false>(a, p, ws, grid, stream);
    else
        e4m3 ? launch_nd<4, true>(a, p, ws, grid, stream) : launch_nd<4, false>(a, p, ws, grid, stream);
}

}  // namespace tsv
