// attn_mfma.hip -- tree attention over the paged cache on bf16 matrix
// instructions (head_dim 64 or 128, cache in bf16 or e4m3).
//
// Both kernels form the scores transposed, S^T = K Q^T (16 keys x 16 rows a
// tile, or 32 x 32): a lane then holds the keys 4 (l / 16) + r of one row l % 16, so
// that the softmax statistics of a row are a reduction in registers and over four
// lanes, the factor of a rescaling is one value per lane, and two tiles of weights
// are the operand of the next product, O^T = V^T P^T, as they are. V^T comes from
// LDS through the transposing read, in the same order of keys.
//   rows   up to 16 rows (node, query head) share a key head: one new token, or a
//          small tree. Four waves take 32 keys each in turn and meet at the end;
//          K goes from memory into the operand registers directly. Bound by the
//          cache's bytes: 65533 positions, 8 key heads of 128, 51 us (5.2 TB/s);
//          64 items of 17 to 8190 positions in e4m3, 111 us (5.0 TB/s).
//   tiles  more rows: a wave has 16 or 32 rows of its own, and 64 keys at a time
//          are shared in LDS by four waves. 32 rows halve the LDS reads of a row
//          (and keep two waves a SIMD). Bound by matrix and vector work, which
//          hardly overlap: 32 trees of 63 nodes over 300 to 4099 positions, 32
//          query heads, 124 us (0.6 PFLOP/s; matrix unit busy 32% of the time, vector
//          issue 37%). Tried and not kept there: two LDS buffers and one barrier a
//          tile (127 to 145 us), requests while the scores' product runs (124 us).
// In both, the loads of the next keys are under way while these are worked on,
// and the page of a key is looked up one step before its row is loaded.
#include <cfloat>

#include "attn_lanes.hpp"
#include "mfma_util.hpp"

namespace tsv {
namespace {

constexpr int kStepKeys = 32;  // keys of a wave's step in the row kernel

// q with the sign of the scores' factor
__device__ __forceinline__ bf16x8 query_operand(const AttnArgs& a, uint4 u) {
    const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;
    return as_operand(make_uint4(u.x ^ flip, u.y ^ flip, u.z ^ flip, u.w ^ flip));
}

// A node's value that is not finite may reach the rows that see the node only,
// but a product would carry it to all rows, at weight 0. So such elements enter
// the product as 0 (only_finite), and afterwards each row adds those of the nodes it sees.
// v: the node's values from this lane's first d on; o's element e holds d = e / 4 * STEP + e % 4
template <int NO, int STEP = 16, class Acc>
__device__ __forceinline__ void add_nonfinite(const uint16_t* v, Acc* o) {
    constexpr int NR = sizeof(Acc) / 4;
#pragma unroll
    for (int i = 0; i < NO * NR; ++i) {
        const uint16_t b = gload(v + i / 4 * STEP + i % 4);
        if ((b & 0x7f80) == 0x7f80) o[i / NR][i % NR] += bf16_bits_to_f32(b);
    }
}

// ---------------------------------------------------------------- rows
// ND = D / 32; E4M3: the cache's type
template <int ND, bool E4M3>
__global__ __launch_bounds__(256, 3) void attn_rows_kernel(AttnArgs a, AttnPlan plan, AttnWorkspace ws) {
    constexpr int D = ND * 32, kVs = D + 16, kOs = D + 4;
    __shared__ __attribute__((aligned(8))) int s_red[6];
    __shared__ Part s_part;
    __shared__ __attribute__((aligned(16))) uint16_t s_V[4][kStepKeys * kVs];  // then the waves' outputs
    __shared__ __attribute__((aligned(16))) float s_ks[4][kStepKeys], s_vs[4][kStepKeys], s_ml[4][16][2];
    __shared__ uint32_t s_row[4][2][kStepKeys];
    __shared__ uint32_t s_anc[16];
    __shared__ int s_par[16];
    static_assert(sizeof(s_V) >= 4 * 16 * kOs * sizeof(float), "outputs take the place of V");
    const int tid = threadIdx.x, lane = tid & (kWave - 1), w = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int l16 = lane & 15, lg = lane >> 4;
    const int hk = blockIdx.x % a.Hk, part = blockIdx.x / a.Hk;
    const Part pt = find_part<256>(a.cache_len, a.batch, a.room, plan, part, false, s_red, &s_part);
    if (!pt.ok) return;
    const int b = pt.item, T = a.T, H = a.H, g = H / a.Hk, R = T * g;
    const bool last = pt.k == pt.n - 1;
    int st = pt.bad_len ? kStBadCache : 0;

    // this lane's row: query operand, k-slot e of step 2 j + h is d = 64 j + 16 lg + 8 h + e
    const int row = min(l16, R - 1), node = row / g, head = hk * g + row % g;
    bf16x8 q[ND];
    {
        const uint16_t* qp = (const uint16_t*)a.q + (((size_t)b * T + node) * H + head) * D + 16 * lg;
#pragma unroll
        for (int i = 0; i < ND; ++i) q[i] = query_operand(a, gload((const uint4*)(qp + 64 * (i / 2) + 8 * (i % 2))));
    }
    const float c = score_factor(a);
    if (last) {  // at most 16 nodes: one word of ancestors each
        int bits = 0;
        if (tid < T) {
            const int p = a.parent[(size_t)b * T + tid];
            s_par[tid] = p;
            bits = tid == 0 ? (p != -1 ? kStBadRoot : 0) : (p < 0 || p >= tid ? kStBadParent : 0);
        }
        if (__syncthreads_or(bits)) {
            st |= __syncthreads_or(bits & kStBadRoot) ? kStBadRoot : 0;
            st |= __syncthreads_or(bits & kStBadParent) ? kStBadParent : 0;
        } else {
            if (tid < T) {
                uint32_t m = 0;
                for (int j = tid; j >= 0; j = s_par[j]) m |= 1u << j;
                s_anc[tid] = m;
            }
            __syncthreads();
        }
    }

    float base = -FLT_MAX, l = 0.f;  // the row's maximum, c times its largest score, as it is rounded
    f32x4 o[D / 16];
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[i] = f32x4{0.f, 0.f, 0.f, 0.f};

    // softmax and product of 32 keys: s the raw scores (masked: -inf), vs the factor
    // of each value row; V in this wave's LDS
    auto take = [&](const f32x4* s, const f32x4* vs) {
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
        if (E4M3 && vs) {
#pragma unroll
            for (int e = 0; e < 8; ++e) p[e] *= vs[e / 4][e % 4];  // (0 of a key past the last one)
        }
        // weights as two bf16 parts: with the cache's bytes the bound, their rounding
        // need not be a part of the result's error. The upper 16 bits, and what is left
        // with 2^-23 of the weight: both parts are positive, so that an infinite value
        // times them is one infinity (0 times it, or a part of the other sign, makes a NaN)
        uint32_t hi[4], lo[4];
        constexpr float kUp = 1.f + 0x1p-23f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            hi[e] = __builtin_amdgcn_perm(__float_as_uint(p[2 * e + 1]), __float_as_uint(p[2 * e]), 0x07060302u);
            lo[e] = pack_bf16x2(fmaf(p[2 * e], kUp, -__uint_as_float(hi[e] << 16)),
                                fmaf(p[2 * e + 1], kUp, -__uint_as_float(hi[e] & 0xffff0000u)));
        }
        const bf16x8 pf = as_operand(make_uint4(hi[0], hi[1], hi[2], hi[3])), pl = as_operand(make_uint4(lo[0], lo[1], lo[2], lo[3]));
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            const bf16x8 v = read_columns(&s_V[w][16 * i], kVs, lane);
            o[i] = mma(v, pf, o[i]);
            o[i] = mma(v, pl, o[i]);
        }
    };

    // the tree's own keys, in the wave that has the fewest cache steps, while the
    // first of the cache's are on their way
    auto take_tree = [&]() {
        if (!last || st || w != 3) return;
        const uint16_t* kp = (const uint16_t*)a.k + ((size_t)b * T * a.Hk + hk) * D;
        const uint16_t* vp = (const uint16_t*)a.v + ((size_t)b * T * a.Hk + hk) * D;
        const size_t stride = (size_t)a.Hk * D;
        f32x4 s[2];
        s[0] = s[1] = f32x4{0.f, 0.f, 0.f, 0.f};
        const uint16_t* krow = kp + (size_t)min(l16, T - 1) * stride + 16 * lg;
#pragma unroll
        for (int i = 0; i < ND; ++i)
            s[0] = mma(as_operand(gload((const uint4*)(krow + 64 * (i / 2) + 8 * (i % 2)))), q[i], s[0]);
        const uint32_t anc = s_anc[node];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int j = 4 * lg + r;
            s[0][r] = j < T && (anc >> j & 1) ? s[0][r] : -INFINITY;
            s[1][r] = -INFINITY;
        }
        uint32_t strange = 0;  // nodes whose values are not all finite, of this lane's pieces
        for (int i = lane; i < kStepKeys * (D / 8); i += kWave) {
            const int key = i / (D / 8), c = i % (D / 8) * 8;
            uint4 u = key < T ? gload((const uint4*)(vp + (size_t)key * stride + c)) : make_uint4(0, 0, 0, 0);
            if (nonfinite_bits(u) & 0x80008000u) {
                strange |= 1u << key;
                u = only_finite(u);
            }
            *(uint4*)&s_V[w][key * kVs + c] = u;
        }
        wave_sync();
        take(s, nullptr);
        if (__ballot(strange != 0)) {
#pragma unroll
            for (int x = 1; x < kWave; x <<= 1) strange |= __shfl_xor(strange, x, kWave);
            for (int j = 0; j < T; ++j)
                if (strange & anc & (1u << j)) add_nonfinite<D / 16>(vp + (size_t)j * stride + 4 * lg, o);
        }
        wave_sync();
    };

    // the cache: wave w has steps w, w + 4, ...
    const int k0 = pt.k * pt.keys, k1 = last ? pt.len : min(pt.len, k0 + pt.keys);
    int bad = 0;
    if (k1 > k0 && a.n_pages > 0) {
        constexpr int EB = E4M3 ? 1 : 2;          // bytes of an element
        constexpr int KL = E4M3 ? ND / 2 : ND;    // 16-byte loads of a key's lane
        constexpr int VL = kStepKeys * D * EB / 16 / kWave;  // of V per lane
        constexpr int VR = kWave / (D * EB / 16);            // rows of V a load covers
        const char* kc = (const char*)a.k_cache;
        const char* vc = (const char*)a.v_cache;
        const int32_t* table = a.page_table + (size_t)b * a.max_pages;
        uint4 rk[2][KL], rv[VL];
        float rks = 1.f, rvs = 1.f;
        int page = 0;  // of this lane's key (lane % 32) of the step after the one being requested
        auto key_of = [&](int t) { return min(t + (lane & 31), k1 - 1); };
        auto look_up = [&](int t) { page = table[page_of(key_of(t), a.div)]; };
        auto request_rows = [&](int t, int set) {  // row of each key, to all lanes
            const bool fine = page_ok(a, page);
            bad |= !fine;
            const uint32_t r = cache_row(a, fine ? page : 0, hk, key_of(t));
            if (lane < kStepKeys) s_row[w][set][lane] = r;
            if (E4M3) {
                rks = gload(a.k_scale + r);
                rvs = gload(a.v_scale + r);
            }
            wave_sync();
        };
        auto request_K = [&](int set) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const char* p = kc + (size_t)s_row[w][set][16 * t + l16] * (D * EB) + lg * (E4M3 ? 16 : 32);
#pragma unroll
                for (int i = 0; i < KL; ++i)
                    rk[t][i] = gload((const uint4*)(p + (E4M3 ? 64 * i : 128 * (i / 2) + 16 * (i % 2))));
            }
        };
        auto request_V = [&](int set) {
#pragma unroll
            for (int i = 0; i < VL; ++i) {
                const int key = i * VR + lane / (D * EB / 16), c = lane % (D * EB / 16) * 16;
                rv[i] = gload((const uint4*)(vc + (size_t)s_row[w][set][key] * (D * EB) + c));
            }
        };
        int t = k0 + w * kStepKeys, set = 0;
        if (t < k1) {
            look_up(t);
            request_rows(t, 0);
            request_K(0);
            request_V(0);
            look_up(t + 4 * kStepKeys);
        }
        take_tree();
        for (; t < k1; t += 4 * kStepKeys, set ^= 1) {
            const bool more = t + 4 * kStepKeys < k1;
            if (E4M3) {
                if (lane < kStepKeys) {
                    s_ks[w][lane] = rks;
                    s_vs[w][lane] = t + lane < k1 ? rvs : 0.f;
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
                request_rows(t + 4 * kStepKeys, set ^ 1);
                request_K(set ^ 1);
            }
            // V into LDS, its registers free for the next step
#pragma unroll
            for (int i = 0; i < VL; ++i) {
                const int key = i * VR + lane / (D * EB / 16), c = lane % (D * EB / 16) * (16 / EB);
                if (E4M3) {
                    *(uint4*)&s_V[w][key * kVs + c] = e4m3_to_bf16(make_uint2(rv[i].x, rv[i].y));
                    *(uint4*)&s_V[w][key * kVs + c + 8] = e4m3_to_bf16(make_uint2(rv[i].z, rv[i].w));
                } else {
                    *(uint4*)&s_V[w][key * kVs + c] = rv[i];
                }
            }
            if (more) {
                request_V(set ^ 1);
                look_up(t + 8 * kStepKeys);
            }
            if (t + kStepKeys > k1) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (t + 16 * (e / 4) + 4 * lg + e % 4 >= k1) s[e / 4][e % 4] = -INFINITY;
                // past the last key its row was read again: 0 in its place, since the weight 0
                // would make a NaN of a value that is not finite
                for (int i = (k1 - t) * (D / 8) + lane; i < kStepKeys * (D / 8); i += kWave)
                    *(uint4*)&s_V[w][i / (D / 8) * kVs + i % (D / 8) * 8] = make_uint4(0, 0, 0, 0);
            }
            wave_sync();
            take(s, vs);
            wave_sync();
        }
    } else {
        bad = k1 > k0;  // positions without a page
        take_tree();
    }
    l = row_sum(l);

    // the four waves
    if (lg == 0) {
        s_ml[w][l16][0] = base;
        s_ml[w][l16][1] = l;
    }
    st |= __syncthreads_or(bad) ? kStBadCache : 0;
    float mt = -FLT_MAX, lt = 0.f;
#pragma unroll
    for (int x = 0; x < 4; ++x) mt = fmaxf(mt, s_ml[x][l16][0]);
#pragma unroll
    for (int x = 0; x < 4; ++x) lt += s_ml[x][l16][1] * __builtin_amdgcn_exp2f(s_ml[x][l16][0] - mt);
    {
        const float al = __builtin_amdgcn_exp2f(base - mt);
        float* so = (float*)s_V + (w * 16 + l16) * kOs + 4 * lg;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) *(f32x4*)(so + 16 * i) = o[i] * al;
    }
    // a row's m and l for all threads
    __shared__ float s_m[16], s_l[16];
    if (tid < 16) {
        s_m[tid] = mt;
        s_l[tid] = lt;
    }
    __syncthreads();
    if (hk == 0 && tid == 0) {
        if (pt.n > 1)
            ws.bits[part] = st;
        else if (a.status)
            a.status[b] = st;
    }
    if (pt.n == 1 && st) return;
    for (int i = tid; i < R * (D / 4); i += 256) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int x = 0; x < 4; ++x) v += *(const f32x4*)((const float*)s_V + (x * 16 + r) * kOs + d);
        const size_t at = (size_t)(r / g) * H + hk * g + r % g;
        if (pt.n > 1) {
            *(f32x4*)(ws.o + ((size_t)part * T * H + at) * D + d) = v;
            if (d == 0) {
                ws.ml[((size_t)part * T * H + at) * 2] = s_m[r];
                ws.ml[((size_t)part * T * H + at) * 2 + 1] = s_l[r];
            }
        } else {
            const float lr = s_l[r];
            gstore((uint2*)((uint16_t*)a.o + ((size_t)b * T * H + at) * D + d),
                   make_uint2(pack_bf16x2(v[0] / lr, v[1] / lr), pack_bf16x2(v[2] / lr, v[3] / lr)));
        }
    }
}

// ---------------------------------------------------------------- tiles
// NW waves of RW rows. Of a product's result, 16 x 16 or 32 x 32, a lane holds one
// column in pieces of four rows: its element e is in row e / 4 * (4 G) + 4 g + e % 4,
// with G = 64 / RW lanes per column, this lane the g-th of them.
template <int ND, bool E4M3, int NW, int RW>
__global__ __launch_bounds__(64 * NW, RW == 32 ? 2 : 3) void attn_tiles_kernel(AttnArgs a, AttnPlan plan, AttnWorkspace ws, int row_blocks) {
    typedef typename std::conditional<RW == 32, f32x16, f32x4>::type Acc;
    constexpr int D = ND * 32, TH = 64 * NW, M = RW * NW, G = kWave / RW, NR = RW * RW / kWave;
    constexpr int KS = 512 / RW;  // keys, or d, of one instruction
    constexpr int kKs = D + 8, kVs = D + RW;
    __shared__ __attribute__((aligned(8))) int s_red[NW + 2];
    __shared__ Part s_part;
    __shared__ __attribute__((aligned(16))) uint16_t s_K[kTileKeys * kKs], s_V[kTileKeys * kVs];
    __shared__ __attribute__((aligned(16))) float s_ks[kTileKeys], s_vs[kTileKeys];
    __shared__ uint32_t s_row[2][kTileKeys];
    __shared__ int s_par[1024];
    __shared__ uint32_t s_odd[32];  // nodes whose values are not all finite
    extern __shared__ uint32_t s_anc[];  // [nodes of the block][words of T bits]
    const int tid = threadIdx.x, lane = tid & (kWave - 1), w = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int lr = lane & (RW - 1), lg = lane / RW;
    // the row blocks that read one part of a key head run on one XCD; the parts
    // that there are come first, so neighbours go to different ones
    const int turn = blockIdx.x / 8, rb = turn % row_blocks, unit = turn / row_blocks * 8 + blockIdx.x % 8;
    const int hk = unit % a.Hk;
    Part pt = find_part<TH>(a.cache_len, a.batch, a.room, plan, unit / a.Hk, false, s_red, &s_part);
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
    if (last) st |= tree_words<TH>(a.parent + (size_t)b * T, T, first, last_node - first + 1, words, s_par, s_anc);
    if (tid < 32) s_odd[tid] = 0;

    // this lane's row
    const int row = row0 + RW * w + lr, node = min(row, R - 1) / g;
    bf16x8 q[D / KS];
    {
        const uint16_t* qp = (const uint16_t*)a.q + (((size_t)b * T + node) * H + hk * g + min(row, R - 1) % g) * D + 8 * lg;
#pragma unroll
        for (int i = 0; i < D / KS; ++i) q[i] = query_operand(a, gload((const uint4*)(qp + KS * i)));
    }
    const float c = score_factor(a);
    // The weights are 2^(c score - base). base is a maximum that moves, and all sums
    // with it, only when a score passes it by kSlack: the sums have room for 2^8 more
    // in fp32, and most tiles need neither their rows' maximum nor a rescaling
    // (moved for every new maximum: 164 us against 159, 32 trees of 63 nodes)
    float base = -FLT_MAX, l = 0.f;
    Acc o[D / RW];
#pragma unroll
    for (int i = 0; i < D / RW; ++i) o[i] = Acc{};

    // One tile of keys in LDS, `limit` of them: scores, softmax, product. TREE: keys
    // j0 + ... of the tree, by ancestors
    auto take = [&](auto tree, int limit, int j0) {
        constexpr bool TREE = decltype(tree)::value, SCALED = E4M3 && !TREE;
        constexpr int NX = kTileKeys / RW;
        Acc s[NX];
#pragma unroll
        for (int x = 0; x < NX; ++x) s[x] = Acc{};
        // (fences: the compiler would read all of K, or of V, into registers first)
#pragma unroll
        for (int i = 0; i < D / KS; ++i) {
#pragma unroll
            for (int x = 0; x < NX; ++x) s[x] = mma(*(const bf16x8*)&s_K[(RW * x + lr) * kKs + KS * i + 8 * lg], q[i], s[x]);
            if ((i + 1) * NX % 8 == 0) __builtin_amdgcn_sched_barrier(0);
        }
        float sc[RW];
#pragma unroll
        for (int e = 0; e < RW; ++e) sc[e] = s[e / NR][e % NR];
#pragma unroll
        for (int e = 0; e < RW; e += 4) {
            const int j = e * G + 4 * lg;  // the key of element e
            if (SCALED) {
                const f32x4 ks = *(const f32x4*)&s_ks[j];
#pragma unroll
                for (int r = 0; r < 4; ++r) sc[e + r] *= ks[r];
            }
            if (TREE) {
                const uint32_t bits = s_anc[(node - first) * words + min((j0 + j) / 32, words - 1)] >> ((j0 + j) % 32);
#pragma unroll
                for (int r = 0; r < 4; ++r) sc[e + r] = j + r < limit && (bits >> r & 1) ? sc[e + r] : -INFINITY;
            }
        }
        if (!TREE && limit < kTileKeys) {
            const int left = limit - 4 * lg;
#pragma unroll
            for (int e = 0; e < RW; ++e) sc[e] = e / 4 * 4 * G + e % 4 < left ? sc[e] : -INFINITY;
        }
        float mx = sc[0], my = sc[1];
#pragma unroll
        for (int e = 2; e < RW; e += 4) {
            mx = max3(mx, sc[e], sc[e + 1]);
            if (e + 2 < RW) my = max3(my, sc[e + 2], sc[e + 3]);
        }
        mx = max3(mx, my, my);
        if (__ballot(fmaf(mx, c, -base) > kSlack)) {
            const float top = row_max<RW>(mx);  // a row moves by its own scores alone: its bits do not follow from its neighbours'
            const float to = fmaf(top, c, -base) > kSlack ? top * c : base, al = __builtin_amdgcn_exp2f(base - to);
            l *= al;
#pragma unroll
            for (int i = 0; i < D / RW; ++i) o[i] *= al;
            base = to;
        }
        uint32_t u[RW / 2];
#pragma unroll
        for (int e = 0; e < RW; e += 4) {
            f32x4 p;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                p[r] = __builtin_amdgcn_exp2f(fmaf(sc[e + r], c, -base));
                l += p[r];  // of this lane's keys; the lanes of a row meet at the end
            }
            if (SCALED) {
                const f32x4 vs = *(const f32x4*)&s_vs[e * G + 4 * lg];
#pragma unroll
                for (int r = 0; r < 4; ++r) p[r] *= vs[r];  // (0 of a key past the last one)
            }
            // rounded once, unlike the row kernel's (at most 2^-8 of a weight; the outputs are
            // off by 0.0022 to 0.0023 of their size on average, by 0.0017 with exact weights):
            // a second part would be half of the matrix products again, which bound this kernel
            u[e / 2] = pack_bf16x2(p[0], p[1]);
            u[e / 2 + 1] = pack_bf16x2(p[2], p[3]);
        }
#pragma unroll
        for (int x = 0; x < kTileKeys / KS; ++x) {
            const bf16x8 pf = as_operand(make_uint4(u[4 * x], u[4 * x + 1], u[4 * x + 2], u[4 * x + 3]));
#pragma unroll
            for (int i = 0; i < D / RW; ++i) {
                const uint16_t* tile = &s_V[KS * x * kVs + RW * i];
                const bf16x8 v = RW == 32 ? read_columns32(tile, kVs, lane) : read_columns(tile, kVs, lane);
                o[i] = mma(v, pf, o[i]);
                if (i % 4 == 3) __builtin_amdgcn_sched_barrier(0);
            }
        }
    };

    // the tree's own keys, up to the block's last node, while the first of the
    // cache's are on their way
    auto take_tree = [&]() {
        if (!last || st) return;
        const size_t stride = (size_t)a.Hk * D;
        const uint16_t* kp = (const uint16_t*)a.k + ((size_t)b * T * a.Hk + hk) * D;
        const uint16_t* vp = (const uint16_t*)a.v + ((size_t)b * T * a.Hk + hk) * D;
        for (int j0 = 0; j0 <= last_node; j0 += kTileKeys) {
            lds_barrier();
            for (int i = tid; i < kTileKeys * (D / 8); i += TH) {
                const int key = i / (D / 8), c = i % (D / 8) * 8;
                uint4 ku = make_uint4(0, 0, 0, 0), vu = ku;
                if (j0 + key < T) {
                    ku = gload((const uint4*)(kp + (size_t)(j0 + key) * stride + c));
                    vu = gload((const uint4*)(vp + (size_t)(j0 + key) * stride + c));
                }
                if (nonfinite_bits(vu) & 0x80008000u) {
                    atomicOr(&s_odd[(j0 + key) / 32], 1u << ((j0 + key) % 32));
                    vu = only_finite(vu);
                }
                *(uint4*)&s_K[key * kKs + c] = ku;
                *(uint4*)&s_V[key * kVs + c] = vu;
            }
            lds_barrier();
            take(std::true_type(), T - j0, j0);
        }
        for (int x = 0; x < words; ++x) {
            if (!s_odd[x]) continue;
            for (int j = 0; j < 32; ++j)
                if (s_odd[x] & s_anc[(node - first) * words + x] & (1u << j))
                    add_nonfinite<D / RW, 4 * G>(vp + (size_t)(32 * x + j) * stride + 4 * lg, o);
        }
    };

    int bad = 0;
    if (k1 > k0 && a.n_pages > 0) {
        constexpr int EB = E4M3 ? 1 : 2;
        constexpr int L = kTileKeys * D * EB / 16 / TH;  // 16-byte loads of K, and of V, per thread
        static_assert(L * TH * 16 == kTileKeys * D * EB, "whole loads");
        constexpr int RR = TH / (D * EB / 16);           // rows that one of them covers
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
        find_rows(k0, 0);
        look_up(k0 + kTileKeys);
        __syncthreads();
        request(0);
        take_tree();
        int set = 0;
        for (int t = k0; t < k1; t += kTileKeys, set ^= 1) {
            lds_barrier();  // the last tile's reads are done
            if (t + kTileKeys > k1) {  // past the last key: as in the row kernel
#pragma unroll
                for (int i = 0; i < L; ++i)
                    if (prow + i * RR >= k1 - t) rv[i] = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const int key = prow + i * RR, c = pcol / EB;
                if (E4M3) {
                    *(uint4*)&s_K[key * kKs + c] = e4m3_to_bf16(make_uint2(rk[i].x, rk[i].y));
                    *(uint4*)&s_K[key * kKs + c + 8] = e4m3_to_bf16(make_uint2(rk[i].z, rk[i].w));
                    *(uint4*)&s_V[key * kVs + c] = e4m3_to_bf16(make_uint2(rv[i].x, rv[i].y));
                    *(uint4*)&s_V[key * kVs + c + 8] = e4m3_to_bf16(make_uint2(rv[i].z, rv[i].w));
                } else {
                    *(uint4*)&s_K[key * kKs + c] = rk[i];
                    *(uint4*)&s_V[key * kVs + c] = rv[i];
                }
            }
            if (E4M3 && w == 0) {
                s_ks[lane] = rks;
                s_vs[lane] = t + lane < k1 ? rvs : 0.f;
            }
            find_rows(t + kTileKeys, set ^ 1);
            lds_barrier();
            if (t + kTileKeys < k1) {
                request(set ^ 1);
                look_up(t + 2 * kTileKeys);
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
    l = row_sum<RW>(l);
    if (row >= R) return;
    const size_t at = (size_t)node * H + hk * g + row % g;
    if (pt.n > 1) {
        float* to = ws.o + ((size_t)part * T * H + at) * D + 4 * lg;
#pragma unroll
        for (int e = 0; e < D / G; e += 4) {
            const Acc& v = o[e / NR];
            *(f32x4*)(to + e * G) = f32x4{v[e % NR], v[e % NR + 1], v[e % NR + 2], v[e % NR + 3]};
        }
        if (lg == 0) {
            ws.ml[((size_t)part * T * H + at) * 2] = base;
            ws.ml[((size_t)part * T * H + at) * 2 + 1] = l;
        }
    } else {
        const float inv = 1.f / l;
        uint16_t* to = (uint16_t*)a.o + ((size_t)b * T * H + at) * D + 4 * lg;
#pragma unroll
        for (int e = 0; e < D / G; e += 4) {
            const Acc& v = o[e / NR];
            gstore((uint2*)(to + e * G), make_uint2(pack_bf16x2(v[e % NR] * inv, v[e % NR + 1] * inv),
                                                    pack_bf16x2(v[e % NR + 2] * inv, v[e % NR + 3] * inv)));
        }
    }
}

template <int ND, bool E4M3>
void launch_nd(const AttnArgs& a, const AttnPlan& p, const AttnWorkspace& ws, int block_rows, int row_blocks, hipStream_t stream) {
    const long long units = (long long)p.parts * a.Hk;
    const dim3 grid((unsigned)(block_rows == 16 ? units : (units + 7) / 8 * 8 * row_blocks));
    const int g = a.H / a.Hk;
    const unsigned words = (a.T + 31) / 32;
    const unsigned nodes = min(a.T, (block_rows + g - 2) / g + 1);
    const unsigned lds = nodes * words * 4;
    if (block_rows == 16)
        hipLaunchKernelGGL((attn_rows_kernel<ND, E4M3>), grid, dim3(256), 0, stream, a, p, ws);
    else if (block_rows == 64)
        hipLaunchKernelGGL((attn_tiles_kernel<ND, E4M3, 4, 16>), grid, dim3(256), lds, stream, a, p, ws, row_blocks);
    else
        hipLaunchKernelGGL((attn_tiles_kernel<ND, E4M3, 4, 32>), grid, dim3(256), lds, stream, a, p, ws, row_blocks);
}

}  // namespace

void launch_attn_mfma(const AttnArgs& a, bool e4m3, const AttnPlan& p, const AttnWorkspace& ws, int block_rows, int row_blocks,
                      hipStream_t stream) {
    if (a.D == 64)
        e4m3 ? launch_nd<2, true>(a, p, ws, block_rows, row_blocks, stream)
             : launch_nd<2, false>(a, p, ws, block_rows, row_blocks, stream);
    else
        e4m3 ? launch_nd<4, true>(a, p, ws, block_rows, row_blocks, stream)
             : launch_nd<4, false>(a, p, ws, block_rows, row_blocks, stream);
}

}  // namespace tsv
