// attn_rope.hip -- norms of the heads of queries and keys with the position rotation,
// in one pass: of rows of any kind (tree_attn_rope), or on the way of packed rows into
// the paged cache (tree_attn_append_rope).
//
//   z = w x / sqrt(mean x^2 + eps)   (without a weight: z = x)
//   (z_a, z_b) -> (z_a cos t - z_b sin t, z_b cos t + z_a sin t),  t = position inv_freq[i],
// for the R / 2 pairs (a, b) = (i, i + R/2), or (2 i, 2 i + 1), of a head; the other
// elements stay z.
//
// Bound by the rows' traffic. A lane has eight pairs of a head, so that both elements of a
// pair are its own and only the sum of squares leaves it: a head of D has D / 16 lanes
// (rounded up to a power of two), two 16-byte pieces each in bf16. The angles of a row are
// the same for all of its heads: the work-group forms them once, in LDS. An angle is a
// product in 64 bits, in revolutions, of which the whole ones are dropped before it is
// rounded to 32: at position 10^6 a product in 32 bits would be off by 0.06.
#include "attn_cache.hpp"

namespace tsv {
namespace {

constexpr int kRopeRows = 16;  // most rows of a work-group

// Element numbers of pair p
__device__ __forceinline__ int2 pair_of(const RopeArgs& a, int p) {
    const int half = a.R / 2;
    return p < half && !a.interleaved ? make_int2(p, p + half) : make_int2(2 * p, 2 * p + 1);
}

struct Pairs {
    float a[8], b[8];
};

// A lane's eight pairs: VEC: 8 j + i, as two pieces of eight elements; otherwise j + LPH i
template <typename TIO, int LPH, bool VEC>
struct Piece {
    Raw<TIO, VEC> lo, hi;
};

// First elements of the two pieces: the pairs' first and second ones, or (interleaved pairs,
// and elements that are not rotated) sixteen neighbours
__device__ __forceinline__ int2 pieces_of(const RopeArgs& a, int j) {
    return !a.interleaved && 16 * j < a.R ? make_int2(8 * j, a.R / 2 + 8 * j) : make_int2(16 * j, 16 * j + 8);
}

template <typename TIO, int LPH, bool VEC>
__device__ __forceinline__ Piece<TIO, LPH, VEC> load_pairs(const RopeArgs& a, const TIO* row, int j, int2 at) {
    Piece<TIO, LPH, VEC> p{};
    if constexpr (VEC) {
        if (16 * j >= a.D) return p;
        p.lo = load8<TIO, true>(row + at.x, 8);
        p.hi = load8<TIO, true>(row + at.y, 8);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int2 e = pair_of(a, j + LPH * i);
            p.lo.e[i] = e.x < a.D ? gload(row + e.x) : TIO(0);
            p.hi.e[i] = e.y < a.D ? gload(row + e.y) : TIO(0);
        }
    }
    return p;
}

// Pieces in the elements' order <-> pairs. Only interleaved pairs are not in their places
// (elements that are not rotated may pair in any way)
template <bool VEC>
__device__ __forceinline__ Pairs to_pairs(const RopeArgs& a, const Quad& lo, const Quad& hi) {
    Pairs p;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        p.a[i] = lo.v[i];
        p.b[i] = hi.v[i];
    }
    if (VEC && a.interleaved) {
        asm volatile("");  // (or the compiler selects, for both kinds)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            p.a[i] = i < 4 ? lo.v[2 * i] : hi.v[2 * i - 8];
            p.b[i] = i < 4 ? lo.v[2 * i + 1] : hi.v[2 * i - 7];
        }
    }
    return p;
}
template <bool VEC>
__device__ __forceinline__ void to_pieces(const RopeArgs& a, const Pairs& p, Quad& lo, Quad& hi) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo.v[i] = p.a[i];
        hi.v[i] = p.b[i];
    }
    if (VEC && a.interleaved) {
        asm volatile("");
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo.v[i] = i % 2 ? p.b[i / 2] : p.a[i / 2];
            hi.v[i] = i % 2 ? p.b[4 + i / 2] : p.a[4 + i / 2];
        }
    }
}

template <int LPH, bool VEC>
__device__ __forceinline__ Pairs load_weight(const RopeArgs& a, const float* w, int j, int2 at) {
    if (!w) return Pairs{};
    if constexpr (VEC) {
        if (16 * j >= a.D) return Pairs{};
        return to_pairs<true>(a, floats<float, true>(load8<float, true>(w + at.x, 8)), floats<float, true>(load8<float, true>(w + at.y, 8)));
    } else {
        Pairs p;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int2 e = pair_of(a, j + LPH * i);
            p.a[i] = e.x < a.D ? gload(w + e.x) : 0.f;
            p.b[i] = e.y < a.D ? gload(w + e.y) : 0.f;
        }
        return p;
    }
}

// Sum over the LPH <= 16 neighbouring lanes of a head
template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
#define TSV_ADD_DPP(ctrl) v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), ctrl, 0xf, 0xf, true))
    if (LPH >= 2) TSV_ADD_DPP(0xb1);    // quad_perm [1,0,3,2]
    if (LPH >= 4) TSV_ADD_DPP(0x4e);    // quad_perm [2,3,0,1]
    if (LPH >= 8) TSV_ADD_DPP(0x141);   // row_half_mirror
    if (LPH >= 16) TSV_ADD_DPP(0x140);  // row_mirror
#undef TSV_ADD_DPP
    return v;
}

// 8 neighbours, rounded to nearest even
template <typename TIO>
__device__ __forceinline__ void store_piece(TIO* to, const Quad& q) {
    if constexpr (sizeof(TIO) == 2) {
        gstore((uint4*)to, make_uint4(pack_bf16x2(q.v[0], q.v[1]), pack_bf16x2(q.v[2], q.v[3]), pack_bf16x2(q.v[4], q.v[5]),
                                      pack_bf16x2(q.v[6], q.v[7])));
    } else {
        gstore((float4*)to, make_float4(q.v[0], q.v[1], q.v[2], q.v[3]));
        gstore((float4*)to + 1, make_float4(q.v[4], q.v[5], q.v[6], q.v[7]));
    }
}
template <typename TIO, int LPH, bool VEC>
__device__ __forceinline__ void store_head(const RopeArgs& a, TIO* row, const Quad& lo, const Quad& hi, int j, int2 to) {
    if constexpr (VEC) {
        if (16 * j >= a.D) return;
        store_piece<TIO>(row + to.x, lo);
        store_piece<TIO>(row + to.y, hi);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int2 e = pair_of(a, j + LPH * i);
            if (e.x < a.D) Elem<TIO>::st(row, e.x, lo.v[i]);
            if (e.y < a.D) Elem<TIO>::st(row, e.y, hi.v[i]);
        }
    }
}
template <int LPH, bool VEC>
__device__ __forceinline__ void store_head_e4m3(const RopeArgs& a, uint8_t* row, const Quad& lo, const Quad& hi, int j, int2 to, float scale) {
    const bool finite = scale == scale;
    const uint2 ul = e4m3_bytes(lo, scale, finite), uh = e4m3_bytes(hi, scale, finite);
    if constexpr (VEC) {
        if (16 * j >= a.D) return;
        gstore((uint2*)(row + to.x), ul);
        gstore((uint2*)(row + to.y), uh);
    } else {
        const uint32_t wl[2] = {ul.x, ul.y}, wh[2] = {uh.x, uh.y};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int2 e = pair_of(a, j + LPH * i);
            if (e.x < a.D) row[e.x] = (uint8_t)(wl[i / 4] >> (8 * (i % 4)));
            if (e.y < a.D) row[e.y] = (uint8_t)(wh[i / 4] >> (8 * (i % 4)));
        }
    }
}

// Heads of a row: H of q, Hk of k, and where they go into the cache Hk of v.
// `rb` rows a work-group.
template <typename TIO, int LPH, bool VEC, bool APPEND, bool E4M3>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a, CacheWriteArgs c, int rb, int row_blocks) {
    __shared__ __attribute__((aligned(16))) float s_cos[kRopeRows][128], s_sin[kRopeRows][128];
    __shared__ RowPlaces<kRopeRows> places;
    constexpr int kSlots = 256 / LPH;
    const int tid = threadIdx.x, j = tid % LPH;
    const int2 at = pieces_of(a, j);
    const bool rows = (int)blockIdx.x < row_blocks;
    const int r0 = blockIdx.x * rb, n = rows ? min(rb, a.rows - r0) : 0;
    const int Hq = a.q ? a.H : 0, Hx = a.k ? a.Hk : 0, heads = Hq + (APPEND ? 2 : 1) * Hx, units = n * heads;
    typedef Piece<TIO, LPH, VEC> P;
    auto fetch = [&](int u) {
        P p{};
        if (u >= units) return p;
        const int row = page_of(u, a.heads), h = u - row * heads;
        const size_t r = (size_t)(r0 + row);
        const TIO* from = h < Hq ? (const TIO*)a.q + r * a.qs + (size_t)h * a.D
                                 : h < Hq + Hx ? (const TIO*)a.k + r * a.ks + (size_t)(h - Hq) * a.D
                                               : (const TIO*)a.v + r * a.vs + (size_t)(h - Hq - Hx) * a.D;
        return load_pairs<TIO, LPH, VEC>(a, from, j, at);
    };
    // the first rows are on their way while their places and angles are found
    int u = tid / LPH;
    P next = fetch(u);
    const Pairs wq = load_weight<LPH, VEC>(a, a.qw, j, at), wk = load_weight<LPH, VEC>(a, a.kw, j, at);
    if (APPEND) {
        if (!find_places<kRopeRows>(c, r0, n, rows ? -1 : (int)blockIdx.x - row_blocks, places)) return;
    } else {
        if (tid < n) places.place[tid] = a.position[r0 + tid];
        lds_barrier();
    }
    for (int i = tid; i < n * (a.R / 2); i += 256) {
        const int row = i / (a.R / 2), p = i - row * (a.R / 2);
        const double turns = (double)places.place[row] * (double)gload(a.inv_freq + p) * 0.15915494309189533577;  // 1 / (2 pi)
        const float t = (float)(turns - rint(turns));
        float sn, cs;
        sincospif(2.f * t, &sn, &cs);
        s_cos[row][p] = cs;
        s_sin[row][p] = sn;
    }
    lds_barrier();
    for (; u < units; u += kSlots) {
        const P now = next;
        next = fetch(u + kSlots);
        const int row = page_of(u, a.heads), h = u - row * heads;
        const int place = places.place[row];
        if (place < 0) continue;  // a row of no sequence, or left out by its position (the same for a head's lanes)
        const bool is_q = h < Hq, is_v = APPEND && h >= Hq + Hx;
        Quad lo = floats<TIO, VEC>(now.lo), hi = floats<TIO, VEC>(now.hi);
        if (!is_v) {
            Pairs x = to_pairs<VEC>(a, lo, hi);
            if (is_q ? a.qw != nullptr : a.kw != nullptr) {
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) sum = fmaf(x.a[i], x.a[i], fmaf(x.b[i], x.b[i], sum));
                sum = head_sum<LPH>(sum);
                const float r = 1.f / sqrtf(sum / (float)a.D + a.eps);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x.a[i] *= r * (is_q ? wq.a[i] : wk.a[i]);
                    x.b[i] *= r * (is_q ? wq.b[i] : wk.b[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int p = VEC ? 8 * j + i : j + LPH * i;
                if (2 * p < a.R) {
                    const float cs = s_cos[row][p], sn = s_sin[row][p], xa = x.a[i];
                    x.a[i] = fmaf(xa, cs, -x.b[i] * sn);
                    x.b[i] = fmaf(x.b[i], cs, xa * sn);
                }
            }
            to_pieces<VEC>(a, x, lo, hi);
        }
        if (is_q) {
            store_head<TIO, LPH, VEC>(a, (TIO*)a.q_out + ((size_t)(r0 + row) * a.H + h) * a.D, lo, hi, j, at);
        } else if (!APPEND) {
            store_head<TIO, LPH, VEC>(a, (TIO*)a.k_out + ((size_t)(r0 + row) * a.Hk + (h - Hq)) * a.D, lo, hi, j, at);
        } else {
            const int hk = is_v ? h - Hq - Hx : h - Hq;
            const size_t dst = (size_t)(places.dst[row] + (long long)hk * c.page_size);
            if (E4M3) {
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    top = max(top, max(__float_as_uint(lo.v[i]) & 0x7fffffffu, __float_as_uint(hi.v[i]) & 0x7fffffffu));
                const float scale = scale_of(max_of<LPH>(top));
                store_head_e4m3<LPH, VEC>(a, (uint8_t*)(is_v ? c.v_cache : c.k_cache) + dst * a.D, lo, hi, j, at, scale);
                if (j == 0) (is_v ? c.v_scale : c.k_scale)[dst] = scale;
            } else {
                store_head<TIO, LPH, VEC>(a, (TIO*)(is_v ? c.v_cache : c.k_cache) + dst * a.D, lo, hi, j, at);
            }
        }
    }
}

template <typename TIO, int LPH, bool VEC>
void launch_one(const RopeArgs& a, const CacheWriteArgs* c, bool e4m3, int rb, int blocks, int all, hipStream_t stream) {
    if (!c)
        hipLaunchKernelGGL((rope_kernel<TIO, LPH, VEC, false, false>), dim3(all), dim3(256), 0, stream, a, CacheWriteArgs{}, rb, blocks);
    else if (e4m3)
        hipLaunchKernelGGL((rope_kernel<TIO, LPH, VEC, true, true>), dim3(all), dim3(256), 0, stream, a, *c, rb, blocks);
    else
        hipLaunchKernelGGL((rope_kernel<TIO, LPH, VEC, true, false>), dim3(all), dim3(256), 0, stream, a, *c, rb, blocks);
}

template <typename TIO>
hipError_t launch_type(const RopeArgs& a, const CacheWriteArgs* c, bool e4m3, hipStream_t stream) {
    const int rb = rope_rows(a.rows), blocks = (int)rope_blocks(a.rows, 0), all = (int)rope_blocks(a.rows, c && c->status ? c->batch : 0);
    if (all == 0) return hipSuccess;
    // eight elements at a time where heads, strides and pointers allow it
    uintptr_t bits = (uintptr_t)a.q | (uintptr_t)a.k | (uintptr_t)a.v | (uintptr_t)a.q_out | (uintptr_t)a.k_out;
    bits |= (uintptr_t)((a.qs | a.ks | a.vs) * sizeof(TIO)) | (uintptr_t)a.qw | (uintptr_t)a.kw;
    if (c) bits |= (uintptr_t)c->k_cache | (uintptr_t)c->v_cache;
    const bool vec = a.D % 16 == 0 && a.R % 16 == 0 && bits % 16 == 0;
    if (!vec)
        launch_one<TIO, 16, false>(a, c, e4m3, rb, blocks, all, stream);
    else if (a.D <= 64)
        launch_one<TIO, 4, true>(a, c, e4m3, rb, blocks, all, stream);
    else if (a.D <= 128)
        launch_one<TIO, 8, true>(a, c, e4m3, rb, blocks, all, stream);
    else
        launch_one<TIO, 16, true>(a, c, e4m3, rb, blocks, all, stream);
    return hipGetLastError();
}

}  // namespace

int rope_rows(int rows) { return rows <= 1024 ? 1 : rows <= 8192 ? 4 : kRopeRows; }
long long rope_blocks(int rows, int items) { return ((long long)rows + rope_rows(rows) - 1) / rope_rows(rows) + items; }

hipError_t launch_rope(const RopeArgs& a, const CacheWriteArgs* c, bool bf16, bool e4m3, hipStream_t stream) {
    return bf16 ? launch_type<uint16_t>(a, c, e4m3, stream) : launch_type<float>(a, c, e4m3, stream);
}

}  // namespace tsv
