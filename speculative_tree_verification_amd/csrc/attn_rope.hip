// attn_rope.hip -- norms of the heads of queries and keys with the position rotation,
// in one pass: of rows of any kind (tree_attn_rope), or on the way of packed rows into
// the paged cache (tree_attn_append_rope).
//
//   z = w x / sqrt(mean x^2 + eps)   (without a weight: z = x)
//   (z_a, z_b) -> (z_a cos t - z_b sin t, z_b cos t + z_a sin t),  t = position inv_freq[i],
// for the R / 2 pairs (a, b) = (i, i + R/2), or (2 i, 2 i + 1), of a head; the other
// elements stay z.
//
// Bound by the rows' traffic, and in 8 bits by the vector unit beside it: 32 trees of 63 nodes,
// 32 query and 8 key heads of 128 in bf16, 41 MB, 10 us in the kernel (11.5 a call, the host's
// time); 16 prompts of 1 to 2047 tokens into an e4m3 cache, 370 MB, 80 us (4.6 TB/s; a large
// copy reaches 5.1); one token 3.8 us.
//
// A lane has eight pairs of a head, so that both elements of a pair are its own and only the
// sum of squares leaves it: a head of D has D / 16 lanes (rounded up to a power of two), two
// 16-byte pieces each in bf16, with the next head's on their way (two heads ahead gained
// nothing). The angles of a row are the same for all of its heads: the work-group forms them
// once, in LDS. An angle is a product in 64 bits, in revolutions, of which the whole ones are
// dropped before it is rounded to 32: at position 10^6 a product in 32 bits would be off by
// 0.06. That rounding is 2^-26 of a turn at most, 1e-7 of an output, as much as the sine's and
// cosine's own; a second float for it would be two products more a pair and row.
#include "attn_cache.hpp"

namespace tsv {
namespace {

constexpr int kRopeRows = 4;  // most rows of a work-group

// How a lane has its eight pairs:
//   kHalves       pairs 8 j + i of (i, i + R / 2), as two pieces of eight neighbours; past the
//                 rotated elements sixteen neighbours, as two pieces
//   kInterleaved  pairs 8 j + i of (2 i, 2 i + 1), sixteen neighbours
//   kAny          pairs j + LPH i of either kind, element by element
enum Pairing { kHalves, kInterleaved, kAny };

// Element numbers of pair p
__device__ __forceinline__ int2 pair_of(const RopeArgs& a, int p) {
    const int half = a.R / 2;
    return p < half && !a.interleaved ? make_int2(p, p + half) : make_int2(2 * p, 2 * p + 1);
}

// A lane's sixteen elements: its two pieces, or (kAny) its pairs' first and second ones
template <typename TIO, bool VEC>
struct Piece {
    Raw<TIO, VEC> lo, hi;
};
struct Lane16 {
    float lo[8], hi[8];
};

template <typename TIO, int LPH, Pairing P>
__device__ __forceinline__ Piece<TIO, P != kAny> load_head(const RopeArgs& a, const TIO* row, int j, int2 at) {
    Piece<TIO, P != kAny> p{};
    if constexpr (P != kAny) {
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
__device__ __forceinline__ void store_piece(TIO* to, const float (&v)[8]) {
    if constexpr (sizeof(TIO) == 2) {
        gstore((uint4*)to, make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
    } else {
        gstore((float4*)to, make_float4(v[0], v[1], v[2], v[3]));
        gstore((float4*)to + 1, make_float4(v[4], v[5], v[6], v[7]));
    }
}
template <typename TIO, int LPH, Pairing P>
__device__ __forceinline__ void store_head(const RopeArgs& a, TIO* row, const Lane16& x, int j, int2 to) {
    if constexpr (P != kAny) {
        if (16 * j >= a.D) return;
        store_piece<TIO>(row + to.x, x.lo);
        store_piece<TIO>(row + to.y, x.hi);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int2 e = pair_of(a, j + LPH * i);
            if (e.x < a.D) Elem<TIO>::st(row, e.x, x.lo[i]);
            if (e.y < a.D) Elem<TIO>::st(row, e.y, x.hi[i]);
        }
    }
}
// The row of a head in 8 bits, and its scale
template <int LPH, Pairing P>
__device__ __forceinline__ void store_head_e4m3(const RopeArgs& a, uint8_t* row, float* scale_to, const Lane16& x, int j, int2 to) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, max(__float_as_uint(x.lo[i]) & 0x7fffffffu, __float_as_uint(x.hi[i]) & 0x7fffffffu));
    const float scale = scale_of(max_of<LPH>(top));
    const bool finite = scale == scale;
    Quad q;
#pragma unroll
    for (int i = 0; i < 8; ++i) q.v[i] = x.lo[i];
    const uint2 ul = e4m3_bytes(q, scale, finite);
#pragma unroll
    for (int i = 0; i < 8; ++i) q.v[i] = x.hi[i];
    const uint2 uh = e4m3_bytes(q, scale, finite);
    if constexpr (P != kAny) {
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
    if (j == 0) *scale_to = scale;
}

template <typename TIO, bool VEC>
__device__ __forceinline__ Lane16 to_floats(const Piece<TIO, VEC>& p) {
    Lane16 x;
    const Quad lo = floats<TIO, VEC>(p.lo), hi = floats<TIO, VEC>(p.hi);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x.lo[i] = lo.v[i];
        x.hi[i] = hi.v[i];
    }
    return x;
}

// (z_a, z_b) turned
__device__ __forceinline__ void turn(float& za, float& zb, float cs, float sn) {
    const float x = za;
    za = fmaf(x, cs, -zb * sn);
    zb = fmaf(zb, cs, x * sn);
}

// Heads of a row: H of q and Hk of k, which are normed and turned, and where they go into the
// cache Hk of v. `rb` rows a work-group.
template <typename TIO, int LPH, Pairing P, bool APPEND, bool E4M3>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a, CacheWriteArgs c, int rb, int row_blocks) {
    __shared__ __attribute__((aligned(16))) float s_cos[kRopeRows][128], s_sin[kRopeRows][128], s_w[2][256];
    __shared__ RowPlaces<kRopeRows> places;
    constexpr bool VEC = P != kAny;
    constexpr int kSlots = 256 / LPH;
    const int tid = threadIdx.x, j = tid % LPH;
    // first elements of the lane's two pieces
    const bool turned = 16 * j < a.R;
    const int2 at = P == kHalves && turned ? make_int2(8 * j, a.R / 2 + 8 * j) : make_int2(16 * j, 16 * j + 8);
    const bool rows = (int)blockIdx.x < row_blocks;
    const int r0 = blockIdx.x * rb, n = rows ? min(rb, a.rows - r0) : 0;
    const int Hq = a.q ? a.H : 0, Hx = a.k ? a.Hk : 0, heads = Hq + Hx, units = n * heads;
    typedef Piece<TIO, VEC> Raw16;
    auto fetch = [&](int u) {
        if (u >= units) return Raw16{};
        const int row = page_of(u, a.heads), h = u - row * heads;
        const size_t r = (size_t)(r0 + row);
        return load_head<TIO, LPH, P>(a, h < Hq ? (const TIO*)a.q + r * a.qs + (size_t)h * a.D : (const TIO*)a.k + r * a.ks + (size_t)(h - Hq) * a.D, j, at);
    };
    auto fetch_v = [&](int u) {
        if (u >= n * Hx) return Raw16{};
        const int row = page_of(u, a.key_heads), h = u - row * Hx;
        return load_head<TIO, LPH, P>(a, (const TIO*)a.v + (size_t)(r0 + row) * a.vs + (size_t)h * a.D, j, at);
    };
    // the first rows are on their way while their places and angles are found
    int u = tid / LPH;
    Raw16 next = fetch(u);
    s_w[0][tid] = a.qw && tid < a.D ? a.qw[tid] : 1.f;
    s_w[1][tid] = a.kw && tid < a.D ? a.kw[tid] : 1.f;
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
        const Raw16 now = next;
        next = fetch(u + kSlots);
        const int row = page_of(u, a.heads), h = u - row * heads;
        if (places.place[row] < 0) continue;  // a row of no sequence, or left out by its position (the same for a head's lanes)
        const bool is_q = h < Hq;
        const float* wt = s_w[!is_q];
        Lane16 x = to_floats<TIO, VEC>(now);
        float by = 1.f;
        if (is_q ? a.qw != nullptr : a.kw != nullptr) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fmaf(x.lo[i], x.lo[i], fmaf(x.hi[i], x.hi[i], sum));
            by = 1.f / sqrtf(head_sum<LPH>(sum) / (float)a.D + a.eps);
        }
        // (the weights are 1 where there is no norm; a lane past the head's end has zeros)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int2 e = VEC ? make_int2(at.x + i, at.y + i) : pair_of(a, j + LPH * i);
            x.lo[i] *= by * wt[e.x];
            x.hi[i] *= by * wt[e.y];
        }
        if (!VEC) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int p = j + LPH * i;
                if (2 * p < a.R) turn(x.lo[i], x.hi[i], s_cos[row][p], s_sin[row][p]);
            }
        } else if (turned) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float cs = s_cos[row][8 * j + i], sn = s_sin[row][8 * j + i];
                if (P == kHalves)
                    turn(x.lo[i], x.hi[i], cs, sn);
                else if (i < 4)
                    turn(x.lo[2 * i], x.lo[2 * i + 1], cs, sn);
                else
                    turn(x.hi[2 * i - 8], x.hi[2 * i - 7], cs, sn);
            }
        }
        if (is_q) {
            store_head<TIO, LPH, P>(a, (TIO*)a.q_out + ((size_t)(r0 + row) * a.H + h) * a.D, x, j, at);
        } else if (!APPEND) {
            store_head<TIO, LPH, P>(a, (TIO*)a.k_out + ((size_t)(r0 + row) * a.Hk + (h - Hq)) * a.D, x, j, at);
        } else {
            const size_t dst = (size_t)(places.dst[row] + (long long)(h - Hq) * c.page_size);
            if constexpr (E4M3)
                store_head_e4m3<LPH, P>(a, (uint8_t*)c.k_cache + dst * a.D, c.k_scale + dst, x, j, at);
            else
                store_head<TIO, LPH, P>(a, (TIO*)c.k_cache + dst * a.D, x, j, at);
        }
    }
    if (!APPEND) return;
    u = tid / LPH;
    next = fetch_v(u);
    for (; u < n * Hx; u += kSlots) {
        const Raw16 now = next;
        next = fetch_v(u + kSlots);
        const int row = page_of(u, a.key_heads), h = u - row * Hx;
        if (places.place[row] < 0) continue;
        const size_t dst = (size_t)(places.dst[row] + (long long)h * c.page_size);
        const Lane16 x = to_floats<TIO, VEC>(now);
        if constexpr (E4M3)
            store_head_e4m3<LPH, P>(a, (uint8_t*)c.v_cache + dst * a.D, c.v_scale + dst, x, j, at);
        else
            store_head<TIO, LPH, P>(a, (TIO*)c.v_cache + dst * a.D, x, j, at);
    }
}

// One row each while there are few, so that all compute units have one; of many, the weights' way
// into LDS and the search for the rows' sequences are paid by four (one row a work-group and four,
// in the kernel: 64 rows into the cache 6.4 and 9.6 us, 1024 rows 9.4 and 11.3, 2048 rows 14.9 and
// 13.8, 16000 rows 106 and 85; without a cache 992 rows 6.7 and 8.8, 2016 rows 9.7 and 10.9, 8160
// rows 29.2 and 27.7)
int rope_rows(int rows, bool append) { return rows <= (append ? 1024 : 2048) ? 1 : kRopeRows; }

template <typename TIO, int LPH, Pairing P>
void launch_one(const RopeArgs& a, const CacheWriteArgs* c, bool e4m3, int rb, int blocks, int all, hipStream_t stream) {
    if (!c)
        hipLaunchKernelGGL((rope_kernel<TIO, LPH, P, false, false>), dim3(all), dim3(256), 0, stream, a, CacheWriteArgs{}, rb, blocks);
    else if (e4m3)
        hipLaunchKernelGGL((rope_kernel<TIO, LPH, P, true, true>), dim3(all), dim3(256), 0, stream, a, *c, rb, blocks);
    else
        hipLaunchKernelGGL((rope_kernel<TIO, LPH, P, true, false>), dim3(all), dim3(256), 0, stream, a, *c, rb, blocks);
}

template <typename TIO, Pairing P>
void launch_pairing(const RopeArgs& a, const CacheWriteArgs* c, bool e4m3, int rb, int blocks, int all, hipStream_t stream) {
    if (a.D <= 64)
        launch_one<TIO, 4, P>(a, c, e4m3, rb, blocks, all, stream);
    else if (a.D <= 128)
        launch_one<TIO, 8, P>(a, c, e4m3, rb, blocks, all, stream);
    else
        launch_one<TIO, 16, P>(a, c, e4m3, rb, blocks, all, stream);
}

template <typename TIO>
hipError_t launch_type(const RopeArgs& a, const CacheWriteArgs* c, bool e4m3, hipStream_t stream) {
    const int rb = rope_rows(a.rows, c != nullptr), blocks = (int)rope_blocks(a.rows, c != nullptr, 0);
    const int all = blocks + (c && c->status ? c->batch : 0);
    if (all == 0) return hipSuccess;
    // eight elements at a time where heads, strides and pointers allow it
    uintptr_t bits = (uintptr_t)a.q | (uintptr_t)a.k | (uintptr_t)a.v | (uintptr_t)a.q_out | (uintptr_t)a.k_out;
    bits |= (uintptr_t)((a.qs | a.ks | a.vs) * sizeof(TIO));
    if (c) bits |= (uintptr_t)c->k_cache | (uintptr_t)c->v_cache;
    const bool vec = a.D % 16 == 0 && a.R % 16 == 0 && bits % 16 == 0;
    if (!vec)
        launch_one<TIO, 16, kAny>(a, c, e4m3, rb, blocks, all, stream);
    else if (a.interleaved)
        launch_pairing<TIO, kInterleaved>(a, c, e4m3, rb, blocks, all, stream);
    else
        launch_pairing<TIO, kHalves>(a, c, e4m3, rb, blocks, all, stream);
    return hipGetLastError();
}

}  // namespace

long long rope_blocks(int rows, bool append, int items) { return ((long long)rows + rope_rows(rows, append) - 1) / rope_rows(rows, append) + items; }

hipError_t launch_rope(const RopeArgs& a, const CacheWriteArgs* c, bool bf16, bool e4m3, hipStream_t stream) {
    return bf16 ? launch_type<uint16_t>(a, c, e4m3, stream) : launch_type<float>(a, c, e4m3, stream);
}

}  // namespace tsv
