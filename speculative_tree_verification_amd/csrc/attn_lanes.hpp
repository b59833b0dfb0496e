// attn_lanes.hpp -- what the matrix kernels of the attention share: a row's
// statistics over lanes, the scores' factor, the cache's rows.
#pragma once

#include "attn_common.hpp"

namespace tsv {

constexpr int kTileKeys = 64;  // keys of a tile that a work-group shares in LDS
constexpr float kSlack = 8.f;  // a maximum moves when a weight would pass 2^kSlack

// max of three, one instruction (v_maximum3_f32). A NaN among them stays, where
// fmaxf would first make each product's result quiet; a row whose maximum is a NaN
// has a key with a NaN score and is NaN whatever its maximum. An instruction of the
// compiler's and not assembly: only for its own does it count the cycles that a
// matrix product's result needs before it may be read.
__device__ __forceinline__ float max3(float a, float b, float c) {
    return __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, b), c);
}
// Largest of / sum over the four lanes (16 apart) that hold a row's keys: halves
// and rows of 16 lanes change places with a copy of themselves
struct Two {
    float a, b;
};
__device__ __forceinline__ Two swap32(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return {__uint_as_float(r[0]), __uint_as_float(r[1])};
}
__device__ __forceinline__ Two swap16(float v) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return {__uint_as_float(r[0]), __uint_as_float(r[1])};
}
template <int RW = 16>
__device__ __forceinline__ float row_max(float v) {
    const Two h = swap32(v);
    if (RW == 32) return fmaxf(h.a, h.b);
    const Two q = swap16(fmaxf(h.a, h.b));
    return fmaxf(q.a, q.b);
}
template <int RW = 16>
__device__ __forceinline__ float row_sum(float v) {
    const Two h = swap32(v);
    if (RW == 32) return h.a + h.b;
    const Two q = swap16(h.a + h.b);
    return q.a + q.b;
}

// Whether `page`, what the table holds, is a page of the pool; and the row index of
// position `pos`, which lies on it, in the cache's arrays (of another page, or of
// none: take page 0, whose rows exist, and the item's status bit).
__device__ __forceinline__ bool page_ok(const AttnArgs& a, int page) { return (uint32_t)page < (uint32_t)a.n_pages; }
__device__ __forceinline__ uint32_t cache_row(const AttnArgs& a, int page, int hk, int pos) {
    const int off = pos - page_of(pos, a.div) * a.page_size;
    return ((uint32_t)page * a.Hk + hk) * a.page_size + off;
}

// Scores stay as the product gives them, and their factor enters the exponent's
// multiply-add: it has to be positive, so a negative one turns q's signs (exact),
// and 0 becomes the smallest normal number (a masked score of -inf stays one).
__device__ __forceinline__ float score_factor(const AttnArgs& a) { return fmaxf(fabsf(a.scale_log2), 1.17549435e-38f); }
}  // namespace tsv
