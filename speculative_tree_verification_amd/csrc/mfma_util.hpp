// mfma_util.hpp -- operands of the bf16 matrix products of the prompt scan and
// of the attention.
#pragma once

#include "common.hpp"

namespace tsv {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// Columns of a row-major LDS tile as an operand: the lane with column l % 16 of
// `tile` gets rows 4 (l / 16) + e, e < 4, and the same 16 rows on. (Each 16-lane
// group names 4 rows of 16 columns, 4 columns a lane, and receives them
// transposed.) The 16 columns are 4 pieces of 4, PIECE elements apart.
template <int PIECE = 4>
__device__ __forceinline__ bf16x8 read_columns(const uint16_t* tile, int stride, int lane) {
    const uint16_t* p = tile + lane / 4 * stride + lane % 4 * PIECE;
    typedef s16x4 __attribute__((address_space(3))) lds_s16x4;
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 16 * stride));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// The same of 32 columns: the lane with column l % 32 gets rows 4 (l / 32) + e and
// the same 8 rows on.
__device__ __forceinline__ bf16x8 read_columns32(const uint16_t* tile, int stride, int lane) {
    const uint16_t* p = tile + (lane / 32 * 4 + lane % 16 / 4) * stride + (lane & 16) + lane % 4 * 4;
    typedef s16x4 __attribute__((address_space(3))) lds_s16x4;
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 8 * stride));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Two 4-element pieces of a row, 16 elements apart, in the same order
__device__ __forceinline__ bf16x8 read_row(const uint16_t* p) {
    const s16x4 a = *(const s16x4*)p, b = *(const s16x4*)(p + 16);
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

__device__ __forceinline__ f32x4 mma(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ f32x16 mma(bf16x8 a, bf16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Sign bits of the halves of the result: whether a bf16 of `u` is not finite
// (an exponent of ones carries into the sign)
__device__ __forceinline__ uint32_t nonfinite_bits(uint4 u) {
    return ((u.x & 0x7fff7fffu) + 0x00800080u) | ((u.y & 0x7fff7fffu) + 0x00800080u) |
           ((u.z & 0x7fff7fffu) + 0x00800080u) | ((u.w & 0x7fff7fffu) + 0x00800080u);
}

// 8 bf16 values as an operand, and with 0 in place of those that are not finite
__device__ __forceinline__ bf16x8 as_operand(uint4 u) { return __builtin_bit_cast(bf16x8, u); }
__device__ __forceinline__ uint4 only_finite(uint4 u) {
    uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if ((w[i] & 0x7f80u) == 0x7f80u) w[i] &= 0xffff0000u;
        if ((w[i] & 0x7f800000u) == 0x7f800000u) w[i] &= 0x0000ffffu;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// 8 e4m3 bytes as bf16 (exact)
__device__ __forceinline__ uint4 e4m3_to_bf16(uint2 u) {
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = i < 2 ? u.x : u.y;
        r[i] = i & 1 ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true))
                     : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

}  // namespace tsv
