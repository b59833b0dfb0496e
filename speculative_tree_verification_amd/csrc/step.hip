// step.hip -- one token of each item through an SSD layer: the state advanced
// in place and read out in the same pass.
//
//   h[p][n] <- exp(dt A) h[p][n] + dt x[p] B[n],   y[p] = sum_n h[p][n] C[n] + D x[p]
//
// Bound by the state's traffic: P N floats read and written per item and head
// (64 KB at P = 64, N = 128) for 5 P N operations. A row of the state is spread
// over N / 4 lanes as one 16-byte piece each, so that a wave reads whole
// kilobytes; every thread has its four pieces requested before the first is
// used, and the state streams past the caches (nontemporal), which it would
// only sweep. The sum over n is a butterfly over the row's lanes. 64 items of 80
// heads, N = 128 (337 MB): 59 us, 5.7 TB/s.
#include "common.hpp"
#include "seq_launch.hpp"

namespace tsv {
namespace {

constexpr int kStepRows = 4;  // state rows of each lane

// LPR lanes hold a row of N <= 4 * LPR; VEC: N % 4 == 0 and 16-byte aligned state, 4 elements' alignment of B, C
template <typename TIO, int LPR, bool VEC>
__global__ __launch_bounds__(256) void step_kernel(StepArgs a, int slices) {
    constexpr int RPI = kWave / LPR;           // rows a wave touches at once
    constexpr int RPW = RPI * kStepRows;       // rows of a wave
    constexpr int RPB = RPW * (256 / kWave);   // rows of a block
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int slice = blockIdx.x % slices;
    const int bh = blockIdx.x / slices, b = bh / a.H, h = bh % a.H;
    const int n = (lane % LPR) * 4, rem = a.N - n;
    const int p0 = slice * RPB + wave * RPW + lane / LPR;
    const TIO* x = (const TIO*)a.x + (size_t)bh * a.P;
    const size_t bc = ((size_t)b * a.G + h / (a.H / a.G)) * a.N + n;
    float* hp = a.h + (size_t)bh * a.P * a.N + n;

    float4 s[kStepRows];
#pragma unroll
    for (int r = 0; r < kStepRows; ++r) {
        const int p = p0 + r * RPI;
        if (p < a.P && rem > 0) {
            if (VEC)
                s[r] = gload_nt((const float4*)(hp + (size_t)p * a.N));
            else
                s[r] = ld4<false>(hp + (size_t)p * a.N, rem);
        } else {
            s[r] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    float4 Bv = make_float4(0.f, 0.f, 0.f, 0.f), Cv = Bv;
    if (rem > 0) {
        Bv = ld4io<TIO, VEC>((const TIO*)a.B + bc, rem);
        Cv = ld4io<TIO, VEC>((const TIO*)a.C + bc, rem);
    }
    const float dt = Elem<TIO>::ld((const TIO*)a.dt, bh);
    const float decay = expf(dt * a.A[h]), Dh = a.D[h];
#pragma unroll
    for (int r = 0; r < kStepRows; ++r) {
        const int p = p0 + r * RPI;
        if (p >= a.P) continue;  // the same for all lanes of a row
        const float xv = Elem<TIO>::ld(x, p), wx = dt * xv;
        float4 v = s[r];
        v.x = fmaf(decay, v.x, wx * Bv.x);
        v.y = fmaf(decay, v.y, wx * Bv.y);
        v.z = fmaf(decay, v.z, wx * Bv.z);
        v.w = fmaf(decay, v.w, wx * Bv.w);
        if (rem > 0) {
            float* o = hp + (size_t)p * a.N;
            if (VEC) {
                gstore_nt((float4*)o, v);
            } else {
                o[0] = v.x;
                if (rem > 1) o[1] = v.y;
                if (rem > 2) o[2] = v.z;
                if (rem > 3) o[3] = v.w;
            }
        }
        // lanes past N hold zeros of B, C and the state: their term is 0 even where the decay is not finite
        float y = rem > 0 ? v.x * Cv.x : 0.f;
        if (rem > 1) y = fmaf(v.y, Cv.y, y);
        if (rem > 2) y = fmaf(v.z, Cv.z, y);
        if (rem > 3) y = fmaf(v.w, Cv.w, y);
#pragma unroll
        for (int m = 1; m < LPR; m <<= 1) y += __shfl_xor(y, m, kWave);
        if (lane % LPR == 0) Elem<TIO>::st((TIO*)a.y, (size_t)bh * a.P + p, fmaf(Dh, xv, y));
    }
}

// lanes of a state row of N elements; work-groups of a state of P rows
constexpr int row_lanes(int N) { return N <= 64 ? 16 : N <= 128 ? 32 : 64; }
constexpr int row_slices(int P, int lanes) { return (P + kWave / lanes * kStepRows * 4 - 1) / (kWave / lanes * kStepRows * 4); }

template <typename TIO, int LPR>
hipError_t launch_lpr(const StepArgs& a, bool vec, hipStream_t stream) {
    const int slices = row_slices(a.P, LPR);
    const dim3 grid((unsigned)((long long)a.batch * a.H * slices));
    if (vec)
        hipLaunchKernelGGL((step_kernel<TIO, LPR, true>), grid, dim3(256), 0, stream, a, slices);
    else
        hipLaunchKernelGGL((step_kernel<TIO, LPR, false>), grid, dim3(256), 0, stream, a, slices);
    return hipGetLastError();
}

template <typename TIO>
hipError_t launch_io(const StepArgs& a, hipStream_t stream) {
    const bool vec = a.N % 4 == 0 && (uintptr_t)a.h % 16 == 0 && (uintptr_t)a.B % (4 * sizeof(TIO)) == 0 &&
                     (uintptr_t)a.C % (4 * sizeof(TIO)) == 0;
    if (row_lanes(a.N) == 16) return launch_lpr<TIO, 16>(a, vec, stream);
    if (row_lanes(a.N) == 32) return launch_lpr<TIO, 32>(a, vec, stream);
    return launch_lpr<TIO, 64>(a, vec, stream);
}

}  // namespace

long long step_blocks(const tsv_shape* s) {
    return (long long)s->batch * s->n_heads * row_slices(s->head_dim, row_lanes(s->d_state));
}

hipError_t launch_step(const StepArgs& a, bool bf16, hipStream_t stream) {
    return bf16 ? launch_io<uint16_t>(a, stream) : launch_io<float>(a, stream);
}

}  // namespace tsv
