// prefill_mfma.hip -- the prompt scan's bf16 kernel (head_dim 64, d_state 64 or
// 128): one work-group walks one segment of one head, 64 tokens at a time.
//
// With cum_i the sum of log decays dt A of a chunk up to token i, and S the
// state before the chunk (P x N):
//   Y    = (C B^T o W) X + exp(cum) C S^T + D X,  W_ij = exp(cum_i - cum_j) dt_j  (j <= i)
//   S'   = exp(cum_end) S + sum_j w_j x_j (outer) B_j,  w_j = exp(cum_end - cum_j) dt_j
// cum_end - cum_j is summed from the chunk's end, so that it is exact where it
// is small and the weight counts.
//
// Four waves; wave w owns rows p = 16 w .. 16 w + 15 of the state for the whole
// segment, transposed in its accumulators (N / 16 tiles of 16 n x 16 p). That
// tile is already an operand of the next product (the read-out): a lane holds
// n = 4 (l / 16) + r of column p = l % 16 of each tile, and two tiles make the 8
// consecutive k-slots of a lane if C is read with the same order of n. Products
// per chunk and wave (16x16x32): scores 4 N / 32 on up to 3 of the 10 lower
// tiles, read-out 2 (high and low part of S) x 4 x N / 32, masked product 6,
// update 3 (parts of w x) x 2 x N / 16.
//  - Operands that are needed with tokens as the inner dimension (x for the
//    masked product and the update, B for the update) come from LDS through the
//    transposing read (ds_read_b64_tr_b16).
//  - Outputs are formed transposed (a lane holds 4 consecutive p of a token), so
//    that they leave as 8-byte pieces, and the row factor exp(cum_i) is one
//    value per lane.
//  - Rows are padded by 16 bytes: 16 consecutive rows of a 16-byte column piece
//    fall on all 64 banks.
//  - The next chunk's rows are requested before the products of this one.
#include "seq_common.hpp"

namespace tsv {
namespace {

constexpr int kQ = 64;        // tokens per chunk
constexpr int kP = 64;        // head_dim
constexpr int kXs = kP + 8;   // LDS row strides (elements)
constexpr int kPs = kQ + 8;

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

// Columns of a row-major LDS tile as an operand: of rows k0 .. k0 + 7 and 16
// columns from `col`, the lane with column l % 16 gets its 8 values. (Each
// 16-lane group names 4 rows of 16 columns, 4 columns a lane, and receives them
// transposed.) `row0`: tile + col + stride * k0 of the lane's group.
__device__ __forceinline__ bf16x8 read_columns(const uint16_t* row0, int stride, int lane) {
    const uint16_t* p = row0 + (lane % 16 / 4) * stride + lane % 4 * 4;
    typedef s16x4 __attribute__((address_space(3))) lds_s16x4;
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * stride));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

__device__ __forceinline__ f32x4 mma(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// 8 floats as bf16 and what that leaves (exact)
__device__ __forceinline__ bf16x8 split(float* v) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        u[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        v[2 * i] -= __uint_as_float(u[i] << 16);
        v[2 * i + 1] -= __uint_as_float(u[i] & 0xffff0000u);
    }
    return __builtin_bit_cast(bf16x8, make_uint4(u[0], u[1], u[2], u[3]));
}

__device__ __forceinline__ bool any_nonfinite(uint4 u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    bool r = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) r |= (w[i] & 0x7f80u) == 0x7f80u || (w[i] & 0x7f800000u) == 0x7f800000u;
    return r;
}

template <int NT, bool LOCAL>
__global__ __launch_bounds__(256, LOCAL ? 4 : 3) void prefill_mfma_kernel(PrefillArgs a, SeqPlan plan, SeqWorkspace ws) {
    constexpr int N = NT * 16, KS = N / 32, kNs = N + 8;
    constexpr int BP = kQ * N / 8 / 256;  // 16-byte pieces of B (and C) per thread
    __shared__ int s_red[4];
    __shared__ Segment s_seg;
    __shared__ int s_odd;
    __shared__ __attribute__((aligned(16))) float s_cum[kQ], s_dt[kQ], s_w[kQ];
    __shared__ float s_tot;
    __shared__ __attribute__((aligned(16))) uint16_t s_B[kQ * kNs], s_X[kQ * kXs];
    __shared__ __attribute__((aligned(16))) uint16_t s_C[LOCAL ? 8 : kQ * kNs], s_P[LOCAL ? 8 : kQ * kPs];

    const int tid = threadIdx.x, lane = tid & (kWave - 1), w = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int lid = xcd_block(blockIdx.x, gridDim.x);  // the heads of a segment read the same rows of B and C
    const int h = lid % a.H;
    const Segment sg = find_segment<256>(a.seq_start, a.n_seqs, a.n_tokens, plan.seg, lid / a.H, false, s_red, &s_seg);
    if (!sg.ok || (LOCAL && sg.k == sg.n - 1)) return;
    const int l16 = lane & 15, lg = lane >> 4;
    const int g = h / (a.H / a.G);
    const float Ah = a.A[h], Dh = LOCAL ? 0.f : a.D[h];
    constexpr size_t PN = (size_t)kP * N;
    const int p = 16 * w + l16;

    // state: tile nt, element r of this lane is n = 16 nt + 4 lg + r of row p
    f32x4 st[NT];
    if (LOCAL) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) st[nt] = f32x4{0.f, 0.f, 0.f, 0.f};
    } else {
        const float* from = sg.n == 1 ? a.h + ((size_t)sg.seq * a.H + h) * PN
                                      : ws.state + ((size_t)(sg.base + (sg.k ? sg.k - 1 : sg.n - 1)) * a.H + h) * PN;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) st[nt] = *(const f32x4*)(from + (size_t)p * N + 16 * nt + 4 * lg);
    }
    if (!LOCAL)  // tiles above the diagonal that a 32-token product covers stay zero
        for (int i = tid; i < kQ * kPs / 8; i += 256) ((uint4*)s_P)[i] = make_uint4(0, 0, 0, 0);
    if (tid == 0) s_odd = 0;

    uint4 rB[BP], rC[LOCAL ? 1 : BP], rX[2];
    float rdt = 0.f;
    auto request = [&](int t0) {
        const int cnt = sg.t1 - t0;
#pragma unroll
        for (int i = 0; i < BP; ++i) {
            const int piece = tid + i * 256, row = piece / (N / 8), c = piece % (N / 8) * 8;
            const size_t at = ((size_t)(t0 + row) * a.G + g) * N + c;
            rB[i] = make_uint4(0, 0, 0, 0);
            if (!LOCAL) rC[i] = make_uint4(0, 0, 0, 0);
            if (row < cnt) {
                rB[i] = gload((const uint4*)((const uint16_t*)a.B + at));
                if (!LOCAL) rC[i] = gload((const uint4*)((const uint16_t*)a.C + at));
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int piece = tid + i * 256, row = piece / 8, c = piece % 8 * 8;
            rX[i] = make_uint4(0, 0, 0, 0);
            if (row < cnt) rX[i] = gload((const uint4*)((const uint16_t*)a.x + ((size_t)(t0 + row) * a.H + h) * kP + c));
        }
        if (tid < kQ) rdt = tid < cnt ? Elem<uint16_t>::ld((const uint16_t*)a.dt, (size_t)(t0 + tid) * a.H + h) : 0.f;
    };
    request(sg.t0);
    float sum = 0.f;

    for (int t0 = sg.t0; t0 < sg.t1; t0 += kQ) {
        const int cnt = min(kQ, sg.t1 - t0);
        __syncthreads();  // the last chunk's reads are done
#pragma unroll
        for (int i = 0; i < BP; ++i) {
            const int piece = tid + i * 256, o = piece / (N / 8) * kNs + piece % (N / 8) * 8;
            *(uint4*)&s_B[o] = rB[i];
            if (!LOCAL) *(uint4*)&s_C[o] = rC[i];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int piece = tid + i * 256;
            *(uint4*)&s_X[piece / 8 * kXs + piece % 8 * 8] = rX[i];
            if (!LOCAL && any_nonfinite(rX[i])) s_odd = 1;
        }
        if (w == 0) {
            float up = rdt * Ah;
            up = up < -128.f ? -128.f : up;  // exp is 0 either way, and sums stay exact enough
            float down = up;
            const float own = up;
#pragma unroll
            for (int o = 1; o < kWave; o <<= 1) {
                const float u = __shfl_up(up, o, kWave), d = __shfl_down(down, o, kWave);
                if (lane >= o) up += u;
                if (lane + o < kWave) down += d;
            }
            const float after = __shfl_down(down, 1, kWave);  // sum of the later tokens
            s_cum[lane] = up;
            s_dt[lane] = rdt;
            s_w[lane] = __expf(lane == kWave - 1 ? 0.f : after) * rdt;
            if (lane == 0) s_tot = down;
        }
        __syncthreads();
        if (t0 + kQ < sg.t1) request(t0 + kQ);
        const float tot = s_tot;
        f32x4 y[4];
        bool odd = false;
        if (!LOCAL) {
            odd = s_odd;
            // scores of the lower tiles, weighted, as P[i][j]: wave 0 has (3,0) (3,1) (0,0),
            // wave 1 (3,2) (3,3) (1,0), wave 2 (2,0) (2,1), wave 3 (2,2) (1,1)
#pragma unroll
            for (int u = 0; u < 3; ++u) {
                if (u == 2 && w >= 2) break;
                const int it = w < 2 ? (u == 2 ? w : 3) : (w == 3 && u == 1 ? 1 : 2);
                const int jt = w == 0 ? (u == 1) : w == 1 ? (u == 2 ? 0 : 2 + u) : w == 2 ? u : (u == 0 ? 2 : 1);
                f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < KS; ++k)
                    s = mma(*(const bf16x8*)&s_B[(16 * jt + l16) * kNs + 32 * k + 8 * lg],
                            *(const bf16x8*)&s_C[(16 * it + l16) * kNs + 32 * k + 8 * lg], s);
                const int i = 16 * it + l16, j = 16 * jt + 4 * lg;
                const float ci = s_cum[i];
                const f32x4 cj = *(const f32x4*)&s_cum[j], dj = *(const f32x4*)&s_dt[j];
                float v[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) v[r] = j + r <= i ? s[r] * (__expf(ci - cj[r]) * dj[r]) : 0.f;
                *(uint2*)&s_P[i * kPs + j] = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
            }
            // read-out of the state before the chunk
#pragma unroll
            for (int it = 0; it < 4; ++it) y[it] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                float v[8];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    v[r] = st[2 * k][r];
                    v[4 + r] = st[2 * k + 1][r];
                }
                const bf16x8 hi = split(v);
                const bf16x8 lo = split(v);
#pragma unroll
                for (int it = 0; it < 4; ++it) {
                    const uint16_t* c = &s_C[(16 * it + l16) * kNs + 32 * k + 4 * lg];
                    const s16x4 c0 = *(const s16x4*)c, c1 = *(const s16x4*)(c + 16);
                    const bf16x8 cf = __builtin_bit_cast(bf16x8, __builtin_shufflevector(c0, c1, 0, 1, 2, 3, 4, 5, 6, 7));
                    y[it] = mma(hi, cf, y[it]);
                    y[it] = mma(lo, cf, y[it]);
                }
            }
#pragma unroll
            for (int it = 0; it < 4; ++it) y[it] *= __expf(s_cum[16 * it + l16]);
        }
        bf16x8 xf[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) xf[k] = read_columns(&s_X[(32 * k + 8 * lg) * kXs + 16 * w], kXs, lane);
        // update: S' = exp(tot) S + B^T (w x)
        const float keep = __expf(tot);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) st[nt] *= keep;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float v[8];
            const f32x4 w0 = *(const f32x4*)&s_w[32 * k + 8 * lg], w1 = *(const f32x4*)&s_w[32 * k + 8 * lg + 4];
            const s16x8 xs = __builtin_bit_cast(s16x8, xf[k]);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = bf16_bits_to_f32((uint16_t)xs[e]) * (e < 4 ? w0[e] : w1[e - 4]);
            const bf16x8 v0 = split(v);
            const bf16x8 v1 = split(v);
            const bf16x8 v2 = split(v);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const bf16x8 bf = read_columns(&s_B[(32 * k + 8 * lg) * kNs + 16 * nt], kNs, lane);
                st[nt] = mma(bf, v0, st[nt]);
                st[nt] = mma(bf, v1, st[nt]);
                st[nt] = mma(bf, v2, st[nt]);
            }
        }
        if (LOCAL) {
            sum += tot;
            continue;
        }
        __syncthreads();  // P is whole
        if (tid == 0) s_odd = 0;
        if (odd) {
            // an x that is not finite must not reach earlier tokens through a
            // weight of 0: it leaves the matrix product and is added alone
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                s16x8 xs = __builtin_bit_cast(s16x8, xf[k]);
#pragma unroll
                for (int e = 0; e < 8; ++e) xs[e] = (xs[e] & 0x7f80) == 0x7f80 ? (short)0 : xs[e];
                xf[k] = __builtin_bit_cast(bf16x8, xs);
            }
        }
#pragma unroll
        for (int it = 0; it < 4; ++it)
#pragma unroll
            for (int k = 0; k <= it / 2; ++k)
                y[it] = mma(xf[k], *(const bf16x8*)&s_P[(16 * it + l16) * kPs + 32 * k + 8 * lg], y[it]);
        if (odd) {
            for (int j = 0; j < kQ; ++j) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const uint16_t xb = s_X[j * kXs + 16 * w + 4 * lg + r];
                    if ((xb & 0x7f80) != 0x7f80) continue;
#pragma unroll
                    for (int it = 0; it < 4; ++it) {
                        const int i = 16 * it + l16;
                        if (i >= j) y[it][r] += bf16_bits_to_f32(s_P[i * kPs + j]) * bf16_bits_to_f32(xb);
                    }
                }
            }
        }
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            const int i = 16 * it + l16, q = 16 * w + 4 * lg;
            const uint2 xr = *(const uint2*)&s_X[i * kXs + q];
            const float o0 = fmaf(Dh, __uint_as_float(xr.x << 16), y[it][0]);
            const float o1 = fmaf(Dh, __uint_as_float(xr.x & 0xffff0000u), y[it][1]);
            const float o2 = fmaf(Dh, __uint_as_float(xr.y << 16), y[it][2]);
            const float o3 = fmaf(Dh, __uint_as_float(xr.y & 0xffff0000u), y[it][3]);
            if (i < cnt)
                gstore((uint2*)((uint16_t*)a.y + ((size_t)(t0 + i) * a.H + h) * kP + q),
                       make_uint2(pack_bf16x2(o0, o1), pack_bf16x2(o2, o3)));
        }
    }
    if (!LOCAL && sg.k != sg.n - 1) return;
    float* to = (LOCAL ? ws.state + ((size_t)(sg.base + sg.k) * a.H + h) * PN : a.h + ((size_t)sg.seq * a.H + h) * PN) + (size_t)p * N;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) *(f32x4*)(to + 16 * nt + 4 * lg) = st[nt];
    if (LOCAL && tid == 0) ws.sum[(size_t)(sg.base + sg.k) * a.H + h] = sum;
}

template <bool LOCAL>
void launch_pass(const PrefillArgs& a, const SeqPlan& p, const SeqWorkspace& ws, hipStream_t stream) {
    const dim3 grid((unsigned)((long long)p.slots * a.H));
    if (a.N == 64)
        hipLaunchKernelGGL((prefill_mfma_kernel<4, LOCAL>), grid, dim3(256), 0, stream, a, p, ws);
    else
        hipLaunchKernelGGL((prefill_mfma_kernel<8, LOCAL>), grid, dim3(256), 0, stream, a, p, ws);
}

}  // namespace

bool prefill_mfma_supported(const PrefillArgs& a) {
    const uintptr_t all = (uintptr_t)a.x | (uintptr_t)a.B | (uintptr_t)a.C | (uintptr_t)a.y | (uintptr_t)a.h;
    return a.P == kP && (a.N == 64 || a.N == 128) && all % 16 == 0;
}

void launch_prefill_mfma(const PrefillArgs& a, const SeqPlan& p, const SeqWorkspace& ws, bool local, hipStream_t stream) {
    if (local)
        launch_pass<true>(a, p, ws, stream);
    else
        launch_pass<false>(a, p, ws, stream);
}

}  // namespace tsv
