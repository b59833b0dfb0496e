// prefill_mfma.hip -- the prompt scan's bf16 kernel (head_dim 64, d_state 64 or
// 128): one work-group walks one segment of one head or of two heads of a
// group, 64 tokens at a time.
//
// With cum_i the sum of log decays dt A of a chunk up to token i, and S the
// state before the chunk (P x N):
//   Y    = (C B^T o W) X + exp(cum) C S^T + D X,  W_ij = exp(cum_i - cum_j) dt_j  (j <= i)
//   S'   = exp(cum_end) S + sum_j w_j x_j (outer) B_j,  w_j = exp(cum_end - cum_j) dt_j
// cum_end - cum_j is summed from the chunk's end, so that it is exact where it
// is small and the weight counts.
//
// Four waves share HW heads; a wave owns 16 HW rows p of one head's state for
// the whole segment, transposed in its accumulators (tiles of 16 n x 16 p). Such
// a tile is already an operand of the next product (the read-out): a lane holds
// n = 4 (l / 16) + r of column p = l % 16, and two tiles make the 8 k-slots of a
// lane if C is read with the same order of n. Two heads at once read B and C
// from LDS, and form the scores, once for both.
//
// What bounds it: the matrix work (184 products of 16 cycles a chunk and wave at
// N = 128) and the vector work (about 830 operations: splitting, decays,
// weights) of the two waves of a SIMD, which hardly overlap on this GPU (a wave
// of products and a wave of multiply-adds side by side take three quarters of
// the sum of their times): 14,000 cycles a chunk, 58 us for the scan of 4096
// tokens, 80 heads. With two heads and N = 128 all 256 registers are taken and 13
// values go to scratch, five words out and seven back a chunk. Tried and not kept: four waves a SIMD with half the rows
// (spills at 128 registers, 79 us); vector work laid between the products by
// hand (62 us); residuals by dot products instead of subtractions (60 us); one
// head (104 us, LDS bound).
//  - Operands that are needed with tokens as the inner dimension (x for the
//    masked product and the update, B for the update) come from LDS through the
//    transposing read (ds_read_b64_tr_b16); 16 lanes read 4 rows, so rows are
//    padded to 8 banks apart and a wave's reads take 16 consecutive rows. The
//    token order of these products is therefore 4 (l / 16) + e and 16 more.
//  - Outputs are formed transposed (a lane holds 4 consecutive p of a token), so
//    that the row factor exp(cum_i) is one value per lane, and with two p-tiles
//    taken from alternating pieces of 4 rows they leave as 16-byte pieces.
//  - S is read out as two bf16 parts (what is left is at most 2^-18 of an
//    element, below the rounding of y), w x enters the update as three, so that
//    the state keeps its 24 bits. W o C B^T is rounded once, as y is (y is off by
//    0.0020 to 0.0021 of its size on average, by 0.0017 from its own rounding): a
//    second part would be as many products again as the masked one has.
//  - The next chunk's rows are requested between the products of this one, a
//    third at a time: a compute unit takes about 32 bytes a cycle from its L2,
//    and a wave waits where it asks for more at once.
#include "mfma_util.hpp"
#include "seq_common.hpp"

namespace tsv {
namespace {

constexpr int kQ = 64;        // tokens per chunk
constexpr int kP = 64;        // head_dim
constexpr int kXs = kP + 16;  // LDS row strides (elements)
constexpr int kPs = kQ + 8;

// 8 floats as NP bf16 parts, each the rounding of what the ones before leave (exact)
template <int NP>
struct Parts {
    bf16x8 part[NP];
};
template <int NP>
__device__ __forceinline__ Parts<NP> split(const float* v) {
    uint32_t u[NP][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a = v[2 * i], b = v[2 * i + 1];
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            u[n][i] = pack_bf16x2(a, b);
            a -= __uint_as_float(u[n][i] << 16);
            b -= __uint_as_float(u[n][i] & 0xffff0000u);
        }
    }
    Parts<NP> p;
#pragma unroll
    for (int n = 0; n < NP; ++n) p.part[n] = __builtin_bit_cast(bf16x8, make_uint4(u[n][0], u[n][1], u[n][2], u[n][3]));
    return p;
}

// inclusive sum over the wave's lanes 0 .. lane (row shifts, then the last lane
// of each row of 16 to the rows behind it)
__device__ __forceinline__ float prefix_sum(float v) {
#define TSV_DPP_ADD(ctrl, rows) \
    v += __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), ctrl, rows, 0xf, false))
    TSV_DPP_ADD(0x111, 0xf);  // row_shr:1
    TSV_DPP_ADD(0x112, 0xf);
    TSV_DPP_ADD(0x114, 0xf);
    TSV_DPP_ADD(0x118, 0xf);
    TSV_DPP_ADD(0x142, 0xa);  // row_bcast:15 into rows 1 and 3
    TSV_DPP_ADD(0x143, 0xc);  // row_bcast:31 into rows 2 and 3
#undef TSV_DPP_ADD
    return v;
}

template <int NT, int HW, bool LOCAL>
__global__ __launch_bounds__(256, 2) void prefill_mfma_kernel(PrefillArgs a, SeqPlan plan, SeqWorkspace ws) {
    constexpr int N = NT * 16, KS = N / 32, kBs = N + 16, kCs = N + 8;
    constexpr int TH = 256;               // threads
    constexpr int PT = HW;                // 16-row tiles of p per wave
    constexpr int BP = kQ * N / 8 / TH;   // 16-byte pieces of B (and C) per thread
    constexpr int XP = 2 * HW;            // of x
    __shared__ int s_red[TH / kWave];
    __shared__ Segment s_seg;
    __shared__ int s_odd, s_len[kSortMax];
    // per chunk (two sets in turn): log decays summed forward, steps, steps
    // decayed to the end of their 16 tokens, and to the chunk's end (the update's
    // weights), the chunk's sum; and the raw steps of the chunk after
    __shared__ __attribute__((aligned(16))) float s_cum[2][HW][kQ], s_dt[2][HW][kQ], s_f[2][HW][kQ], s_w[2][HW][kQ], s_raw[HW][kQ];
    __shared__ float s_tot[2][HW];
    __shared__ __attribute__((aligned(16))) uint16_t s_B[kQ * kBs], s_X[HW][kQ * kXs];
    __shared__ __attribute__((aligned(16))) uint16_t s_C[LOCAL ? 8 : kQ * kCs], s_P[LOCAL ? 1 : HW][LOCAL ? 8 : kQ * kPs];

    const int tid = threadIdx.x, lane = tid & (kWave - 1), w = __builtin_amdgcn_readfirstlane(tid / kWave);
    int slot, hb;
    place_block(plan, a.H / HW, &slot, &hb);
    const int h0 = hb * HW;
    const Segment sg = find_segment<TH, LOCAL>(a.seq_start, a.n_seqs, a.n_tokens, plan, slot, false, s_red, &s_seg, s_len);
    if (!sg.ok || (LOCAL && sg.k == sg.n - 1)) return;
    const int l16 = lane & 15, lg = lane >> 4;
    const int wh = HW == 2 ? w >> 1 : 0, h = h0 + wh, pw = HW == 2 ? 32 * (w & 1) : 16 * w;  // this wave's head, first row
    const int g = h0 / (a.H / a.G);
    const float Dh = LOCAL ? 0.f : a.D[h];
    constexpr size_t PN = (size_t)kP * N;
    // row m of p-tile t is p = pw + 4 PT (m / 4) + 4 t + m % 4: a lane then holds
    // 4 PT consecutive p of an output, one 16-byte piece for two tiles
    const int pl = pw + 4 * PT * (l16 >> 2) + (l16 & 3);  // of this lane's state column, + 4 t

    // state: tile nt, element r of this lane is n = 16 nt + 4 lg + r of row pl + 4 t
    f32x4 st[PT][NT];
    if (LOCAL) {
#pragma unroll
        for (int t = 0; t < PT; ++t)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) st[t][nt] = f32x4{0.f, 0.f, 0.f, 0.f};
    } else {
        const float* from = sg.n == 1 ? a.h + ((size_t)sg.seq * a.H + h) * PN
                                      : ws.state + ((size_t)(sg.base + (sg.k ? sg.k - 1 : sg.n - 1)) * a.H + h) * PN;
#pragma unroll
        for (int t = 0; t < PT; ++t)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                st[t][nt] = *(const f32x4*)(from + (size_t)(pl + 4 * t) * N + 16 * nt + 4 * lg);
    }
    if (!LOCAL)  // tiles above the diagonal that a 32-token product covers stay zero
        for (int i = tid; i < HW * kQ * kPs / 8; i += TH) ((uint4*)s_P)[i] = make_uint4(0, 0, 0, 0);
    if (tid == 0) s_odd = 0;

    // A wave fetches 16 tokens' steps (HW heads in one load), two chunks ahead.
    // Waves 0 and 1 sum the log decays of a head forward, waves 2 and 3 from the
    // chunk's end (lanes reversed), one chunk ahead.
    const int sh = HW == 2 ? w & 1 : 0, stok = w < 2 ? lane : kQ - 1 - lane;
    const float Ash = a.A[h0 + sh];
    uint32_t rdt = 0;  // as loaded: a conversion here would wait for the load
    int rdt_rows = 0;
    auto request_dt = [&](int t0) {
        rdt_rows = sg.t1 - t0;
        const int t = max(min(t0 + 16 * w + l16, sg.t1 - 1), sg.t0);
        const uint16_t* d = (const uint16_t*)a.dt + (size_t)t * a.H + h0;
        rdt = HW == 2 ? gload((const uint32_t*)d) : gload(d);
    };
    auto stage_dt = [&]() {
        const uint32_t u = 16 * w + l16 < rdt_rows ? rdt : 0;
        if (lane < 16) {
            s_raw[0][16 * w + l16] = __uint_as_float(u << 16);
            if (HW == 2) s_raw[HW - 1][16 * w + l16] = __uint_as_float(u & 0xffff0000u);
        }
    };
    auto sum_decays = [&](int set) {
        if (HW == 1 && (w & 1)) return;
        const float dt = s_raw[sh][stok];
        float da = dt * Ash;
        da = da < -128.f ? -128.f : da;  // exp is 0 either way, and sums stay exact enough
        const float to = prefix_sum(da);
        if (w < 2) {
            s_cum[set][sh][lane] = to;
            s_dt[set][sh][lane] = dt;
            s_f[set][sh][lane] = __expf(__shfl(to, lane | 15, kWave) - to) * dt;
        } else {
            // the sum of the later tokens: that of the lane before
            const float after = __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(
                0, (int)__float_as_uint(to), 0x138, 0xf, 0xf, false));  // wave_shr:1, 0 into lane 0
            s_w[set][sh][stok] = __expf(after) * dt;
            if (lane == kWave - 1) s_tot[set][sh] = to;
        }
    };

    uint4 rB[BP], rC[LOCAL ? 1 : BP], rX[XP];
    const int sB = a.G * N, sX = a.H * kP;  // row strides
    // A thread's pieces of a tile are BR (XR) rows apart; `rows` of the segment are
    // left (in a last, short chunk the rows behind it are read again from it)
    constexpr int BR = TH / (N / 8), XR = TH / (8 * HW);
    const int brow = tid / (N / 8), bcol = tid % (N / 8) * 8, xrow = tid / (8 * HW), xcol = tid % (8 * HW) * 8;
    const uint32_t boff = (uint32_t)brow * sB + bcol, xoff = (uint32_t)xrow * sX + xcol;
    auto request_tile = [&](uint4* r, const uint16_t* p, int rows) {
        if (rows >= kQ) {
#pragma unroll
            for (int i = 0; i < BP; ++i) r[i] = gload((const uint4*)(p + (size_t)i * BR * sB + boff));
        } else {
#pragma unroll
            for (int i = 0; i < BP; ++i) r[i] = gload((const uint4*)(p + ((uint32_t)min(brow + i * BR, rows - 1) * sB + bcol)));
        }
    };
    auto request_B = [&](int t0) { request_tile(rB, (const uint16_t*)a.B + ((size_t)t0 * a.G + g) * N, sg.t1 - t0); };
    auto request_C = [&](int t0) { request_tile(rC, (const uint16_t*)a.C + ((size_t)t0 * a.G + g) * N, sg.t1 - t0); };
    auto request_x = [&](int t0) {
        const uint16_t* p = (const uint16_t*)a.x + ((size_t)t0 * a.H + h0) * kP;
        const int rows = sg.t1 - t0;
        if (rows >= kQ) {
#pragma unroll
            for (int i = 0; i < XP; ++i) rX[i] = gload((const uint4*)(p + (size_t)i * XR * sX + xoff));
        } else {
#pragma unroll
            for (int i = 0; i < XP; ++i) rX[i] = gload((const uint4*)(p + ((uint32_t)min(xrow + i * XR, rows - 1) * sX + xcol)));
        }
    };
    request_B(sg.t0);
    if (!LOCAL) request_C(sg.t0);
    request_x(sg.t0);
    request_dt(sg.t0);
    stage_dt();
    request_dt(sg.t0 + kQ);
    __syncthreads();
    sum_decays(0);
    float sum = 0.f;
    int set = 0;

    for (int t0 = sg.t0; t0 < sg.t1; t0 += kQ, set ^= 1) {
        const int cnt = min(kQ, sg.t1 - t0);
        lds_barrier();  // the last chunk's reads are done
        if (cnt < kQ) {   // rows behind the segment are zero
#pragma unroll
            for (int i = 0; i < BP; ++i)
                if (brow + i * BR >= cnt) {
                    rB[i] = make_uint4(0, 0, 0, 0);
                    if (!LOCAL) rC[i] = make_uint4(0, 0, 0, 0);
                }
#pragma unroll
            for (int i = 0; i < XP; ++i)
                if (xrow + i * XR >= cnt) rX[i] = make_uint4(0, 0, 0, 0);
        }
        stage_dt();
        uint32_t strange = 0;
#pragma unroll
        for (int i = 0; i < XP; ++i) {
            *(uint4*)&s_X[xcol / kP][(xrow + i * XR) * kXs + xcol % kP] = rX[i];
            if (!LOCAL) strange |= nonfinite_bits(rX[i]);
        }
        if (!LOCAL && (strange & 0x80008000u)) s_odd = 1;
#pragma unroll
        for (int i = 0; i < BP; ++i) {
            *(uint4*)&s_B[(brow + i * BR) * kBs + bcol] = rB[i];
            if (!LOCAL) *(uint4*)&s_C[(brow + i * BR) * kCs + bcol] = rC[i];
        }
        lds_barrier();
        const bool more = t0 + kQ < sg.t1;
        if (more) request_B(t0 + kQ);
        const float tot = s_tot[set][wh];
        f32x4 y[PT][4];
        bool odd = false;
        if (!LOCAL) {
            odd = s_odd;
            // Scores, weighted, as P[i][j]: of the 10 lower tiles of 16 x 16, wave w has the
            // one on the diagonal and (3, 0), (1, 0), (2, 0 1), (3, 1 2). Below the diagonal
            // exp(cum_i - cum_j) = exp(cum_i - cum_end of j's tile) times a factor of j that
            // is one table; on it every element takes its own exponential.
            {
                const int it1 = w == 0 ? 3 : w, jt1 = w == 3;
                f32x4 s[3];
#pragma unroll
                for (int u = 0; u < 3; ++u) s[u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    const int o = l16 * kBs + 32 * k + 8 * lg, oc = l16 * kCs + 32 * k + 8 * lg;
                    s[0] = mma(*(const bf16x8*)&s_B[16 * w * kBs + o], *(const bf16x8*)&s_C[16 * w * kCs + oc], s[0]);
                    const bf16x8 c1 = *(const bf16x8*)&s_C[16 * it1 * kCs + oc];
                    s[1] = mma(*(const bf16x8*)&s_B[16 * jt1 * kBs + o], c1, s[1]);
                    s[2] = mma(*(const bf16x8*)&s_B[(16 * jt1 + 16) * kBs + o], c1, s[2]);
                }
#pragma unroll
                for (int x = 0; x < HW; ++x) {
                    const int i = 16 * w + l16, j = 16 * w + 4 * lg;
                    const float ci = s_cum[set][x][i];
                    const f32x4 cj = *(const f32x4*)&s_cum[set][x][j], dj = *(const f32x4*)&s_dt[set][x][j];
                    float v[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        v[r] = s[0][r] * (__expf(ci - cj[r]) * dj[r]);  // before the choice: it would become a branch
                        v[r] = 4 * lg + r <= l16 ? v[r] : 0.f;
                    }
                    *(uint2*)&s_P[x][i * kPs + j] = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
                }
#pragma unroll
                for (int u = 1; u < 3; ++u) {
                    if (u == 2 && w < 2) break;
                    const int i = 16 * it1 + l16, j0 = 16 * (jt1 + u - 1), j = j0 + 4 * lg;
#pragma unroll
                    for (int x = 0; x < HW; ++x) {
                        const float ei = __expf(s_cum[set][x][i] - s_cum[set][x][j0 + 15]);
                        const f32x4 v = s[u] * (ei * *(const f32x4*)&s_f[set][x][j]);
                        *(uint2*)&s_P[x][i * kPs + j] = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
                    }
                }
            }
            // read-out of the state before the chunk
#pragma unroll
            for (int t = 0; t < PT; ++t)
#pragma unroll
                for (int it = 0; it < 4; ++it) y[t][it] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                Parts<2> sp[PT];
#pragma unroll
                for (int t = 0; t < PT; ++t) {
                    float v[8];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        v[r] = st[t][2 * k][r];
                        v[4 + r] = st[t][2 * k + 1][r];
                    }
                    sp[t] = split<2>(v);
                }
                bf16x8 cf[4];
#pragma unroll
                for (int it = 0; it < 4; ++it) cf[it] = read_row(&s_C[(16 * it + l16) * kCs + 32 * k + 4 * lg]);
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int t = 0; t < PT; ++t)
#pragma unroll
                        for (int it = 0; it < 4; ++it) y[t][it] = mma(sp[t].part[n], cf[it], y[t][it]);
            }
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const float e = __expf(s_cum[set][wh][16 * it + l16]);
#pragma unroll
                for (int t = 0; t < PT; ++t) y[t][it] *= e;
            }
        }
        if (more) {
            if (!LOCAL) request_C(t0 + kQ);
            request_x(t0 + kQ);
        }
        request_dt(t0 + 2 * kQ);
        // update: S' = exp(tot) S + B^T (w x)
        const float keep = __expf(tot);
#pragma unroll
        for (int t = 0; t < PT; ++t)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) st[t][nt] *= keep;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const f32x4 w0 = *(const f32x4*)&s_w[set][wh][32 * k + 4 * lg], w1 = *(const f32x4*)&s_w[set][wh][32 * k + 16 + 4 * lg];
            Parts<3> wx[PT];
#pragma unroll
            for (int t = 0; t < PT; ++t) {
                float v[8];
                const s16x8 xs = __builtin_bit_cast(s16x8, read_columns<4 * PT>(&s_X[wh][32 * k * kXs + pw + 4 * t], kXs, lane));
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = bf16_bits_to_f32((uint16_t)xs[e]) * (e < 4 ? w0[e] : w1[e - 4]);
                wx[t] = split<3>(v);
            }
#pragma unroll
            for (int n2 = 0; n2 < NT; n2 += 2) {
                bf16x8 bf[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) bf[i] = read_columns(&s_B[32 * k * kBs + 16 * (n2 + i)], kBs, lane);
#pragma unroll
                for (int n = 0; n < 3; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int t = 0; t < PT; ++t) st[t][n2 + i] = mma(bf[i], wx[t].part[n], st[t][n2 + i]);
            }
        }
        sum_decays(set ^ 1);
        if (LOCAL) {
            sum += tot;
            continue;
        }
        lds_barrier();  // P is whole
        if (tid == 0) s_odd = 0;
        bf16x8 xf[PT][2];
#pragma unroll
        for (int t = 0; t < PT; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                xf[t][k] = read_columns<4 * PT>(&s_X[wh][32 * k * kXs + pw + 4 * t], kXs, lane);
                if (odd) {
                    // an x that is not finite must not reach earlier tokens through a
                    // weight of 0: it leaves the matrix product and is added alone
                    s16x8 xs = __builtin_bit_cast(s16x8, xf[t][k]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) xs[e] = (xs[e] & 0x7f80) == 0x7f80 ? (short)0 : xs[e];
                    xf[t][k] = __builtin_bit_cast(bf16x8, xs);
                }
            }
#pragma unroll
        for (int it = 0; it < 4; ++it)
#pragma unroll
            for (int k = 0; k <= it / 2; ++k) {
                const bf16x8 pf = read_row(&s_P[wh][(16 * it + l16) * kPs + 32 * k + 4 * lg]);
#pragma unroll
                for (int t = 0; t < PT; ++t) y[t][it] = mma(xf[t][k], pf, y[t][it]);
            }
        if (odd) {
            for (int j = 0; j < kQ; ++j) {
#pragma unroll
                for (int t = 0; t < PT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const uint16_t xb = s_X[wh][j * kXs + pw + 4 * PT * lg + 4 * t + r];
                        if ((xb & 0x7f80) != 0x7f80) continue;
#pragma unroll
                        for (int it = 0; it < 4; ++it) {
                            const int i = 16 * it + l16;
                            if (i >= j) y[t][it][r] += bf16_bits_to_f32(s_P[wh][i * kPs + j]) * bf16_bits_to_f32(xb);
                        }
                    }
            }
        }
        uint16_t* yp = (uint16_t*)a.y + ((size_t)t0 * a.H + h) * kP;
        const int q = pw + 4 * PT * lg;
        uint32_t o[4][2 * PT];
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            uint32_t xr[2 * PT];
            if constexpr (PT == 2)
                *(uint4*)xr = *(const uint4*)&s_X[wh][(16 * it + l16) * kXs + q];
            else
                *(uint2*)xr = *(const uint2*)&s_X[wh][(16 * it + l16) * kXs + q];
#pragma unroll
            for (int t = 0; t < PT; ++t)
#pragma unroll
                for (int r = 0; r < 4; r += 2) {
                    const uint32_t u = xr[2 * t + r / 2];
                    o[it][2 * t + r / 2] = pack_bf16x2(fmaf(Dh, __uint_as_float(u << 16), y[t][it][r]),
                                                       fmaf(Dh, __uint_as_float(u & 0xffff0000u), y[t][it][r + 1]));
                }
        }
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            uint16_t* to = yp + (size_t)it * 16 * sX + ((uint32_t)l16 * sX + q);
            if (16 * it + l16 < cnt) {
                if constexpr (PT == 2)
                    gstore((uint4*)to, make_uint4(o[it][0], o[it][1], o[it][2], o[it][3]));
                else
                    gstore((uint2*)to, make_uint2(o[it][0], o[it][1]));
            }
        }
    }
    if (!LOCAL && sg.k != sg.n - 1) return;
    float* to = LOCAL ? ws.state + ((size_t)(sg.base + sg.k) * a.H + h) * PN : a.h + ((size_t)sg.seq * a.H + h) * PN;
#pragma unroll
    for (int t = 0; t < PT; ++t)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) *(f32x4*)(to + (size_t)(pl + 4 * t) * N + 16 * nt + 4 * lg) = st[t][nt];
    if (LOCAL && lane == 0 && pw == 0) ws.sum[(size_t)(sg.base + sg.k) * a.H + h] = sum;
}

template <int NT, bool LOCAL>
void launch_pass(const PrefillArgs& a, const SeqPlan& p, const SeqWorkspace& ws, hipStream_t stream) {
    // Two heads of a group at once where the groups have an even number (their
    // steps are then one aligned word) and the GPU is full that way; a few short
    // prompts are sooner done with twice the work-groups (77 tokens, 80 heads:
    // 13.1 against 18.4 us of kernel time).
    const bool even = a.H / a.G % 2 == 0 && (uintptr_t)a.dt % 4 == 0;
    const int hw = even && (long long)p.slots * a.H >= 512 ? 2 : 1;
    const dim3 grid((unsigned)((long long)p.slots * (a.H / hw)));
    if (hw == 2)
        hipLaunchKernelGGL((prefill_mfma_kernel<NT, 2, LOCAL>), grid, dim3(256), 0, stream, a, p, ws);
    else
        hipLaunchKernelGGL((prefill_mfma_kernel<NT, 1, LOCAL>), grid, dim3(256), 0, stream, a, p, ws);
}

}  // namespace

bool prefill_mfma_aligned(const PrefillArgs& a) {
    const uintptr_t all = (uintptr_t)a.x | (uintptr_t)a.B | (uintptr_t)a.C | (uintptr_t)a.y | (uintptr_t)a.h;
    return all % 16 == 0;
}

void launch_prefill_mfma(const PrefillArgs& a, const SeqPlan& p, const SeqWorkspace& ws, bool local, hipStream_t stream) {
    if (a.N == 64)
        local ? launch_pass<4, true>(a, p, ws, stream) : launch_pass<4, false>(a, p, ws, stream);
    else
        local ? launch_pass<8, true>(a, p, ws, stream) : launch_pass<8, false>(a, p, ws, stream);
}

}  // namespace tsv
