// prefill.hip -- the prompt scan over packed sequences: the launches (segments'
// local states, their combination, the scan; seq_common.hpp) and the plain fp32
// kernel for any P, N <= 256. The bf16 kernel is in prefill_mfma.hip.
//
// Plain kernel: the recurrence token by token. A lane holds one row p of the
// state and a wave a quarter of the columns n, so the decay, the update and the
// read-out of a token are 3 NS operations per lane without a reduction across
// lanes; the four waves' parts of y meet in LDS once per 16 tokens. The scan of
// 1360 tokens, 24 heads, N = 128 takes 45 us and the local pass 30. Their vector
// work, 3 P N and 2 P N operations per token and head at four cycles for each 64,
// is 20 and 13 us of that; what the rest waits for (few waves a SIMD, each of
// which steps from token to token) was not taken apart.
#include "seq_common.hpp"

namespace tsv {
namespace {

constexpr int kTok = 16;  // tokens staged at a time

// FULL: fp32 with N == 4 NS, 16-byte aligned states. B and C are then the same
// four cache lines for all lanes of a wave and come through the scalar cache into
// scalar registers; broadcast from LDS they bound the kernel (a 16-byte read
// returns 1 KB to the lanes: 51 and 65 us against 34 and 54 us for the two passes over
// 1360 tokens, 24 heads, in segments of 64; 30 and 45 us in those of 48).
template <typename TIO, int NS, bool LOCAL, bool FULL>
__global__ __launch_bounds__(256) void prefill_plain_kernel(PrefillArgs a, SeqPlan plan, SeqWorkspace ws, int pblocks) {
    __shared__ int s_red[4];
    __shared__ Segment s_seg;
    __shared__ int s_len[kSortMax];
    __shared__ __attribute__((aligned(16))) float s_B[FULL ? 1 : kTok][4 * NS], s_C[FULL || LOCAL ? 1 : kTok][4 * NS];
    __shared__ float s_x[kTok][kWave], s_y[4][kTok][kWave], s_dec[kTok], s_da[kTok], s_dt[kTok];
    const int tid = threadIdx.x, lane = tid & (kWave - 1), w = __builtin_amdgcn_readfirstlane(tid / kWave);
    int slot, hb;
    place_block(plan, a.H * pblocks, &slot, &hb);
    const int pb = hb % pblocks, h = hb / pblocks;
    const Segment sg = find_segment<256, LOCAL>(a.seq_start, a.n_seqs, a.n_tokens, plan, slot, false, s_red, &s_seg, s_len);
    if (!sg.ok) return;
    if (LOCAL && sg.k == sg.n - 1) return;
    const int p = pb * kWave + lane, P = a.P, N = a.N;
    const size_t PN = (size_t)P * N;
    const bool row = p < P;
    // the state before this segment: the caller's where the sequence has one
    // segment, else what the combining pass left (its copy of the caller's
    // state for segment 0: the last segment overwrites the caller's)
    float st[NS];
    const float* from = sg.n == 1 ? a.h + ((size_t)sg.seq * a.H + h) * PN
                                  : ws.state + ((size_t)(sg.base + (sg.k ? sg.k - 1 : sg.n - 1)) * a.H + h) * PN;
    if (LOCAL) {
#pragma unroll
        for (int i = 0; i < NS; ++i) st[i] = 0.f;
    } else if (FULL) {
#pragma unroll
        for (int i = 0; i < NS; i += 4) {
            const float4 v = gload((const float4*)(from + (size_t)min(p, P - 1) * N + w * NS + i));
            st[i] = v.x; st[i + 1] = v.y; st[i + 2] = v.z; st[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NS; ++i) st[i] = gload(from + (size_t)min(p, P - 1) * N + min(w * NS + i, N - 1));
#pragma unroll
        for (int i = 0; i < NS; ++i) st[i] = w * NS + i < N ? st[i] : 0.f;
    }
    const float Ah = a.A[h], Dh = a.D[h];
    const int g = h / (a.H / a.G);
    float sum = 0.f;
    // the next tokens' rows are loaded while these are worked on, from clamped
    // addresses (a load under a condition would be waited for at once) and kept as
    // loaded
    constexpr int BI = FULL ? 0 : kTok * 4 * NS / 256, XI = kTok * kWave / 256;
    TIO rB[BI + 1], rC[BI + 1], rx[XI], rdt;
    auto request = [&](int t0) {
        const int most = sg.t1 - 1;
#pragma unroll
        for (int i = 0; i < BI; ++i) {
            const int e = tid + i * 256, t = e / (4 * NS), n = e % (4 * NS);
            const size_t at = ((size_t)min(t0 + t, most) * a.G + g) * N + min(n, N - 1);
            rB[i] = gload((const TIO*)a.B + at);
            if (!LOCAL) rC[i] = gload((const TIO*)a.C + at);
        }
#pragma unroll
        for (int i = 0; i < XI; ++i) {
            const int e = tid + i * 256, t = e / kWave, q = pb * kWave + e % kWave;
            rx[i] = gload((const TIO*)a.x + ((size_t)min(t0 + t, most) * a.H + h) * P + min(q, P - 1));
        }
        rdt = gload((const TIO*)a.dt + (size_t)min(t0 + tid % kTok, most) * a.H + h);
    };
    request(sg.t0);
    for (int t0 = sg.t0; t0 < sg.t1; t0 += kTok) {
        const int cnt = min(kTok, sg.t1 - t0);
        lds_barrier();
#pragma unroll
        for (int i = 0; i < BI; ++i) {
            const int e = tid + i * 256, t = e / (4 * NS), n = e % (4 * NS);
            const bool in = t < cnt && n < N;
            s_B[t][n] = in ? to_f32(rB[i]) : 0.f;
            if (!LOCAL) s_C[t][n] = in ? to_f32(rC[i]) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < XI; ++i) {
            const int e = tid + i * 256, t = e / kWave, q = pb * kWave + e % kWave;
            s_x[t][e % kWave] = t < cnt && q < P ? to_f32(rx[i]) : 0.f;
        }
        if (tid < cnt) {
            const float dt = to_f32(rdt);
            s_dt[tid] = dt;
            s_da[tid] = dt * Ah;
            s_dec[tid] = expf(dt * Ah);
        }
        lds_barrier();
        if (t0 + kTok < sg.t1) request(t0 + kTok);
#pragma unroll 2
        for (int t = 0; t < cnt; ++t) {
            const float decay = s_dec[t];
            if (LOCAL) sum += s_da[t];
            const float wx = s_dt[t] * s_x[t][lane];
            float y[4] = {0.f, 0.f, 0.f, 0.f};
            typedef const float __attribute__((address_space(4))) uniform_float;  // not written by this launch
            const size_t at = ((size_t)(t0 + t) * a.G + g) * N + w * NS;
            uniform_float* Bu = (uniform_float*)((const float*)a.B + at);
            uniform_float* Cu = (uniform_float*)((const float*)a.C + at);
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                st[i] = fmaf(decay, st[i], wx * (FULL ? Bu[i] : s_B[t][w * NS + i]));
                if (!LOCAL) y[i % 4] = fmaf(st[i], FULL ? Cu[i] : s_C[t][w * NS + i], y[i % 4]);
            }
            if (!LOCAL) s_y[w][t][lane] = (y[0] + y[1]) + (y[2] + y[3]);
        }
        if (!LOCAL) {
            lds_barrier();
            for (int i = tid; i < cnt * kWave; i += 256) {
                const int t = i / kWave, c = i % kWave, q = pb * kWave + c;
                if (q < P) {
                    const float y = (s_y[0][t][c] + s_y[1][t][c]) + (s_y[2][t][c] + s_y[3][t][c]);
                    Elem<TIO>::st((TIO*)a.y, ((size_t)(t0 + t) * a.H + h) * P + q, fmaf(Dh, s_x[t][c], y));
                }
            }
        }
    }
    if (!LOCAL && sg.k != sg.n - 1) return;
    float* to = LOCAL ? ws.state + ((size_t)(sg.base + sg.k) * a.H + h) * PN : a.h + ((size_t)sg.seq * a.H + h) * PN;
    if (FULL) {
#pragma unroll
        for (int i = 0; i < NS; i += 4)
            if (row) gstore((float4*)(to + (size_t)p * N + w * NS + i), make_float4(st[i], st[i + 1], st[i + 2], st[i + 3]));
    } else {
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int n = w * NS + i;
            if (row && n < N) to[(size_t)p * N + n] = st[i];
        }
    }
    if (LOCAL && tid == 0 && pb == 0) ws.sum[(size_t)(sg.base + sg.k) * a.H + h] = sum;
}

// The state before each segment, for sequences of more than one: slot base + k
// gets the state after segment k (k < n - 1), slot base + n - 1 the sequence's
// initial state (the scan of segment 0 reads it there, since the scan of the
// last segment overwrites the caller's). A thread takes V consecutive elements
// through all segments; the loads do not depend on the running state, so they
// run ahead of it.
template <int V>
__global__ __launch_bounds__(256) void prefill_combine_kernel(PrefillArgs a, SeqPlan plan, SeqWorkspace ws, int chunks) {
    __shared__ int s_red[4];
    __shared__ Segment s_seg;
    __shared__ int s_len[kSortMax];
    const int c = blockIdx.x % chunks, h = blockIdx.x / chunks % a.H, q = blockIdx.x / chunks / a.H;
    if (a.seq_start[q + 1] - a.seq_start[q] <= plan.seg) return;
    const Segment sg = find_segment<256, true>(a.seq_start, a.n_seqs, a.n_tokens, plan, q, true, s_red, &s_seg, s_len);
    if (!sg.ok || sg.n < 2) return;
    const size_t PN = (size_t)a.P * a.N;
    const size_t e = ((size_t)c * 256 + threadIdx.x) * V;
    if (e >= PN) return;
    typedef float vec __attribute__((ext_vector_type(V)));
    vec st = *(const vec*)(a.h + ((size_t)sg.seq * a.H + h) * PN + e);
    float* slot = ws.state + ((size_t)sg.base * a.H + h) * PN + e;
    const float* sum = ws.sum + (size_t)sg.base * a.H + h;
    *(vec*)(slot + (size_t)(sg.n - 1) * a.H * PN) = st;
#pragma unroll 4
    for (int k = 0; k < sg.n - 1; ++k) {
        vec* at = (vec*)(slot + (size_t)k * a.H * PN);
        st = expf(sum[(size_t)k * a.H]) * st + *at;
        *at = st;
    }
}

__global__ __launch_bounds__(256) void seq_status_kernel(const int32_t* seq_start, int n_seqs, int n_tokens,
                                                         int32_t* status) {
    int bad = 0;
    for (int q = threadIdx.x; q < n_seqs; q += 256) {
        const int a = seq_start[q], b = seq_start[q + 1];
        bad |= a < 0 || b < a || b > n_tokens;
    }
    bad = __syncthreads_or(bad);
    for (int q = threadIdx.x; q < n_seqs; q += 256) status[q] = bad ? kStBadSeq : 0;
}

template <typename TIO, int NS, bool LOCAL>
void launch_plain_pass(const PrefillArgs& a, const SeqPlan& p, const SeqWorkspace& ws, hipStream_t stream) {
    const int pblocks = (a.P + kWave - 1) / kWave;
    const dim3 grid((unsigned)((long long)p.slots * a.H * pblocks));
    const bool full = sizeof(TIO) == 4 && a.N == 4 * NS && (uintptr_t)a.h % 16 == 0;
    if (full && sizeof(TIO) == 4)
        hipLaunchKernelGGL((prefill_plain_kernel<TIO, NS, LOCAL, sizeof(TIO) == 4>), grid, dim3(256), 0, stream, a, p, ws, pblocks);
    else
        hipLaunchKernelGGL((prefill_plain_kernel<TIO, NS, LOCAL, false>), grid, dim3(256), 0, stream, a, p, ws, pblocks);
}

template <typename TIO, bool LOCAL>
void launch_plain(const PrefillArgs& a, const SeqPlan& p, const SeqWorkspace& ws, hipStream_t stream) {
    if (a.N <= 64)
        launch_plain_pass<TIO, 16, LOCAL>(a, p, ws, stream);
    else if (a.N <= 128)
        launch_plain_pass<TIO, 32, LOCAL>(a, p, ws, stream);
    else
        launch_plain_pass<TIO, 64, LOCAL>(a, p, ws, stream);
}

// Work-groups of the combining pass for a sequence's head
int combine_chunks(int P, int N, bool vec) { return (P * N + 256 * (vec ? 4 : 1) - 1) / (256 * (vec ? 4 : 1)); }

void launch_combine(const PrefillArgs& a, const SeqPlan& p, const SeqWorkspace& ws, hipStream_t stream) {
    const bool vec = prefill_states_vec(a, ws.state);
    const int chunks = combine_chunks(a.P, a.N, vec);
    const dim3 grid((unsigned)((long long)a.n_seqs * a.H * chunks));
    if (vec)
        hipLaunchKernelGGL((prefill_combine_kernel<4>), grid, dim3(256), 0, stream, a, p, ws, chunks);
    else
        hipLaunchKernelGGL((prefill_combine_kernel<1>), grid, dim3(256), 0, stream, a, p, ws, chunks);
}

// Whether the bf16 MFMA kernel takes the shape (its tensors' alignment is looked at
// per call: the plain kernel then runs with the same segments)
bool matrix_shape(const tsv_seq_shape* s) {
    return s->in_dtype == TSV_BF16 && s->head_dim == 64 && (s->d_state == 64 || s->d_state == 128) &&
           !(s->flags & TSV_FLAG_FORCE_GENERIC);
}

}  // namespace

uint64_t prefill_workspace_bytes(const tsv_seq_shape* s) {
    return seq_workspace_bytes(seq_plan(s->n_seqs, s->n_tokens, s->n_heads, matrix_shape(s)), s->n_heads, s->head_dim, s->d_state);
}

bool prefill_states_vec(const PrefillArgs& a, const void* workspace) {
    return a.P * a.N % 4 == 0 && (uintptr_t)a.h % 16 == 0 && (uintptr_t)workspace % 16 == 0;
}

long long prefill_blocks(const tsv_seq_shape* s, bool states_vec) {
    const SeqPlan p = seq_plan(s->n_seqs, s->n_tokens, s->n_heads, matrix_shape(s));
    const long long scan = (long long)p.slots * s->n_heads * ((s->head_dim + kWave - 1) / kWave);
    const long long combine = p.split ? (long long)s->n_seqs * s->n_heads * combine_chunks(s->head_dim, s->d_state, states_vec) : 0;
    return scan > combine ? scan : combine;
}

hipError_t launch_prefill(const PrefillArgs& a, const tsv_seq_shape* s, int32_t* status, void* workspace, hipStream_t stream) {
    const bool bf16 = s->in_dtype == TSV_BF16;
    if (status)
        hipLaunchKernelGGL(seq_status_kernel, dim3(1), dim3(256), 0, stream, a.seq_start, a.n_seqs, a.n_tokens, status);
    if (a.n_tokens > 0) {
        const bool matrix = matrix_shape(s) && prefill_mfma_aligned(a);
        const SeqPlan p = seq_plan(a.n_seqs, a.n_tokens, a.H, matrix_shape(s));
        const SeqWorkspace ws = seq_workspace(workspace, p, a.H, a.P, a.N);
        for (int pass = p.split ? 0 : 1; pass < 2; ++pass) {
            const bool local = pass == 0;
            if (matrix)
                launch_prefill_mfma(a, p, ws, local, stream);
            else if (bf16)
                local ? launch_plain<uint16_t, true>(a, p, ws, stream) : launch_plain<uint16_t, false>(a, p, ws, stream);
            else
                local ? launch_plain<float, true>(a, p, ws, stream) : launch_plain<float, false>(a, p, ws, stream);
            if (local) launch_combine(a, p, ws, stream);
        }
    }
    return hipGetLastError();
}

}  // namespace tsv
