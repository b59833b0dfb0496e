// prefill.hip -- the prompt scan over packed sequences: the launches (segments'
// local states, their combination, the scan; seq_common.hpp) and the plain fp32
// kernel for any P, N <= 256. The bf16 kernel is in prefill_mfma.hip.
//
// Plain kernel: the recurrence token by token. A lane holds one row p of the
// state and a wave a quarter of the columns n, so the decay, the update and the
// read-out of a token are 3 NS operations per lane without a reduction across
// lanes; the four waves' parts of y meet in LDS once per 16 tokens. Bound by
// the vector ALU: 3 P N operations per token and head, four cycles for each 64
// of them.
#include "seq_common.hpp"

namespace tsv {
namespace {

constexpr int kTok = 16;  // tokens staged at a time

template <typename TIO, int NS, bool LOCAL>
__global__ __launch_bounds__(256) void prefill_plain_kernel(PrefillArgs a, SeqPlan plan, SeqWorkspace ws, int pblocks) {
    __shared__ int s_red[4];
    __shared__ Segment s_seg;
    __shared__ int s_len[kSortMax];
    __shared__ __attribute__((aligned(16))) float s_B[kTok][4 * NS], s_C[kTok][4 * NS];
    __shared__ float s_x[kTok][kWave], s_y[4][kTok][kWave], s_dec[kTok], s_dt[kTok];
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
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const int n = w * NS + i;
        st[i] = !LOCAL && row && n < N ? from[(size_t)p * N + n] : 0.f;
    }
    const float Ah = a.A[h], Dh = a.D[h];
    const int g = h / (a.H / a.G);
    float sum = 0.f;
    for (int t0 = sg.t0; t0 < sg.t1; t0 += kTok) {
        const int cnt = min(kTok, sg.t1 - t0);
        __syncthreads();
        for (int i = tid; i < kTok * 4 * NS; i += 256) {
            const int t = i / (4 * NS), n = i % (4 * NS);
            const bool in = t < cnt && n < N;
            const size_t at = ((size_t)(t0 + t) * a.G + g) * N + n;
            s_B[t][n] = in ? Elem<TIO>::ld((const TIO*)a.B, at) : 0.f;
            if (!LOCAL) s_C[t][n] = in ? Elem<TIO>::ld((const TIO*)a.C, at) : 0.f;
        }
        for (int i = tid; i < kTok * kWave; i += 256) {
            const int t = i / kWave, q = pb * kWave + i % kWave;
            s_x[t][i % kWave] =
                t < cnt && q < P ? Elem<TIO>::ld((const TIO*)a.x, ((size_t)(t0 + t) * a.H + h) * P + q) : 0.f;
        }
        if (tid < cnt) {
            const float dt = Elem<TIO>::ld((const TIO*)a.dt, (size_t)(t0 + tid) * a.H + h);
            s_dt[tid] = dt;
            s_dec[tid] = LOCAL ? dt * Ah : expf(dt * Ah);
        }
        __syncthreads();
#pragma unroll 2
        for (int t = 0; t < cnt; ++t) {
            float decay = s_dec[t];
            if (LOCAL) {
                sum += decay;
                decay = expf(decay);
            }
            const float wx = s_dt[t] * s_x[t][lane];
            float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < NS; i += 4) {
                const float4 B4 = *(const float4*)&s_B[t][w * NS + i];
                st[i] = fmaf(decay, st[i], wx * B4.x);
                st[i + 1] = fmaf(decay, st[i + 1], wx * B4.y);
                st[i + 2] = fmaf(decay, st[i + 2], wx * B4.z);
                st[i + 3] = fmaf(decay, st[i + 3], wx * B4.w);
                if (!LOCAL) {
                    const float4 C4 = *(const float4*)&s_C[t][w * NS + i];
                    y[0] = fmaf(st[i], C4.x, y[0]);
                    y[1] = fmaf(st[i + 1], C4.y, y[1]);
                    y[2] = fmaf(st[i + 2], C4.z, y[2]);
                    y[3] = fmaf(st[i + 3], C4.w, y[3]);
                }
            }
            if (!LOCAL) s_y[w][t][lane] = (y[0] + y[1]) + (y[2] + y[3]);
        }
        if (!LOCAL) {
            __syncthreads();
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
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const int n = w * NS + i;
        if (row && n < N) to[(size_t)p * N + n] = st[i];
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
    hipLaunchKernelGGL((prefill_plain_kernel<TIO, NS, LOCAL>), grid, dim3(256), 0, stream, a, p, ws, pblocks);
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

void launch_combine(const PrefillArgs& a, const SeqPlan& p, const SeqWorkspace& ws, hipStream_t stream) {
    const bool vec = a.P * a.N % 4 == 0 && (uintptr_t)a.h % 16 == 0 && (uintptr_t)ws.state % 16 == 0;
    const int chunks = (a.P * a.N + 256 * (vec ? 4 : 1) - 1) / (256 * (vec ? 4 : 1));
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
int min_seg_of(const tsv_seq_shape* s) { return matrix_shape(s) ? kMinSegMatrix : kMinSegPlain; }

}  // namespace

uint64_t prefill_workspace_bytes(const tsv_seq_shape* s) {
    return seq_workspace_bytes(seq_plan(s->n_seqs, s->n_tokens, s->n_heads, min_seg_of(s)), s->n_heads, s->head_dim, s->d_state);
}

long long prefill_blocks(const tsv_seq_shape* s) {
    const SeqPlan p = seq_plan(s->n_seqs, s->n_tokens, s->n_heads, min_seg_of(s));
    const long long scan = (long long)p.slots * s->n_heads * ((s->head_dim + kWave - 1) / kWave);
    const long long combine = (long long)s->n_seqs * s->n_heads * (((long long)s->head_dim * s->d_state + 255) / 256);
    return scan > combine ? scan : combine;
}

hipError_t launch_prefill(const PrefillArgs& a, const tsv_seq_shape* s, int32_t* status, void* workspace, hipStream_t stream) {
    const bool bf16 = s->in_dtype == TSV_BF16;
    if (status)
        hipLaunchKernelGGL(seq_status_kernel, dim3(1), dim3(256), 0, stream, a.seq_start, a.n_seqs, a.n_tokens, status);
    if (a.n_tokens > 0) {
        const bool matrix = matrix_shape(s) && prefill_mfma_aligned(a);
        const SeqPlan p = seq_plan(a.n_seqs, a.n_tokens, a.H, min_seg_of(s));
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
