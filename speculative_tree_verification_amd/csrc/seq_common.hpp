// seq_common.hpp -- how the prompt scan cuts packed sequences into segments.
//
// The recurrence is sequential along a sequence, and one sequence has only
// n_heads independent states: 80 work-groups on 256 compute units. A sequence
// of more than `seg` tokens is therefore cut into segments of `seg` tokens:
//   local    every segment but a sequence's last one forms the state it would
//            leave from a zero state, and the sum of its log decays;
//   combine  one pass over the segments of each sequence turns those into the
//            state before each segment (H_k = exp(sum_k) H_{k-1} + local_k);
//   scan     every segment runs from its own state and writes y.
// Segments are numbered through all sequences ("slots"); a work-group finds
// the sequence of its slot from seq_start, so the cut follows the lengths that
// are on the device and the launch needs only an upper bound of the slots.
#pragma once

#include "common.hpp"
#include "seq_launch.hpp"

namespace tsv {

constexpr int kStBadSeq = 32;

// `seg` tokens so that all (segment, head) pairs fit the GPU at once (two
// work-groups of two heads on each of the 256 compute units; every sequence may
// end with a short segment), a multiple of the chunk and at least min_seg
// (four chunks for the matrix kernel: below that the second pass over the inputs
// costs more than the parallelism gives). Many sequences fill the GPU by themselves; half of the
// room is then the measure, so that only sequences much longer than the others
// are cut.
struct SeqPlan {
    int seg;        // tokens per segment
    long long slots;  // upper bound of segments over all sequences
    bool split;     // whether a sequence may have more than one
    bool sorted;    // slots follow the sequences by falling length, dealt to the XCDs in turn
};

// Many sequences of different lengths are taken longest first, so that no long
// one starts last: 32 prompts of 1 to 1531 tokens, 64 heads, took 237 us in
// their own order and 179 us so. Work-groups that share B and C (the heads of
// a slot) stay on one XCD, and slots go to the XCDs forwards and backwards in
// turn. With few sequences there is nothing to deal, and past 256 the search
// would cost more than it gives.
constexpr int kSortMin = 16, kSortMax = 256;

constexpr int kMinSegMatrix = 256;

// The plain kernel works token by token, so it takes shorter segments, cut to 16
// tokens. fp32, N = 128: 3 prompts of 1360 tokens, 24 heads, 88 us with segments of 48,
// 99 with 64; 1 prompt of 128 tokens 45 us in segments of 48, 56 in one, but of 64
// tokens 44 and 31, of 96 tokens 45 and 43; and where the heads of the prompts fill
// the GPU by themselves, a second pass over short ones costs more than it gives
// (16 prompts of 128 tokens 123 us in segments of 80, 92 in one).
inline int min_seg_plain(int n_seqs, int n_tokens, int n_heads) {
    return n_tokens <= 96 ? 96 : (long long)n_seqs * n_heads < 256 ? 48 : 128;
}

inline SeqPlan seq_plan(int n_seqs, int n_tokens, int n_heads, bool matrix) {
    constexpr long long kWant = 1024;
    const int min_seg = matrix ? kMinSegMatrix : min_seg_plain(n_seqs, n_tokens, n_heads), unit = matrix ? 64 : 16;
    long long room = kWant - (long long)n_seqs * n_heads;
    if (room < kWant / 2) room = kWant / 2;
    long long seg = ((long long)n_tokens * n_heads + room - 1) / room;
    seg = (seg + unit - 1) / unit * unit;
    if (seg < min_seg) seg = min_seg;
    if (seg > 0x7fffffc0LL) seg = 0x7fffffc0LL;
    SeqPlan p;
    p.seg = (int)seg;
    p.slots = (long long)(n_tokens / p.seg) + (n_seqs < n_tokens ? n_seqs : n_tokens);
    p.split = n_tokens > p.seg;
    p.sorted = n_seqs >= kSortMin && n_seqs <= kSortMax;
    if (p.sorted) p.slots = (p.slots + 7) / 8 * 8;
    return p;
}

// Slot and head block of a work-group, of HB head blocks
__device__ __forceinline__ void place_block(const SeqPlan& plan, int HB, int* slot, int* hb) {
    if (plan.sorted) {
        const int xcd = blockIdx.x % 8, i = blockIdx.x / 8, row = i / HB;
        *slot = 8 * row + (row & 1 ? 7 - xcd : xcd);
        *hb = i % HB;
    } else {
        const int lid = xcd_block(blockIdx.x, gridDim.x);
        *slot = lid / HB;
        *hb = lid % HB;
    }
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(uint16_t bf16) { return bf16_bits_to_f32(bf16); }

// The states of all slots, then the log-decay sums.
struct SeqWorkspace {
    float* state;  // [slots][H][P * N]
    float* sum;    // [slots][H]
};
inline uint64_t seq_workspace_bytes(const SeqPlan& p, int H, int P, int N) {
    return p.split ? (uint64_t)p.slots * H * ((uint64_t)P * N + 4) * sizeof(float) : 0;
}
inline SeqWorkspace seq_workspace(void* ws, const SeqPlan& p, int H, int P, int N) {
    SeqWorkspace w;
    w.state = (float*)ws;
    w.sum = w.state ? w.state + (size_t)p.slots * H * P * N : nullptr;
    return w;
}

// bf16 MFMA kernel (prefill_mfma.hip): P 64, N 64 or 128, 16-byte aligned tensors
bool prefill_mfma_aligned(const PrefillArgs& a);
void launch_prefill_mfma(const PrefillArgs& a, const SeqPlan& p, const SeqWorkspace& ws, bool local, hipStream_t stream);

struct Segment {
    int ok;           // 0: no such slot, or seq_start is invalid
    int seq, k, n;    // sequence, index among its n segments
    int base;         // slot of the sequence's segment 0
    int t0, t1;       // rows
};

// Whether seq_start is 0 <= start[0] <= ... <= start[n] <= n_tokens (the answer
// is the same in all threads), and, for `want` >= 0, the segment of that slot,
// or, with by_seq, segment 0 of that sequence. `s_red` and `s_out`: LDS scratch
// of NT/64 ints and of one Segment; s_len: of kSortMax ints.
// Acts as a barrier.
// SPLIT: only sequences of more than one segment matter; where there is none the
// search ends early.
template <int NT, bool SPLIT = false>
__device__ __forceinline__ Segment find_segment(const int32_t* __restrict__ seq_start, int n_seqs, int n_tokens,
                                                const SeqPlan& plan, int want, bool by_seq, int* s_red, Segment* s_out,
                                                int* s_len) {
    static_assert(NT >= kSortMax, "a thread for each sequence of a sorted plan");
    const int seg = plan.seg;
    if (threadIdx.x == 0) s_out->ok = 0;
    __syncthreads();
    int run = 0, bad = 0;
    for (int q0 = 0; q0 < n_seqs; q0 += NT) {
        const int q = q0 + threadIdx.x;
        int a = 0, b = 0;
        if (q < n_seqs) {
            a = seq_start[q];
            b = seq_start[q + 1];
        }
        if (a < 0 || b < a || b > n_tokens) {
            bad = 1;
            b = a;
        }
        const int len = b - a;
        const int cnt = len / seg + (len % seg != 0);
        int base = 0, total = 0;
        if (plan.sorted) {
            if (SPLIT && !__syncthreads_or(len > seg)) break;  // all sequences are here (at most NT)
            if (q < n_seqs) s_len[q] = len;
            __syncthreads();
            for (int j = 0; j < n_seqs; ++j) {
                const int l = s_len[j];
                if (l > len || (l == len && j < q)) base += l <= seg ? l > 0 : l / seg + (l % seg != 0);
            }
        } else {
            base = run + block_exclusive_scan<NT>(cnt, s_red, &total);
        }
        const bool mine = q < n_seqs && (by_seq ? q == want : want >= base && want < base + cnt);
        if (mine) {
            const int k = by_seq ? 0 : want - base;
            s_out->seq = q;
            s_out->k = k;
            s_out->n = cnt;
            s_out->base = base;
            s_out->t0 = a + k * seg;
            s_out->t1 = b - s_out->t0 > seg ? s_out->t0 + seg : b;
            s_out->ok = 1;
        }
        run += total;
    }
    bad = __syncthreads_or(bad);
    Segment r = *s_out;
    if (bad) r.ok = 0;
    return r;
}

}  // namespace tsv
