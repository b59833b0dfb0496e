// attn_common.hpp -- the paged cache and the split of an attention pass over it.
#pragma once

#include <type_traits>

#include "common.hpp"
#include "seq_launch.hpp"

namespace tsv {

constexpr int kStBadSeqRows = 32;
constexpr int kStBadCache = 64;

// n / page_size by a product: exact for 0 <= n < 2^31 (mul = floor(2^(31 + s) /
// d) + 1 with 2^(s - 1) < d <= 2^s exceeds 2^(31 + s) / d by at most 2^s / d of
// a unit, which stays below one part in n)
inline PageDiv page_div(int d) {
    int s = 0;
    while ((1 << s) < d) ++s;
    return PageDiv{(uint32_t)(((1ull << (31 + s)) / (uint32_t)d) + 1), 31 + s};
}
__device__ __forceinline__ int page_of(int n, PageDiv d) { return (int)(((uint64_t)(uint32_t)n * d.mul) >> d.shift); }

// ---------------------------------------------------------------- the split
// The cache positions of all items are cut into parts of `keys` positions (a
// multiple of 64); an item has at least one part (it holds the tree's own
// keys, with the last of the positions). `keys` follows from the lengths on
// the device: the sum of all lengths, times the work-groups that read a
// position (key heads, blocks of query rows), over the work-groups wanted. So
// a batch of short items is not split, one long item is, and in a mixed batch
// the long ones are: the parts are of equal length whatever the table's room.
// Every work-group computes the same cut from cache_len. The number of parts
// is at most `want` over the readers plus one for each item.
// A part has at least 128 positions (one tree of 15 nodes over 1021, 8 key heads: 64,
// 128, 256 and 512 give 16.6, 16.5, 18.2 and 22.5 us), and a table with room for twice
// that is not cut at all: the second launch costs more (200 positions 15.7 us in
// two parts, 12.6 in one).
constexpr int kAttnMinKeys = 128;

struct AttnPlan {
    int readers;   // work-groups that read one part
    int want;      // work-groups wanted
    int min_keys;  // smallest part
    int parts;     // upper bound of parts over all items
    bool split;    // whether an item may have more than one
    bool sorted;   // work-groups take the whole parts first, then the items' last ones by falling length
};

inline AttnPlan attn_plan(int batch, long long room, int readers, int min_keys, int want) {
    AttnPlan p;
    p.readers = readers;
    p.want = want;
    p.min_keys = min_keys;
    p.split = room > 2 * min_keys;
    p.sorted = false;
    p.parts = batch + (p.split ? want / readers : 0);
    return p;
}

// Partial results of a part, for each of the T * H rows: the unnormalised
// output, and the running maximum (base 2) and sum of the softmax; and the part's
// status bits.
struct AttnWorkspace {
    float* o;     // [parts][T * H][D]
    float* ml;    // [parts][T * H][2]
    int* bits;    // [parts]
};
inline uint64_t attn_workspace_bytes(const AttnPlan& p, int T, int H, int D) {
    if (!p.split) return 0;
    return (uint64_t)p.parts * (((uint64_t)T * H * (D + 2) + 1) + 3) / 4 * 4 * sizeof(float);
}
inline AttnWorkspace attn_workspace(void* ws, const AttnPlan& p, int T, int H, int D) {
    AttnWorkspace w;
    w.o = (float*)ws;
    w.ml = ws ? w.o + (size_t)p.parts * T * H * D : nullptr;
    w.bits = ws ? (int*)(w.ml + (size_t)p.parts * T * H * 2) : nullptr;
    return w;
}

__device__ __forceinline__ int usable_len(int len, int room) { return len < 0 || len > room ? 0 : len; }

__device__ __forceinline__ int part_keys(const AttnPlan& plan, unsigned long long sum) {
    const unsigned long long want = (sum * plan.readers + plan.want - 1) / plan.want;
    return max((int)min((want + 63) / 64 * 64, 0x7fffffc0ull), plan.min_keys);
}

struct Part {
    int ok;        // 0: no such part
    int item;
    int k, n;      // index among the item's n parts
    int base;      // the item's first part
    int len;       // usable cache length
    int bad_len;   // cache_len is out of range (its len is 0 then)
    int keys;      // positions per part
};

// The same in scalar registers
__device__ __forceinline__ Part uniform(const Part& p) {
    Part u;
#define TSV_U(f) u.f = __builtin_amdgcn_readfirstlane(p.f)
    TSV_U(ok);
    TSV_U(item);
    TSV_U(k);
    TSV_U(n);
    TSV_U(base);
    TSV_U(len);
    TSV_U(bad_len);
    TSV_U(keys);
#undef TSV_U
    return u;
}

// The part whose turn is `want` (or, with by_item, part 0 of item `want`), the same in all
// NT threads. May act as a barrier. s_red: NT / 64 + 2 ints,
// 8-byte aligned; s_out: one Part.
template <int NT>
__device__ __forceinline__ Part find_part(const int32_t* __restrict__ cache_len, int batch, int room, const AttnPlan& plan,
                                          int want, bool by_item, int* s_red, Part* s_out) {
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    if (batch <= kWave) {  // every wave by itself: one load, no barrier
        const int raw = lane < batch ? cache_len[lane] : 0, len = usable_len(raw, room);
        int keys = 0x7fffffc0;  // above any length
        if (plan.split) {
            unsigned long long sum = (unsigned)len;
#pragma unroll
            for (int m = 1; m < kWave; m <<= 1) sum += __shfl_xor(sum, m, kWave);
            keys = part_keys(plan, sum);
        }
        const int cnt = lane < batch ? max(1, (int)(((uint32_t)len + keys - 1) / keys)) : 0;
        const int first = plan.sorted && lane < batch ? cnt - 1 : cnt;  // the parts in the items' order
        int upto = first;
#pragma unroll
        for (int m = 1; m < kWave; m <<= 1) {
            const int o = __shfl_up(upto, m, kWave);
            if (lane >= m) upto += o;
        }
        const int turn = upto - first, base = plan.sorted ? turn + lane : turn;
        const int late = want - __builtin_amdgcn_readlane(upto, kWave - 1);  // place among the last parts
        bool mine = lane < batch && (by_item ? lane == want : want >= turn && want < upto);
        if (plan.sorted && !by_item && late >= 0) {
            const int rest = len - (cnt - 1) * keys;
            int rank = 0;
            for (int j = 0; j < batch; ++j) {
                const int other = __builtin_amdgcn_readlane(rest, j);
                rank += other > rest || (other == rest && j < lane);
            }
            mine = lane < batch && rank == late;
        }
        const unsigned long long who = __ballot(mine);
        Part p;
        p.ok = who != 0;
        const int src = who ? __builtin_ctzll(who) : 0;
        p.item = src;
        p.base = __builtin_amdgcn_readlane(base, src);
        p.n = __builtin_amdgcn_readlane(cnt, src);
        p.k = by_item ? 0 : plan.sorted && late >= 0 ? p.n - 1 : want - __builtin_amdgcn_readlane(turn, src);
        p.len = __builtin_amdgcn_readlane(len, src);
        p.bad_len = __builtin_amdgcn_readlane(raw, src) != p.len;
        p.keys = keys;
        return p;
    }
    if (tid == 0) {
        s_out->ok = 0;
        s_red[0] = s_red[1] = 0;
    }
    __syncthreads();
    int keys = 0x7fffffc0;  // above any length
    if (plan.split) {
        unsigned long long sum = 0;
        for (int b = tid; b < batch; b += NT) sum += usable_len(cache_len[b], room);
#pragma unroll
        for (int m = 1; m < kWave; m <<= 1) sum += __shfl_xor(sum, m, kWave);
        if (lane == 0) atomicAdd((unsigned long long*)s_red, sum);
        __syncthreads();
        sum = *(volatile unsigned long long*)s_red;
        keys = part_keys(plan, sum);
        __syncthreads();
    }
    int run = 0;
    for (int b0 = 0; b0 < batch; b0 += NT) {
        const int b = b0 + tid;
        const int raw = b < batch ? cache_len[b] : 0;
        const int len = usable_len(raw, room);
        const int cnt = b < batch ? max(1, (int)(((uint32_t)len + keys - 1) / keys)) : 0;
        int total;
        const int base = run + block_exclusive_scan<NT>(cnt, s_red, &total);
        if (b < batch && (by_item ? b == want : want >= base && want < base + cnt)) {
            s_out->item = b;
            s_out->k = by_item ? 0 : want - base;
            s_out->n = cnt;
            s_out->base = base;
            s_out->len = len;
            s_out->bad_len = raw != len;
            s_out->keys = keys;
            s_out->ok = 1;
        }
        run += total;
    }
    __syncthreads();
    return *s_out;
}

// bf16 MFMA kernels (attn_mfma.hip): block_rows 16, 64 or 128 rows of a key head
// per work-group
void launch_attn_mfma(const AttnArgs& a, bool e4m3, const AttnPlan& p, const AttnWorkspace& ws, int block_rows, int row_blocks,
                      hipStream_t stream);

// fp32 MFMA kernel (attn_f32.hip): block_rows 16 or 64
void launch_attn_f32(const AttnArgs& a, bool e4m3, const AttnPlan& p, const AttnWorkspace& ws, int block_rows, int row_blocks,
                     hipStream_t stream);

// Status bits of the tree, and each of `rows` rows' ancestors as bit words
// (row i is node first + i); s_par: T ints. Acts as a barrier.
template <int NT>
__device__ __forceinline__ int tree_words(const int32_t* __restrict__ parent, int T, int first, int rows, int words, int* s_par, uint32_t* s_anc) {
    int bits = 0;
    for (int i = threadIdx.x; i < T; i += NT) {
        const int p = parent[i];
        s_par[i] = p;
        bits |= i == 0 ? (p != -1 ? kStBadRoot : 0) : (p < 0 || p >= i ? kStBadParent : 0);
    }
    for (int i = threadIdx.x; i < rows * words; i += NT) s_anc[i] = 0;
    const int any = __syncthreads_or(bits);
    if (any) return (__syncthreads_or(bits & kStBadRoot) ? kStBadRoot : 0) | (__syncthreads_or(bits & kStBadParent) ? kStBadParent : 0);
    for (int i = threadIdx.x; i < rows; i += NT)
        for (int j = first + i; j >= 0; j = s_par[j]) s_anc[i * words + j / 32] |= 1u << (j % 32);
    __syncthreads();
    return 0;
}

__device__ __forceinline__ float e4m3_ld(const uint8_t* p) { return __builtin_amdgcn_cvt_f32_fp8((int)*p, 0); }

}  // namespace tsv
