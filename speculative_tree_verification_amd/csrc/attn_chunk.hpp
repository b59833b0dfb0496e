// attn_chunk.hpp -- how the attention of packed rows over the paged cache
// (tree_attn_prefill) is cut into work-groups.
//
// A sequence of n new tokens has n g rows (token, query head) for each key head, g = H /
// Hk, and `rows` of them make a block. A block's keys are the positions that some row of it
// sees: without a window all up to its last token; with one the first `sinks`, and those
// from its first token's window on. They are numbered through ("virtual" positions), so
// that a kernel has one loop over them. Blocks whose keys would keep a few work-groups busy
// long after the others are cut into parts of equal length, which a second launch joins:
// `keys` positions a part at most, by the lengths on the device, so that blocks and parts
// together make about `want` work-groups. A sequence's blocks have the same number of
// parts, by its longest; the last ones, which see the most, come first.
#pragma once

#include "attn_common.hpp"

namespace tsv {

struct ChunkPlan {
    int rows;      // rows of a block, a power of two
    int shift;     // its logarithm
    int g;         // rows of a token
    int tokens;    // most of a block
    PageDiv by_g;  // n / g
    float share;   // above Hk / want, by more than the sum of the work is rounded
    int want;      // work-groups wanted
    int min_keys;  // smallest part
    bool split;    // whether a block may have more than one part
    bool sorted;   // the sequences' units by falling length (of at most 64 sequences)
};

// Upper bounds over all lengths. A cut block has parts of more than half of `keys`, and
// sum(blocks longest) Hk <= want keys.
inline long long chunk_blocks(const ChunkPlan& p, long long T, int g, int batch) { return T * g / p.rows + (batch < T ? batch : T); }
inline long long chunk_units(const ChunkPlan& p, long long T, int g, int batch, int Hk) {
    return chunk_blocks(p, T, g, batch) + (p.split ? p.want / Hk : 0);
}
inline long long chunk_slots(const ChunkPlan& p, int Hk) { return p.split ? 2LL * p.want / Hk : 0; }

// Partial results of a part for one key head: the rows' unnormalised outputs, running
// maxima (base 2) and sums
// (and whether the sequence is left out)
struct ChunkWorkspace {
    float* o;   // [slots][Hk][rows][D]
    float* ml;  // [slots][Hk][rows][2]
    int* bad;   // [slots][Hk]
};
inline uint64_t chunk_workspace_bytes(const ChunkPlan& p, int Hk, int D) {
    return (uint64_t)chunk_slots(p, Hk) * Hk * ((uint64_t)p.rows * (D + 2) + 1) * sizeof(float);
}
inline ChunkWorkspace chunk_workspace(void* ws, const ChunkPlan& p, int Hk, int D) {
    ChunkWorkspace w;
    const size_t n = (size_t)chunk_slots(p, Hk) * Hk;
    w.o = (float*)ws;
    w.ml = ws ? w.o + n * p.rows * D : nullptr;
    w.bad = ws ? (int*)(w.ml + n * p.rows * 2) : nullptr;
    return w;
}

struct ChunkUnit {
    int ok;            // 0: no such block or part
    int seq;
    int start, n;      // its packed rows
    int old;           // its filled positions
    int block, part, parts;
    int slot;          // of this part (join: of the block's part 0), where parts > 1
    int lead;          // the sequence's first unit
    int bad;           // the packing is none
};

// What one sequence asks for
struct ChunkSeq {
    int start, n, old;
    int bad;       // of the packing
    int fits;      // in its pages
    int blocks;    // 0 where it does not fit
    int longest;   // keys of its longest block, at most
};
__device__ __forceinline__ ChunkSeq chunk_seq(const ChunkArgs& a, const ChunkPlan& plan, int q) {
    ChunkSeq s{};
    s.fits = 1;
    if (q >= a.batch) return s;
    int lo = a.seq_start[q], hi = a.seq_start[q + 1];
    s.old = a.cache_len[q];
    if (lo < 0 || hi < lo || hi > a.T) {
        s.bad = 1;
        hi = lo;
    }
    s.start = lo;
    s.n = hi - lo;
    s.fits = s.old >= 0 && s.old <= a.room && s.n <= a.room - s.old;
    if (!s.fits || s.n == 0) return s;
    s.blocks = (s.n * plan.g + plan.rows - 1) >> plan.shift;
    s.longest = (int)min((long long)s.old + s.n, (long long)a.window + min(s.n, plan.tokens) - 1 + a.sinks);
    return s;
}

// Sums over the lanes up to this one
template <typename T>
__device__ __forceinline__ T lanes_before(T v) {
    static_assert(sizeof(T) == 4, "a word of a lane");
#define TSV_ADD_DPP(ctrl, rows) v += __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), ctrl, rows, 0xf, false))
    TSV_ADD_DPP(0x111, 0xf);  // row_shr:1, of 16 lanes
    TSV_ADD_DPP(0x112, 0xf);
    TSV_ADD_DPP(0x114, 0xf);
    TSV_ADD_DPP(0x118, 0xf);
    TSV_ADD_DPP(0x142, 0xa);  // row_bcast:15, into the second and fourth row
    TSV_ADD_DPP(0x143, 0xc);  // row_bcast:31, into the upper half
#undef TSV_ADD_DPP
    return v;
}

// The unit whose turn is `want`, or with JOIN the cut block whose turn it is. The same in
// all lanes of a wave; no barrier.
template <bool JOIN>
__device__ __forceinline__ ChunkUnit find_unit(const ChunkArgs& a, const ChunkPlan& plan, int want) {
    const int lane = threadIdx.x & (kWave - 1);
    ChunkSeq s = chunk_seq(a, plan, lane);
    unsigned long long work = (unsigned long long)s.blocks * s.longest;
    int bad = s.bad;
    for (int q0 = kWave; q0 < a.batch; q0 += kWave) {
        const ChunkSeq t = chunk_seq(a, plan, q0 + lane);
        work += (unsigned long long)t.blocks * t.longest;
        bad |= t.bad;
    }
    ChunkUnit u{};
    u.bad = __ballot(bad) != 0;
    if (u.bad) return u;
    int keys = 0x7fffffc0;  // above any length
    if (plan.split) {
        // (rounded to 24 bits once and in six sums: `share` has 2^-20 more)
        const int total = __builtin_amdgcn_readlane(__float_as_int(lanes_before((float)work)), kWave - 1);
        const int per = (int)fminf(__int_as_float(total) * plan.share + 1.f, 2147483520.f);
        keys = max((per + 63) / 64 * 64, plan.min_keys);
    }
    int run = 0, slots = 0;
    for (int q0 = 0; q0 < a.batch; q0 += kWave) {
        if (q0) s = chunk_seq(a, plan, q0 + lane);
        const int parts = s.blocks ? (int)(((uint32_t)s.longest + keys - 1) / keys) : 0;
        const int cut = parts > 1 ? s.blocks * parts : 0, cnt = JOIN ? (parts > 1 ? s.blocks : 0) : s.blocks * parts;
        const int upto = lanes_before(cnt), cuts = lanes_before(cut);
        const int at = want - run;
        int from = upto - cnt;
        if (!JOIN && plan.sorted) {
            from = 0;
            for (int j = 0; j < a.batch; ++j) {
                const int other = __builtin_amdgcn_readlane(s.longest, j);
                if (other > s.longest || (other == s.longest && j < lane)) from += __builtin_amdgcn_readlane(cnt, j);
            }
        }
        const unsigned long long who = __ballot(at >= from && at < from + cnt);
        if (who) {
            const int src = __builtin_ctzll(who);
            const int turn = at - __builtin_amdgcn_readlane(from, src);
            u.ok = 1;
            u.seq = q0 + src;
            u.start = __builtin_amdgcn_readlane(s.start, src);
            u.n = __builtin_amdgcn_readlane(s.n, src);
            u.old = __builtin_amdgcn_readlane(s.old, src);
            u.parts = __builtin_amdgcn_readlane(parts, src);
            const int blocks = __builtin_amdgcn_readlane(s.blocks, src);
            const int done = JOIN || u.parts == 1 ? turn : turn / u.parts;
            u.block = blocks - 1 - done;
            u.part = JOIN ? 0 : turn - done * u.parts;
            u.slot = slots + __builtin_amdgcn_readlane(cuts - cut, src) + (JOIN ? turn * u.parts : turn);
            u.lead = turn == 0;
            return u;
        }
        run += __builtin_amdgcn_readlane(upto, kWave - 1);
        slots += __builtin_amdgcn_readlane(cuts, kWave - 1);
    }
    return u;
}

// The keys of a block: positions [0, sinks) and [lo, hi), `keys` of them
struct ChunkKeys {
    int sinks, lo, keys;
    int k0, k1;  // this part's virtual positions
};
__device__ __forceinline__ ChunkKeys chunk_keys(const ChunkArgs& a, const ChunkPlan& plan, const ChunkUnit& u) {
    const int row0 = u.block * plan.rows, row1 = min(u.n * plan.g, row0 + plan.rows) - 1;
    ChunkKeys k;
    const int hi = u.old + page_of(row1, plan.by_g) + 1;
    k.lo = (int)max(0LL, (long long)u.old + page_of(row0, plan.by_g) - a.window + 1);
    k.sinks = min(a.sinks, k.lo);
    k.keys = k.sinks + hi - k.lo;
    const int per = u.parts == 1 ? k.keys : ((k.keys + u.parts - 1) / u.parts + 63) / 64 * 64;
    k.k0 = (int)min((long long)u.part * per, (long long)k.keys);
    k.k1 = (int)min((long long)k.k0 + per, (long long)k.keys);
    return k;
}
// Position of virtual position v
__device__ __forceinline__ int chunk_pos(const ChunkKeys& k, int v) { return v < k.sinks ? v : v - k.sinks + k.lo; }

// The virtual positions v that the row at position `own` sees: v < hi and (v >= lo or v < a.sinks).
// (The sinks' own, below k.sinks, all rows see, and a.sinks is k.sinks unless the sinks go on
// behind k.lo, where virtual positions are positions.)
struct ChunkSeen {
    int lo, hi;
};
__device__ __forceinline__ ChunkSeen chunk_seen(const ChunkArgs& a, const ChunkKeys& k, int own) {
    ChunkSeen s;
    s.lo = max(0, own - a.window + 1 - k.lo + k.sinks);
    s.hi = min(k.k1, own - k.lo + k.sinks + 1);
    return s;
}

// Whether some page that the sequence's rows use is none of the pool's: threads of a
// work-group of NT look at different ones.
template <int NT>
__device__ __forceinline__ bool chunk_pages_bad(const ChunkArgs& a, const ChunkUnit& u) {
    const int32_t* table = a.page_table + (size_t)u.seq * a.max_pages;
    const int lo = (int)max(0LL, (long long)u.old - a.window + 1), sinks = min(a.sinks, lo);
    bool bad = false;
    if (sinks > 0)
        for (int i = threadIdx.x; i <= page_of(sinks - 1, a.div); i += NT) bad |= (uint32_t)table[i] >= (uint32_t)a.n_pages;
    const int last = page_of(u.old + u.n - 1, a.div);
    for (int i = page_of(lo, a.div) + (int)threadIdx.x; i <= last; i += NT) bad |= (uint32_t)table[i] >= (uint32_t)a.n_pages;
    return bad;
}

// The pages' check of a work-group, its status and its word for the join: whether to leave
// the sequence out, the same in all threads. A barrier.
template <int NT>
__device__ __forceinline__ bool chunk_check(const ChunkArgs& a, const ChunkUnit& u, int hk, const ChunkWorkspace& ws) {
    const int bad = __syncthreads_or(chunk_pages_bad<NT>(a, u));
    if (threadIdx.x == 0) {
        if (u.lead && hk == 0 && a.status) a.status[u.seq] = bad ? kStBadCache : 0;
        if (u.parts > 1) ws.bad[(size_t)u.slot * a.Hk + hk] = bad;
    }
    return bad;
}

// Status of the sequences that have no unit (empty, or too long for their pages), and of
// all where the packing is none: one wave of a launch
__device__ __forceinline__ void chunk_status(const ChunkArgs& a, const ChunkPlan& plan, bool bad) {
    if (!a.status) return;
    for (int q = threadIdx.x & (kWave - 1); q < a.batch; q += kWave) {
        const ChunkSeq s = chunk_seq(a, plan, q);
        if (bad)
            a.status[q] = kStBadSeqRows;
        else if (s.blocks == 0)
            a.status[q] = s.fits ? 0 : kStBadCache;
    }
}

// bf16 MFMA kernels (attn_chunk_mfma.hip): plan.rows 16 or 128
void launch_chunk_mfma(const ChunkArgs& a, bool e4m3, const ChunkPlan& p, const ChunkWorkspace& ws, dim3 grid, hipStream_t stream);

// fp32 MFMA kernels (attn_chunk_f32.hip): plan.rows 16 or 64
void launch_chunk_f32(const ChunkArgs& a, bool e4m3, const ChunkPlan& p, const ChunkWorkspace& ws, dim3 grid, hipStream_t stream);

}  // namespace tsv
