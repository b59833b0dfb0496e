// attn_cache.hpp -- what the writes into the paged cache share: a row's pieces, their
// storage (as they are or in 8 bits), the check of an item's pages, and the places of
// packed rows.
#pragma once

#include "attn_common.hpp"

namespace tsv {

struct Quad {
    float v[8];
};

// A row's piece as it is loaded
template <typename TIO, bool VEC>
struct Raw {
    TIO e[8];
};
template <>
struct Raw<uint16_t, true> {
    uint4 u;
};
template <>
struct Raw<float, true> {
    float4 a, b;
};

template <typename TIO, bool VEC>
__device__ __forceinline__ Raw<TIO, VEC> load8(const TIO* p, int rem) {
    Raw<TIO, VEC> q;
    if constexpr (!VEC) {
#pragma unroll
        for (int i = 0; i < 8; ++i) q.e[i] = i < rem ? gload(p + i) : TIO(0);
    } else if constexpr (sizeof(TIO) == 2) {
        q.u = gload((const uint4*)p);
    } else {
        q.a = gload((const float4*)p);
        q.b = gload((const float4*)p + 1);
    }
    return q;
}

template <typename TIO, bool VEC>
__device__ __forceinline__ Quad floats(const Raw<TIO, VEC>& r) {
    Quad q;
    if constexpr (!VEC) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (sizeof(TIO) == 2)
                q.v[i] = bf16_bits_to_f32(r.e[i]);
            else
                q.v[i] = r.e[i];
        }
    } else if constexpr (sizeof(TIO) == 2) {
        const uint32_t wd[4] = {r.u.x, r.u.y, r.u.z, r.u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            q.v[2 * i] = __uint_as_float(wd[i] << 16);
            q.v[2 * i + 1] = __uint_as_float(wd[i] & 0xffff0000u);
        }
    } else {
        q.v[0] = r.a.x; q.v[1] = r.a.y; q.v[2] = r.a.z; q.v[3] = r.a.w;
        q.v[4] = r.b.x; q.v[5] = r.b.y; q.v[6] = r.b.z; q.v[7] = r.b.w;
    }
    return q;
}

// The scale of a row whose largest magnitude has the bits `top` (magnitudes compare as
// their bits do; an infinity or a NaN is above all): NaN for a row that is not finite
__device__ __forceinline__ float scale_of(uint32_t top) {
    return top < 0x7f800000u ? fmaxf(__uint_as_float(top) / 448.f, 1.17549435e-38f) : __uint_as_float(0x7fc00000u);
}

// Eight values of a row as e4m3 bytes, each v / scale to the nearest float from the
// nearest reciprocal: a product, its exact remainder, and one correction (Markstein) give
// the quotient that the division instruction sequence gives, in a quarter of the
// operations (the divisions were the bound: 44.9 us for 16378 rows of 8 heads, then 33
// us). The remainder is formed negated, so that an exact 0 in the correction has the
// quotient's sign: -0 stays -0. Below 2^-100 it may leave the floats' range.
__device__ __forceinline__ uint2 e4m3_bytes(const Quad& q, float scale, bool finite) {
    float t[8];
    if (scale >= 7.8886090522e-31f || !finite) {
        const float r = 1.f / scale;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q0 = q.v[i] * r;
            t[i] = fmaf(-fmaf(q0, scale, -q.v[i]), r, q0);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = q.v[i] / scale;
    }
    uint32_t wd[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int p = __builtin_amdgcn_cvt_pk_fp8_f32(t[4 * i], t[4 * i + 1], 0, false);
        p = __builtin_amdgcn_cvt_pk_fp8_f32(t[4 * i + 2], t[4 * i + 3], p, true);
        wd[i] = finite ? (uint32_t)p : 0x7f7f7f7fu;
    }
    return make_uint2(wd[0], wd[1]);
}

// The cache's element: TIO, or a byte with a scale (E4M3)
template <typename TIO, bool E4M3, bool VEC>
__device__ __forceinline__ void store8(const CacheWriteArgs& a, bool value, size_t at, int d, int rem, const Quad& q,
                                       float scale, bool finite) {
    if (E4M3) {
        const uint2 u = e4m3_bytes(q, scale, finite);
        const uint32_t wd[2] = {u.x, u.y};
        uint8_t* o = (uint8_t*)(value ? a.v_cache : a.k_cache) + at * a.D + d;
        if (VEC) {
            gstore((uint2*)o, make_uint2(wd[0], wd[1]));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < rem) o[i] = (uint8_t)(wd[i / 4] >> (8 * (i % 4)));
        }
        if (d == 0) (value ? a.v_scale : a.k_scale)[at] = scale;
    } else {
        TIO* o = (TIO*)(value ? a.v_cache : a.k_cache) + at * a.D + d;
        if (VEC) {
            if (sizeof(TIO) == 2) {
                // bf16 values: the upper halves are exact
                gstore((uint4*)o, make_uint4(__float_as_uint(q.v[0]) >> 16 | (__float_as_uint(q.v[1]) & 0xffff0000u),
                                             __float_as_uint(q.v[2]) >> 16 | (__float_as_uint(q.v[3]) & 0xffff0000u),
                                             __float_as_uint(q.v[4]) >> 16 | (__float_as_uint(q.v[5]) & 0xffff0000u),
                                             __float_as_uint(q.v[6]) >> 16 | (__float_as_uint(q.v[7]) & 0xffff0000u)));
            } else {
                gstore((float4*)o, make_float4(q.v[0], q.v[1], q.v[2], q.v[3]));
                gstore((float4*)o + 1, make_float4(q.v[4], q.v[5], q.v[6], q.v[7]));
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < rem) {
                    if (sizeof(TIO) == 2)
                        ((uint16_t*)o)[i] = (uint16_t)(__float_as_uint(q.v[i]) >> 16);
                    else
                        ((float*)o)[i] = q.v[i];
                }
        }
    }
}

// Pages of `count` rows at cache_len[b] = len: false if they do not fit
__device__ __forceinline__ bool page_range(const CacheWriteArgs& a, int len, int count, int* first, int* last) {
    const int room = a.max_pages * a.page_size;
    *first = 0;
    *last = -1;
    if (len < 0 || count < 0 || len > room || count > room - len) return false;
    if (count > 0) {
        *first = page_of(len, a.div);
        *last = page_of(len + count - 1, a.div);
    }
    return true;
}
__device__ __forceinline__ bool pages_bad(const CacheWriteArgs& a, int b, int first, int last, int step) {
    bool bad = false;
    for (int i = first; i <= last; i += step) {
        const int pg = a.page_table[(size_t)b * a.max_pages + i];
        bad |= pg < 0 || pg >= a.n_pages;
    }
    return bad;
}

// Status bits of writing `count` rows at cache_len[b]: the same in all threads.
// Acts as a barrier.
__device__ __forceinline__ int check_pages(const CacheWriteArgs& a, int b, int count) {
    int first, last;
    bool bad = !page_range(a, a.cache_len[b], count, &first, &last);
    bad |= pages_bad(a, b, first + threadIdx.x, last, blockDim.x);
    return __syncthreads_or(bad) ? kStBadCache : 0;
}

// Row of head 0 in the cache's arrays for position `pos` of item b (its page is checked)
__device__ __forceinline__ long long cache_place(const CacheWriteArgs& a, int b, int pos) {
    const int page = page_of(pos, a.div), pg = a.page_table[(size_t)b * a.max_pages + page];
    return (long long)pg * a.Hk * a.page_size + (pos - page * a.page_size);
}

// Largest value of each N <= 16 neighbouring lanes, in all of them
template <int N>
__device__ __forceinline__ uint32_t max_of(uint32_t v) {
#define TSV_MAX_DPP(ctrl) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, 0xf, 0xf, true))
    if (N >= 2) TSV_MAX_DPP(0xb1);    // quad_perm [1,0,3,2]
    if (N >= 4) TSV_MAX_DPP(0x4e);    // quad_perm [2,3,0,1]
    if (N >= 8) TSV_MAX_DPP(0x141);   // row_half_mirror
    if (N >= 16) TSV_MAX_DPP(0x140);  // row_mirror
#undef TSV_MAX_DPP
    return v;
}

// Places of ROWS packed rows from r0 on, of which n are rows of the call: `place` is the
// row's position in its sequence's cache, `dst` that position's row of head 0 in the
// cache's arrays (both -1 for a row of no sequence, or of one with a status bit). A
// sequence's pages are checked as a whole, so that one with a status bit is left whole.
template <int ROWS>
struct RowPlaces {
    long long dst[ROWS];
    int place[ROWS];
    // of the rows with which a sequence begins or goes on here: bits of `leads`
    int item[ROWS], pos[ROWS], len[ROWS], count[ROWS], bad[ROWS], is_long[ROWS];
    uint32_t leads;
    int red[4];
};

// False: nothing to write for this work-group. With status_of >= 0 it writes the status of
// that item instead. 256 threads; acts as a barrier (of LDS alone on the common path, so
// that loads from before it stay in flight).
template <int ROWS>
__device__ __forceinline__ bool find_places(const CacheWriteArgs& a, int r0, int n, int status_of, RowPlaces<ROWS>& s) {
    static_assert(ROWS <= 32, "a bit for each row");
    const int tid = threadIdx.x;
    if (tid < ROWS) s.bad[tid] = s.is_long[tid] = 0;
    if (tid == 0) s.leads = 0;
    lds_barrier();
    // the thread of a sequence that has rows here writes what they need of it
    int bad = 0;
    for (int q = tid; q < a.batch; q += 256) {
        const int lo = a.seq_start[q], hi = a.seq_start[q + 1], len = a.cache_len[q], r = max(lo, r0);
        bad |= lo < 0 || hi < lo || hi > a.T;
        if (r < min(hi, r0 + n)) {
            s.item[r - r0] = q;
            s.pos[r - r0] = r - lo;
            s.len[r - r0] = len;
            s.count[r - r0] = hi - lo;
            atomicOr(&s.leads, 1u << (r - r0));
        }
    }
    bad = lds_sync_or<256>(bad, s.red);
    if (status_of >= 0) {
        const int b = status_of;
        const int st = bad ? kStBadSeqRows : check_pages(a, b, a.seq_start[b + 1] - a.seq_start[b]);
        if (tid == 0) a.status[b] = st;
        return false;
    }
    if (bad) return false;
    // a row's page, where its sequence fits the table
    int lead = 0, page = 0, place = -1, pg = 0, first, last;
    if (const uint32_t before = tid < n ? s.leads & ((2u << tid) - 1) : 0) {
        lead = 31 - __builtin_clz(before);
        const int at = s.pos[lead] + tid - lead;
        if (at < s.count[lead] && page_range(a, s.len[lead], s.count[lead], &first, &last)) {
            place = s.len[lead] + at;
            page = page_of(place, a.div);
            pg = a.page_table[(size_t)s.item[lead] * a.max_pages + page];
        }
    }
    // the sequences that begin or go on in these rows: 16 threads each, all at once
    // (16 short prompts one after another took 30 us), and then all threads for
    // each of the few that have many pages
    {
        constexpr int kLong = 64;
        const int i = tid / (256 / ROWS);
        if (s.leads >> i & 1) {
            if (!page_range(a, s.len[i], s.count[i], &first, &last))
                s.bad[i] = 1;
            else if (last - first >= kLong)
                s.is_long[i] = 1;
            else if (pages_bad(a, s.item[i], first + tid % (256 / ROWS), last, 256 / ROWS))
                s.bad[i] = 1;
        }
        lds_barrier();
        for (int j = 0; j < n; ++j) {
            if (!s.is_long[j]) continue;
            const int st = check_pages(a, s.item[j], s.count[j]);
            if (tid == 0 && st) s.bad[j] = 1;
            __syncthreads();
        }
    }
    if (tid < n) {
        if (s.bad[lead]) place = -1;
        s.place[tid] = place;
        s.dst[tid] = place >= 0 ? (long long)pg * a.Hk * a.page_size + (place - page * a.page_size) : -1;
    }
    lds_barrier();
    return true;
}

}  // namespace tsv
