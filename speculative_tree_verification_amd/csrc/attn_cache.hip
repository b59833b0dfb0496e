// attn_cache.hip -- rows of keys and values into the paged cache: the accepted
// path of each item (tree_attn_commit) or packed prompts (tree_attn_append),
// as they are or in 8 bits.
//
//   position p of item b is row p % page_size of page table[b][p / page_size];
//   e4m3: scale = max(max|row| / 448, 2^-126), byte = row / scale to even.
//
// Bound by the rows' traffic (in: Hk D elements of k and of v each, out: the
// same in the cache's type). A row of one head is held by LPR lanes with 8
// elements each: one 16-byte load (bf16), a butterfly over the lanes for the
// largest value, one store of 8 bytes (e4m3) or 16. The division is a true one,
// so that the stored byte is the nearest to row / scale. A work-group first
// checks everything that its rows' items need (path, lengths, pages), so that
// an item with a status bit is left whole; in append the rows are on their way
// meanwhile. 16 prompts, 16378 rows of 8 heads of 128 into e4m3 (102 MB): 30 us,
// 3.4 TB/s, half of it the vector work (fetching after the search 31.6 us against
// 30.0, the butterfly through LDS 30.0 against 29.0).
#include "attn_common.hpp"

namespace tsv {
namespace {

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

// The cache's element: TIO, or a byte with a scale (E4M3)
template <typename TIO, bool E4M3, bool VEC>
__device__ __forceinline__ void store8(const CacheWriteArgs& a, bool value, size_t at, int d, int rem, const Quad& q,
                                       float scale, bool finite) {
    if (E4M3) {
        // v / scale to the nearest float from the nearest reciprocal: a product, its
        // exact remainder, and one correction (Markstein) give the quotient that the
        // division instruction sequence gives, in a quarter of the operations (the
        // divisions were the bound: 44.9 us for 16378 rows of 8 heads, then 33 us).
        // The remainder is formed negated, so that an exact 0 in the correction has
        // the quotient's sign: -0 stays -0. Below 2^-100 it may leave the floats' range.
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

// n rows, keys and values of all heads, LPR lanes a row of a head, 256 / LPR such
// rows, heads fastest, in a step; `fetch` loads a thread's pieces of K steps from
// u0 on (source row src(row); negative: none), `flush` writes them to s_dst (-1:
// not written).
template <typename TIO, int LPR, bool VEC, int K, class Src>
__device__ __forceinline__ void fetch(const CacheWriteArgs& a, int n, int u0, Src src, Raw<TIO, VEC> (&q)[K]) {
    const int d = threadIdx.x % LPR * 8, rem = a.D - d;
#pragma unroll
    for (int x = 0; x < K; ++x) {
        const int u = u0 + x * (256 / LPR);
        const bool in = u < n * a.Hk * 2;
        const int row = in ? page_of(u, a.heads) : 0, hv = in ? u - row * 2 * a.Hk : 0;
        const bool value = hv >= a.Hk;
        const long long r = in && rem > 0 ? src(row) : -1;
        q[x] = Raw<TIO, VEC>{};
        if (r >= 0) q[x] = load8<TIO, VEC>((const TIO*)(value ? a.v : a.k) + ((size_t)r * a.Hk + (value ? hv - a.Hk : hv)) * a.D + d, rem);
    }
}
template <typename TIO, int LPR, bool E4M3, bool VEC, int K>
__device__ __forceinline__ void flush(const CacheWriteArgs& a, int n, int u0, const long long* s_dst, const Raw<TIO, VEC> (&q)[K]) {
    const int d = threadIdx.x % LPR * 8, rem = a.D - d;
#pragma unroll
    for (int x = 0; x < K; ++x) {
        const int u = u0 + x * (256 / LPR);
        const bool in = u < n * a.Hk * 2;
        const int row = in ? page_of(u, a.heads) : 0, hv = in ? u - row * 2 * a.Hk : 0;
        const bool value = hv >= a.Hk;
        const long long at = in && rem > 0 ? s_dst[row] : -1;
        const Quad f = floats<TIO, VEC>(q[x]);
        float scale = 1.f;
        bool finite = true;
        if (E4M3) {
            // magnitudes compare as their bits do; an infinity or a NaN is above all
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(f.v[i]) & 0x7fffffffu);
#pragma unroll
            for (int m = 16; m < LPR; m <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, m, kWave));
            top = max_of<LPR < 16 ? LPR : 16>(top);
            finite = top < 0x7f800000u;
            scale = finite ? fmaxf(__uint_as_float(top) / 448.f, 1.17549435e-38f) : __uint_as_float(0x7fc00000u);
        }
        if (at >= 0)
            store8<TIO, E4M3, VEC>(a, value, (size_t)(at + (long long)(value ? hv - a.Hk : hv) * a.page_size), d, rem, f, scale, finite);
    }
}

// rows of a work-group: prompts have many; an accepted path has few, and its
// latency is what counts (32 paths of 7 nodes: 16 rows 11.9 us, 2 rows 6.0 us)
constexpr int kRows = 16, kPathRows = 2;

template <typename TIO, int LPR, bool E4M3, bool VEC>
__global__ __launch_bounds__(256) void append_kernel(CacheWriteArgs a, int row_blocks) {
    __shared__ long long s_dst[kRows];
    __shared__ int s_item[kRows], s_pos[kRows], s_place[kRows], s_bad[kRows], s_long[kRows], s_first, s_red[4];
    const int tid = threadIdx.x;
    // the packing, and the sequence of this block's first row: the sequences
    // that end at or before it
    const int r0 = blockIdx.x * kRows;
    const bool rows = (int)blockIdx.x < row_blocks;
    const int n = rows ? min(kRows, a.T - r0) : 0;
    // the rows are on their way while their places are found
    constexpr int K = VEC && sizeof(TIO) == 2 ? 8 : 4, kStep = K * (256 / LPR);
    Raw<TIO, VEC> q[K];
    const auto src = [&](int row) { return (long long)r0 + row; };
    fetch<TIO, LPR, VEC>(a, n, tid / LPR, src, q);
    if (tid == 0) s_first = 0;
    lds_barrier();
    int bad = 0, before = 0;
    for (int q = tid; q < a.batch; q += 256) {
        const int lo = a.seq_start[q], hi = a.seq_start[q + 1];
        bad |= lo < 0 || hi < lo || hi > a.T;
        before += hi <= r0;
    }
    if (before) atomicAdd(&s_first, before);
    bad = lds_sync_or<256>(bad, s_red);
    if (!rows) {  // a block for each item's status
        const int b = blockIdx.x - row_blocks;
        const int st = bad ? kStBadSeqRows : check_pages(a, b, a.seq_start[b + 1] - a.seq_start[b]);
        if (tid == 0) a.status[b] = st;
        return;
    }
    if (bad) return;
    if (tid < kRows) {
        int b = s_first, pos = -1;
        const int r = r0 + tid;
        while (b < a.batch && a.seq_start[b + 1] <= r) ++b;
        if (tid < n && b < a.batch && r >= a.seq_start[b]) pos = r - a.seq_start[b];  // in its sequence
        s_item[tid] = b < a.batch ? b : 0;
        s_pos[tid] = pos;
    }
    if (tid < kRows) s_bad[tid] = s_long[tid] = 0;
    lds_barrier();
    // the sequences that begin or go on in these rows: 16 threads each, all at once
    // (16 short prompts one after another took 30 us), and then all threads for
    // each of the few that have many pages
    {
        constexpr int kLong = 64;
        const int i = tid / (256 / kRows), b = s_item[i];
        const bool leads = i < n && s_pos[i] >= 0 && (i == 0 || s_pos[i - 1] < 0 || s_item[i - 1] != b);
        if (leads) {
            const int len = a.cache_len[b];
            int first, last;
            const bool fits = page_range(a, len, a.seq_start[b + 1] - a.seq_start[b], &first, &last);
            if (!fits)
                s_bad[i] = 1;
            else if (last - first >= kLong)
                s_long[i] = 1;
            else if (pages_bad(a, b, first + tid % (256 / kRows), last, 256 / kRows))
                s_bad[i] = 1;
        }
        lds_barrier();
        for (int j = 0; j < n; ++j) {
            if (!s_long[j]) continue;
            const int st = check_pages(a, s_item[j], a.seq_start[s_item[j] + 1] - a.seq_start[s_item[j]]);
            if (tid == 0 && st) s_bad[j] = 1;
            __syncthreads();
        }
    }
    if (tid < n && s_pos[tid] >= 0) {
        int j = tid;  // the first of this sequence's rows here
        while (j > 0 && s_item[j - 1] == s_item[tid] && s_pos[j - 1] >= 0) --j;
        s_place[tid] = s_bad[j] ? -1 : s_pos[tid] + a.cache_len[s_item[tid]];
    } else if (tid < n) {
        s_place[tid] = -1;
    }
    if (tid < n) s_dst[tid] = s_place[tid] >= 0 ? cache_place(a, s_item[tid], s_place[tid]) : -1;
    lds_barrier();
    for (int u0 = tid / LPR; u0 - tid / LPR < n * a.Hk * 2; u0 += kStep) {
        if (u0 != tid / LPR) fetch<TIO, LPR, VEC>(a, n, u0, src, q);
        flush<TIO, LPR, E4M3, VEC>(a, n, u0, s_dst, q);
    }
}

template <typename TIO, int LPR, bool E4M3, bool VEC>
__global__ __launch_bounds__(256) void commit_kernel(CacheWriteArgs a, int chunks) {
    __shared__ long long s_src[kPathRows], s_dst[kPathRows];
    const int tid = threadIdx.x, b = blockIdx.x / chunks, c = blockIdx.x % chunks;
    const int32_t* par = a.parent + (size_t)b * a.T;
    int bits = 0;
    for (int i = tid; i < a.T; i += 256) {
        const int p = par[i];
        bits |= i == 0 ? (p != -1 ? kStBadRoot : 0) : (p < 0 || p >= i ? kStBadParent : 0);
    }
    const int len = a.accepted_len[b];
    const bool fits = len >= 0 && len <= a.Lmax && len <= a.T;
    if (!fits) bits |= kStBadPath;
    const int32_t* acc = a.accepted + (size_t)b * a.Lmax;
    for (int i = tid; fits && i < len; i += 256) {
        const int node = acc[i];
        const int want = i == 0 ? -1 : acc[i - 1];
        if (node < 0 || node >= a.T || (i == 0 ? node != 0 : par[node] != want)) bits |= kStBadPath;
    }
    int st = check_pages(a, b, fits ? len : 0);
    if (__syncthreads_or(bits))  // one barrier on the common path; more tell the errors apart
        for (int bit = 1; bit <= kStBadPath; bit <<= 1) st |= __syncthreads_or(bits & bit) ? bit : 0;
    if (c == 0 && tid == 0 && a.status) a.status[b] = st;
    if (st) return;
    const int n = min(kPathRows, len - c * kPathRows);
    if (n <= 0) return;
    if (tid < n) {
        const int i = c * kPathRows + tid;
        s_src[tid] = (long long)b * a.T + acc[i];
        s_dst[tid] = cache_place(a, b, a.cache_len[b] + i);
    }
    __syncthreads();
    constexpr int K = 4, kStep = K * (256 / LPR);
    Raw<TIO, VEC> q[K];
    for (int u0 = tid / LPR; u0 - tid / LPR < n * a.Hk * 2; u0 += kStep) {
        fetch<TIO, LPR, VEC>(a, n, u0, [&](int row) { return s_src[row]; }, q);
        flush<TIO, LPR, E4M3, VEC>(a, n, u0, s_dst, q);
    }
}

template <typename TIO, int LPR, bool E4M3, bool VEC>
hipError_t launch_one(const CacheWriteArgs& a, hipStream_t stream) {
    if (a.seq_start) {
        const int blocks = (int)append_blocks(a.T, 0);
        const int all = (int)append_blocks(a.T, a.status ? a.batch : 0);
        if (all > 0)
            hipLaunchKernelGGL((append_kernel<TIO, LPR, E4M3, VEC>), dim3(all), dim3(256), 0, stream, a, blocks);
    } else {
        const int chunks = (int)commit_blocks(1, a.T, a.Lmax);
        hipLaunchKernelGGL((commit_kernel<TIO, LPR, E4M3, VEC>), dim3((unsigned)((long long)a.batch * chunks)), dim3(256), 0,
                           stream, a, chunks);
    }
    return hipGetLastError();
}

template <typename TIO, bool E4M3>
hipError_t launch_type(const CacheWriteArgs& a, hipStream_t stream) {
    // 8 elements at a time where rows and pointers allow it
    const uintptr_t in = (uintptr_t)a.k | (uintptr_t)a.v, out = (uintptr_t)a.k_cache | (uintptr_t)a.v_cache;
    const bool vec = a.D % 8 == 0 && in % 16 == 0 && out % (E4M3 ? 8 : 16) == 0;
    if (a.D <= 64) return vec ? launch_one<TIO, 8, E4M3, true>(a, stream) : launch_one<TIO, 8, E4M3, false>(a, stream);
    if (a.D <= 128) return vec ? launch_one<TIO, 16, E4M3, true>(a, stream) : launch_one<TIO, 16, E4M3, false>(a, stream);
    return vec ? launch_one<TIO, 32, E4M3, true>(a, stream) : launch_one<TIO, 32, E4M3, false>(a, stream);
}

}  // namespace

long long commit_blocks(int batch, int T, int max_path_len) {
    return (long long)batch * max(1, (min(max_path_len, T) + kPathRows - 1) / kPathRows);
}
long long append_blocks(int n_rows, int items) { return ((long long)n_rows + kRows - 1) / kRows + items; }

hipError_t launch_cache_write(const CacheWriteArgs& a, bool bf16, bool e4m3, hipStream_t stream) {
    if (bf16) return e4m3 ? launch_type<uint16_t, true>(a, stream) : launch_type<uint16_t, false>(a, stream);
    return e4m3 ? launch_type<float, true>(a, stream) : launch_type<float, false>(a, stream);
}

}  // namespace tsv
