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
// meanwhile. 16 prompts, 16378 rows of 8 heads of 128 into e4m3 (102 MB): 27 us,
// 3.8 TB/s, half of it the vector work (at earlier steps: fetching after the search
// 31.6 us, 30.0 before it; the butterfly through LDS 30.0, by lane moves 29.0).
#include "attn_cache.hpp"

namespace tsv {
namespace {

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
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(f.v[i]) & 0x7fffffffu);
#pragma unroll
            for (int m = 16; m < LPR; m <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, m, kWave));
            top = max_of<LPR < 16 ? LPR : 16>(top);
            finite = top < 0x7f800000u;
            scale = scale_of(top);
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
    __shared__ RowPlaces<kRows> places;
    const int tid = threadIdx.x;
    const int r0 = blockIdx.x * kRows;
    const bool rows = (int)blockIdx.x < row_blocks;
    const int n = rows ? min(kRows, a.T - r0) : 0;
    // the rows are on their way while their places are found
    constexpr int K = VEC && sizeof(TIO) == 2 ? 8 : 4, kStep = K * (256 / LPR);
    Raw<TIO, VEC> q[K];
    const auto src = [&](int row) { return (long long)r0 + row; };
    fetch<TIO, LPR, VEC>(a, n, tid / LPR, src, q);
    if (!find_places<kRows>(a, r0, n, rows ? -1 : (int)blockIdx.x - row_blocks, places)) return;  // a block for each item's status
    for (int u0 = tid / LPR; u0 - tid / LPR < n * a.Hk * 2; u0 += kStep) {
        if (u0 != tid / LPR) fetch<TIO, LPR, VEC>(a, n, u0, src, q);
        flush<TIO, LPR, E4M3, VEC>(a, n, u0, places.dst, q);
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
