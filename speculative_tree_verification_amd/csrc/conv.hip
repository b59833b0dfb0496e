// conv.hip -- the short causal convolution in front of an SSM layer, with its bias and
// activation, over packed prompts, single tokens and the nodes of a tree, and the state
// that it leaves.
//
//   y_t = act(bias + sum_{k < W} w[W - 1 - k] u_{t-k}),   act(y) = y or y / (1 + e^-y),
// for each channel by itself; u_{-1}, ..., u_{-(W-1)} are the state's rows from its last
// one on, and t - k is node t's k-th ancestor in a tree.
//
// Bound by the rows' traffic: every input is read once and every output written once for
// 2 W operations (32 prompts of 1 to 1531 tokens, 5120 channels in bf16, 504 MB: 118 us, 4.3
// TB/s; a large copy reaches 5.1). A lane has 16 bytes of neighbouring channels, whose taps stay in
// registers; a wave goes down a strip of a sequence's rows with the last W - 1 of them in
// registers, so that only a strip's first rows are read twice. Waves work by themselves
// (no barrier): each finds its sequence from seq_start. A sequence's first strip alone
// needs the state, so its wave also writes the new one.
#include "common.hpp"
#include "seq_launch.hpp"

namespace tsv {
namespace {

constexpr int kStBadSeqConv = 32;

// Channels of a lane as they are loaded: VEC: 16 bytes; otherwise one
template <typename TIO, bool VEC>
struct Chan;
template <>
struct Chan<uint16_t, true> {
    static constexpr int N = 8;
    uint4 u;
    __device__ __forceinline__ float f(int i) const {
        const uint32_t w = i / 2 == 0 ? u.x : i / 2 == 1 ? u.y : i / 2 == 2 ? u.z : u.w;
        return i % 2 ? __uint_as_float(w & 0xffff0000u) : __uint_as_float(w << 16);
    }
};
template <>
struct Chan<float, true> {
    static constexpr int N = 4;
    float4 u;
    __device__ __forceinline__ float f(int i) const { return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w; }
};
template <>
struct Chan<uint16_t, false> {
    static constexpr int N = 1;
    uint16_t u;
    __device__ __forceinline__ float f(int) const { return bf16_bits_to_f32(u); }
};
template <>
struct Chan<float, false> {
    static constexpr int N = 1;
    float u;
    __device__ __forceinline__ float f(int) const { return u; }
};

template <typename TIO, bool VEC>
__device__ __forceinline__ Chan<TIO, VEC> get(const void* p, size_t at) {
    typedef decltype(Chan<TIO, VEC>::u) U;
    return Chan<TIO, VEC>{gload((const U*)((const TIO*)p + at))};
}
template <typename TIO, bool VEC>
__device__ __forceinline__ void put(void* p, size_t at, const Chan<TIO, VEC>& c) {
    typedef decltype(Chan<TIO, VEC>::u) U;
    gstore((U*)((TIO*)p + at), c.u);
}
// rounded to nearest even
__device__ __forceinline__ Chan<uint16_t, true> rounded(const float (&v)[8]) {
    return {make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]))};
}
__device__ __forceinline__ Chan<float, true> rounded(const float (&v)[4]) { return {make_float4(v[0], v[1], v[2], v[3])}; }
template <typename TIO>
__device__ __forceinline__ Chan<TIO, false> rounded_one(float v) {
    if constexpr (sizeof(TIO) == 2)
        return {f32_to_bf16_bits(v)};
    else
        return {v};
}

// N floats (VEC: a multiple of 4, 16-byte aligned)
template <int N, bool VEC>
__device__ __forceinline__ void load_floats(const float* p, float (&v)[N]) {
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 u = gload((const float4*)(p + i));
            v[i] = u.x;
            v[i + 1] = u.y;
            v[i + 2] = u.z;
            v[i + 3] = u.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = gload(p + i);
    }
}

// A lane's channels: which, their taps and bias, and where their outputs go
template <typename TIO, int W, bool VEC>
struct Lane {
    static constexpr int N = Chan<TIO, VEC>::N;
    typedef Chan<TIO, VEC> Ch;
    int c;          // first channel
    bool in;        // whether there is one
    float w[W][N], bias[N];
    TIO* out;       // of row 0
    int width;      // elements between its rows

    __device__ __forceinline__ void init(const ConvArgs& a, int chunk) {
        const int C = a.HP + 2 * a.GN;
        c = (chunk * kWave + (threadIdx.x & (kWave - 1))) * N;
        in = c < C;
        if (!in) c = 0;
        const int in_B = c - a.HP, in_C = in_B - a.GN;
        out = in_B < 0 ? (TIO*)a.x + c : in_C < 0 ? (TIO*)a.B + in_B : (TIO*)a.C + in_C;
        width = in_B < 0 ? a.HP : a.GN;
    }
    __device__ __forceinline__ void taps(const ConvArgs& a) {
        float v[N * W];
        load_floats<N * W, VEC>(a.weight + (size_t)c * W, v);
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
            for (int k = 0; k < W; ++k) w[k][i] = v[i * W + k];
            bias[i] = 0.f;
        }
        if (a.bias) load_floats<N, VEC>(a.bias + c, bias);
    }
    // u[0], ..., u[W - 1]: the inputs, oldest first
    __device__ __forceinline__ Ch output(const ConvArgs& a, const Ch* const (&u)[W]) const {
        float y[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            y[i] = bias[i];
#pragma unroll
            for (int k = 0; k < W; ++k) y[i] = fmaf(w[k][i], u[k]->f(i), y[i]);
            // (its quotient off by 2^-22 and |y| 2^-24: below -87.3 the reciprocal is below the normal floats,
            // and the result 0 instead of at most 1.03e-36)
            if (a.silu) y[i] *= __builtin_amdgcn_rcpf(1.f + __expf(-y[i]));
        }
        if constexpr (VEC)
            return rounded(y);
        else
            return rounded_one<TIO>(y[0]);
    }
    __device__ __forceinline__ void store(size_t row, const Ch& v) const {
        if (in) put<TIO, VEC>(out, row * width, v);
    }
};

// Number of this wave among all, and of its unit and channels
__device__ __forceinline__ long long wave_unit() {
    return (long long)xcd_block(blockIdx.x, gridDim.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
}

// ---------------------------------------------------------------- prompts
// Strips of `strip` rows, sequence after sequence
template <typename TIO, int W, bool VEC>
__global__ __launch_bounds__(256) void conv_prefill_kernel(ConvArgs a, int strip, int chunks) {
    typedef Lane<TIO, W, VEC> L;
    typedef typename L::Ch Ch;
    const int lane = threadIdx.x & (kWave - 1);
    const long long unit = wave_unit();
    const int chunk = (int)(unit % chunks);
    const long long turn = unit / chunks;
    // its sequence and strip, and whether the packing is one
    long long run = 0;
    int seq = -1, t0 = 0, first = 0, len = 0, bad = 0;
    for (int q0 = 0; q0 < a.n; q0 += kWave) {
        const int q = q0 + lane;
        int lo = 0, hi = 0;
        if (q < a.n) {
            lo = a.seq_start[q];
            hi = a.seq_start[q + 1];
        }
        if (lo < 0 || hi < lo || hi > a.rows) {
            bad = 1;
            hi = lo;
        }
        const int n = hi - lo, cnt = n / strip + (n % strip != 0);
        int upto = cnt;
#pragma unroll
        for (int m = 1; m < kWave; m <<= 1) {
            const int o = __shfl_up(upto, m, kWave);
            if (lane >= m) upto += o;
        }
        const long long at = turn - run;
        const unsigned long long who = __ballot(at >= upto - cnt && at < upto);
        if (who) {
            const int src = __builtin_ctzll(who);
            seq = q0 + src;
            first = __builtin_amdgcn_readlane(lo, src);
            len = __builtin_amdgcn_readlane(n, src);
            t0 = ((int)at - __builtin_amdgcn_readlane(upto - cnt, src)) * strip;
        }
        run += __builtin_amdgcn_readlane(upto, kWave - 1);
    }
    bad = __ballot(bad) != 0;
    if (unit == 0 && a.status)
        for (int q = lane; q < a.n; q += kWave) a.status[q] = bad ? kStBadSeqConv : 0;
    if (bad || seq < 0) return;
    L l;
    l.init(a, chunk);
    const int C = a.HP + 2 * a.GN, t1 = min(len, t0 + strip);
    const size_t state = (size_t)seq * (W - 1) * C + l.c;
    auto row = [&](int t) { return get<TIO, VEC>(a.xbc, (size_t)(first + t) * a.stride + l.c); };
    constexpr int S = 4;  // rows on their way at once
    Ch u[W - 1 + S];
#pragma unroll
    for (int m = 0; m < W - 1; ++m) {
        if (t0 == 0)
            u[m] = get<TIO, VEC>(a.state, state + (size_t)m * C);
        else
            u[m] = row(t0 - (W - 1) + m);
    }
#pragma unroll
    for (int i = 0; i < S; ++i) u[W - 1 + i] = row(min(t0 + i, t1 - 1));
    l.taps(a);
    if (t0 == 0 && l.in) {  // the new state: the last rows of the old one and the sequence
        Ch s[W - 1];
#pragma unroll
        for (int m = 0; m < W - 1; ++m) {
            const int t = len - (W - 1) + m;  // row t, or state row W - 1 + t
            if (t >= 0) s[m] = row(t);
        }
#pragma unroll
        for (int m = 0; m < W - 1; ++m) {
            const int t = len - (W - 1) + m;
#pragma unroll
            for (int o = 0; o < W - 1; ++o)
                if (t < 0 && W - 1 + t == o) s[m] = u[o];
        }
#pragma unroll
        for (int m = 0; m < W - 1; ++m) put<TIO, VEC>(a.state, state + (size_t)m * C, s[m]);
    }
    for (int t = t0; t < t1; t += S) {
        Ch v[S];
#pragma unroll
        for (int i = 0; i < S; ++i)
            if (t + S < t1) v[i] = row(min(t + S + i, t1 - 1));
#pragma unroll
        for (int i = 0; i < S; ++i) {
            if (t + i >= t1) break;
            const Ch* in[W];
#pragma unroll
            for (int k = 0; k < W; ++k) in[k] = &u[i + k];
            l.store((size_t)(first + t + i), l.output(a, in));
        }
#pragma unroll
        for (int m = 0; m < W - 1; ++m) u[m] = u[S + m];
#pragma unroll
        for (int i = 0; i < S; ++i) u[W - 1 + i] = v[i];
    }
}

// ---------------------------------------------------------------- one token
template <typename TIO, int W, bool VEC>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvArgs a, int chunks) {
    typedef Lane<TIO, W, VEC> L;
    typedef typename L::Ch Ch;
    const long long unit = wave_unit();
    const int b = (int)(unit / chunks);
    if (b >= a.n) return;
    L l;
    l.init(a, (int)(unit % chunks));
    const int C = a.HP + 2 * a.GN;
    const size_t state = (size_t)b * (W - 1) * C + l.c;
    Ch u[W];
#pragma unroll
    for (int m = 0; m < W - 1; ++m) u[m] = get<TIO, VEC>(a.state, state + (size_t)m * C);
    u[W - 1] = get<TIO, VEC>(a.xbc, (size_t)b * a.stride + l.c);
    l.taps(a);
    const Ch* in[W];
#pragma unroll
    for (int k = 0; k < W; ++k) in[k] = &u[k];
    l.store(b, l.output(a, in));
    if (!l.in) return;
#pragma unroll
    for (int m = 0; m < W - 1; ++m) put<TIO, VEC>(a.state, state + (size_t)m * C, u[m + 1]);
}

// Status bits of a tree: the same in all lanes of the wave. *mine: the parent of node `lane`
__device__ __forceinline__ int check_parents(const int32_t* parent, int T, int* mine) {
    int bits = 0;
    *mine = 0;
    for (int i = threadIdx.x & (kWave - 1); i < T; i += kWave) {
        const int p = parent[i];
        if (i < kWave) *mine = p;
        bits |= i == 0 ? (p != -1 ? kStBadRoot : 0) : (p < 0 || p >= i ? kStBadParent : 0);
    }
    return (__ballot(bits & kStBadRoot) ? kStBadRoot : 0) | (__ballot(bits & kStBadParent) ? kStBadParent : 0);
}

// ---------------------------------------------------------------- a tree's nodes
// `nodes` of them a wave, at most 64
template <typename TIO, int W, bool VEC>
__global__ __launch_bounds__(256) void conv_verify_kernel(ConvArgs a, int nodes, int strips, int chunks) {
    typedef Lane<TIO, W, VEC> L;
    typedef typename L::Ch Ch;
    const int lane = threadIdx.x & (kWave - 1), T = a.rows;
    const long long unit = wave_unit();
    const int chunk = (int)(unit % chunks), strip = (int)(unit / chunks % strips), b = (int)(unit / chunks / strips);
    if (b >= a.n) return;
    const int32_t* parent = a.parent + (size_t)b * T;
    L l;
    l.init(a, chunk);
    l.taps(a);
    int par;
    const int st = check_parents(parent, T, &par);
    if (chunk == 0 && strip == 0 && lane == 0 && a.status) a.status[b] = st;
    if (st) return;
    // lane i: the ancestors of node first + i: a node, or -m for the m-th state row from the last one on
    const int first = strip * nodes, n = min(nodes, T - first);
    int up[W - 1], j = first + min(lane, n - 1);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        // (the root's parent is -1: past it the count goes on)
        const int p = T <= kWave ? __shfl(par, max(j, 0), kWave) : j > 0 ? parent[j] : -1;
        j = j > 0 ? p : j - 1;
        up[k] = j;
    }
    const int C = a.HP + 2 * a.GN;
    const size_t state = (size_t)b * (W - 1) * C + l.c;
    auto input = [&](int node) {
        return node >= 0 ? get<TIO, VEC>(a.xbc, ((size_t)b * T + node) * a.stride + l.c)
                         : get<TIO, VEC>(a.state, state + (size_t)(W - 1 + node) * C);
    };
    constexpr int S = 4;
    for (int i0 = 0; i0 < n; i0 += S) {
        Ch u[S][W];
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int i = min(i0 + s, n - 1);
            u[s][W - 1] = input(first + i);
#pragma unroll
            for (int k = 0; k < W - 1; ++k) u[s][W - 2 - k] = input(__builtin_amdgcn_readlane(up[k], i));
        }
#pragma unroll
        for (int s = 0; s < S; ++s) {
            if (i0 + s >= n) break;
            const Ch* in[W];
#pragma unroll
            for (int k = 0; k < W; ++k) in[k] = &u[s][k];
            l.store((size_t)b * T + first + i0 + s, l.output(a, in));
        }
    }
}

// ---------------------------------------------------------------- an accepted path
template <typename TIO, int W, bool VEC>
__global__ __launch_bounds__(256) void conv_commit_kernel(ConvArgs a, int chunks) {
    typedef Lane<TIO, W, VEC> L;
    typedef typename L::Ch Ch;
    const int lane = threadIdx.x & (kWave - 1), T = a.rows;
    const long long unit = wave_unit();
    const int chunk = (int)(unit % chunks), b = (int)(unit / chunks);
    if (b >= a.n) return;
    const int32_t* parent = a.parent + (size_t)b * T;
    const int32_t* acc = a.accepted + (size_t)b * a.Lmax;
    int par, st = check_parents(parent, T, &par);
    const int len = a.accepted_len[b];
    int bad = len < 0 || len > a.Lmax || len > T;
    for (int i = lane; !bad && i < len; i += kWave) {
        const int node = acc[i], want = i == 0 ? -1 : acc[i - 1];
        if (node < 0 || node >= T || (i == 0 ? node != 0 : parent[node] != want)) bad = 1;
    }
    if (__ballot(bad)) st |= kStBadPath;
    if (chunk == 0 && lane == 0 && a.status) a.status[b] = st;
    if (st || len == 0) return;
    L l;
    l.init(a, chunk);
    const int C = a.HP + 2 * a.GN;
    const size_t state = (size_t)b * (W - 1) * C + l.c;
    Ch s[W - 1];
#pragma unroll
    for (int m = 0; m < W - 1; ++m) {
        const int i = len - (W - 1) + m;  // path entry i, or state row W - 1 + i
        s[m] = i >= 0 ? get<TIO, VEC>(a.xbc, ((size_t)b * T + acc[i]) * a.stride + l.c)
                      : get<TIO, VEC>(a.state, state + (size_t)(W - 1 + i) * C);
    }
    if (!l.in) return;
#pragma unroll
    for (int m = 0; m < W - 1; ++m) put<TIO, VEC>(a.state, state + (size_t)m * C, s[m]);
}

int chunks_of(int HP, int GN, int lane_channels) { return (HP + 2 * GN + kWave * lane_channels - 1) / (kWave * lane_channels); }

// Rows of a strip: some 4000 waves, whose first rows are read twice and whose taps are loaded
// once each, or as many as there can be (32 packed prompts of an 8B hybrid: 118 us, 144 in
// strips of 64, 117 of 16; three fp32 prompts of 1360 tokens in all: 7.4 us in strips of 4, 8.0
// of 8, 9.7 of 16)
int strip_of(int rows, int chunks) {
    const long long all = (long long)rows * chunks;
    return all >= 65536 ? 32 : all >= 32768 ? 16 : all >= 16384 ? 8 : 4;
}

// Nodes of a wave, in the kernel with 4, 8 and 32 of them (us; 5376 or 5120 channels): 16 trees of 31
// nodes 8.4, 8.8, 20 (the latency of the launch, the parents, the taps and the inputs), 8 of 255
// 17.8, 15.7, 22, 64 of 63 27.8, 26, 33, 64 of 255 135, 114, 103 (336 MB; every input comes W times,
// from the L2 after the first)
int nodes_of(int n, int T, int chunks) {
    const long long all = (long long)n * T * chunks;
    return min(T, all >= 65536 ? 32 : all >= 16384 ? 8 : 4);
}

// Waves of a launch
long long units_of(ConvKind kind, int n, int rows, int chunks) {
    if (kind == kConvPrefill) return max(1LL, (long long)rows / strip_of(rows, chunks) + min(n, rows)) * chunks;
    if (kind == kConvVerify) {
        const int nodes = nodes_of(n, rows, chunks);
        return (long long)n * ((rows + nodes - 1) / nodes) * chunks;
    }
    return (long long)n * chunks;
}

template <typename TIO, int W, bool VEC>
void launch_one(ConvKind kind, const ConvArgs& a, hipStream_t stream) {
    const int chunks = chunks_of(a.HP, a.GN, Chan<TIO, VEC>::N);
    const dim3 grid((unsigned)((units_of(kind, a.n, a.rows, chunks) + 3) / 4));
    if (kind == kConvPrefill)
        hipLaunchKernelGGL((conv_prefill_kernel<TIO, W, VEC>), grid, dim3(256), 0, stream, a, strip_of(a.rows, chunks), chunks);
    else if (kind == kConvStep)
        hipLaunchKernelGGL((conv_step_kernel<TIO, W, VEC>), grid, dim3(256), 0, stream, a, chunks);
    else if (kind == kConvVerify)
        hipLaunchKernelGGL((conv_verify_kernel<TIO, W, VEC>), grid, dim3(256), 0, stream, a, nodes_of(a.n, a.rows, chunks),
                           (a.rows + nodes_of(a.n, a.rows, chunks) - 1) / nodes_of(a.n, a.rows, chunks), chunks);
    else
        hipLaunchKernelGGL((conv_commit_kernel<TIO, W, VEC>), grid, dim3(256), 0, stream, a, chunks);
}

template <typename TIO, int W>
hipError_t launch_width(ConvKind kind, const ConvArgs& a, hipStream_t stream) {
    // 16 bytes of channels a lane where the outputs' borders, strides and pointers allow it
    constexpr int N = 16 / sizeof(TIO);
    const uintptr_t all = (uintptr_t)a.xbc | (uintptr_t)a.state | (uintptr_t)a.x | (uintptr_t)a.B | (uintptr_t)a.C |
                          (uintptr_t)a.weight | (uintptr_t)a.bias;
    if (all % 16 == 0 && a.HP % N == 0 && a.GN % N == 0 && a.stride % N == 0)
        launch_one<TIO, W, true>(kind, a, stream);
    else
        launch_one<TIO, W, false>(kind, a, stream);
    return hipGetLastError();
}

template <typename TIO>
hipError_t launch_type(ConvKind kind, const ConvArgs& a, int width, hipStream_t stream) {
    return width == 4 ? launch_width<TIO, 4>(kind, a, stream) : width == 3 ? launch_width<TIO, 3>(kind, a, stream) : launch_width<TIO, 2>(kind, a, stream);
}

}  // namespace

// of the kernels that take one channel a lane, which have the most
long long conv_blocks(ConvKind kind, int n, int rows, int HP, int GN) { return (units_of(kind, n, rows, chunks_of(HP, GN, 1)) + 3) / 4; }

hipError_t launch_conv(ConvKind kind, const ConvArgs& a, int width, bool bf16, hipStream_t stream) {
    return bf16 ? launch_type<uint16_t>(kind, a, width, stream) : launch_type<float>(kind, a, width, stream);
}

}  // namespace tsv
