// gradnorm.hip -- the global norm of many gradient buffers, and clipping.
//
//   norm = scale sqrt(sum g^2),   out = g scale f,   f = min(1, max_norm / (norm + eps))
//
// A launch takes a table of buffers by value; its workgroups deal out chunks of
// them.  Squares are added up in 64 bits (their range and their number are the
// lists', not one row's), a partial sum to a workgroup.  Where these are few,
// every workgroup of the scaling launch adds them up by itself; else a launch of
// one workgroup does.  Bounded by HBM bytes: everything is read once for the
// norm and, where it does not stay in the cache, again for the scaling.
#include "dispatch.hpp"
#include "layer_device.hpp"

namespace ar {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

// The table entry of a chunk: entries whose first chunk is at most `chunk`, less one.
__device__ __forceinline__ int entry_of(const GradTable &t, uint32_t chunk, int lane) {
    static_assert(kGradTable <= 128, "two ballots");
    const uint32_t a = t.first[1 + lane], b = lane + 65 <= kGradTable ? t.first[lane + 65 <= kGradTable ? lane + 65 : 0] : ~0u;
    return __popcll(__ballot(a <= chunk)) + __popcll(__ballot(b <= chunk));
}

template <int WAVES = kWaves> __device__ __forceinline__ double block_sum(double v, double *lds) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    v = lanes_sum<64>(v, lane);
    if (lane == 0) lds[wave] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) v += lds[w];
    return v;
}

template <int DT, bool STREAM> __device__ __forceinline__ void add_squares(const char *p, int n, double &sum) {
    constexpr int K = Lanes<DT>::value, U = 4;
    int i = threadIdx.x * K;
    for (; i + (U - 1) * kThreads * K + K <= n; i += U * kThreads * K) {
        Run<DT, K> o[U];
#pragma unroll
        for (int u = 0; u < U; ++u) o[u] = load_run<DT, K, STREAM>(p + (long long)(i + u * kThreads * K) * elem_bytes<DT>());
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float v[K];
            widen<DT, K>(o[u], v);
#pragma unroll
            for (int k = 0; k < K; ++k) sum = __builtin_fma((double)v[k], (double)v[k], sum);
        }
    }
    for (; i < n; i += kThreads * K) {
        float v[K];
        const char *q = p + (long long)i * elem_bytes<DT>();
        if (n - i >= K) widen<DT, K>(load_run<DT, K, STREAM>(q), v);
        else widen<DT, K>(load_short<DT, K>(q, n - i), v);
#pragma unroll
        for (int k = 0; k < K; ++k) sum = __builtin_fma((double)v[k], (double)v[k], sum);
    }
}

// 2.75 GB: 399 us, 6.9 TB/s; 69 MB: 14 us (16 with half as many workgroups).
template <bool STREAM> __global__ __launch_bounds__(kThreads, 8) void grad_sum_kernel(const GradTable t) {
    __shared__ double lds[kWaves];
    const int lane = threadIdx.x & 63;
    const uint32_t chunks = t.first[t.n];
    double sum = 0.0;
    for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int e = __builtin_amdgcn_readfirstlane(entry_of(t, c, lane));
        const uint32_t at = (c - t.first[e]) * t.chunk, left = t.size[e] - at;
        const int n = left < (uint32_t)t.chunk ? (int)left : t.chunk;
        switch (t.dtype[e]) {
        case F32: add_squares<F32, STREAM>(t.in[e] + (long long)at * 4, n, sum); break;
        case BF16: add_squares<BF16, STREAM>(t.in[e] + (long long)at * 2, n, sum); break;
        default: add_squares<F16, STREAM>(t.in[e] + (long long)at * 2, n, sum); break;
        }
    }
    sum = block_sum(sum, lds);
    if (threadIdx.x == 0) t.part[blockIdx.x] = sum;
}

// scale * sqrt of all partial sums, in 64 bits.
template <int WAVES> __device__ __forceinline__ double whole_norm(const GradTable &t, double *lds) {
    double sum = 0.0;
    for (int i = threadIdx.x; i < t.parts; i += WAVES * 64) sum += t.part[i];
    return (double)t.scale * __builtin_sqrt(block_sum<WAVES>(sum, lds));
}

constexpr int kFinishWaves = 16;
__global__ __launch_bounds__(64 * kFinishWaves) void grad_finish_kernel(const GradTable t) {
    __shared__ double lds[kFinishWaves];
    const double norm = whole_norm<kFinishWaves>(t, lds);
    if (threadIdx.x == 0) {
        if (t.norm) *t.norm = (float)norm;
        if (t.wide) *t.wide = norm;
    }
}

// One step of a workgroup: two vectors to a thread.
template <int DT> __device__ __forceinline__ void scale_chunk(const char *in, char *out, int n, float f, float again) {
    constexpr int K = Lanes<DT>::value, U = kGradScaleBytes / 16 / kThreads;
    Run<DT, K> o[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = (u * kThreads + threadIdx.x) * K;
        const char *q = in + (long long)i * elem_bytes<DT>();
        if (n - i >= K) o[u] = load_run<DT, K>(q);
        else if (n > i) o[u] = load_short<DT, K>(q, n - i);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = (u * kThreads + threadIdx.x) * K;
        float v[K];
        widen<DT, K>(o[u], v);
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] *= f;
        if (again != 1.0f) {
#pragma unroll
            for (int k = 0; k < K; ++k) v[k] *= again;
        }
        store_run<DT, K>(out + (long long)i * elem_bytes<DT>(), narrow<DT, K>(v), n - i);
    }
}

// A workgroup scales one chunk: 8 KB each, in the order of their addresses.
// 2.75 GB in bf16 and fp32: 870 us, 6.3 TB/s; dealt out to 1024 or 2048 workgroups
// that stay, 967 and 1040.
__global__ __launch_bounds__(kThreads) void grad_scale_kernel(const GradTable t) {
    __shared__ double lds[kWaves];
    const double norm = t.parts ? whole_norm<kWaves>(t, lds) : *t.wide;
    if (t.norm && blockIdx.x == 0 && threadIdx.x == 0) *t.norm = (float)norm;
    double f = (double)t.max_norm / (norm + (double)t.eps);
    if (!(f < 1.0)) f = norm != norm ? norm : 1.0;
    f *= (double)t.scale;
    // A factor below fp32's normal numbers would lose digits, or all of it: such a one is taken in two steps.  (1.36 G
    // elements, norm included, take 1269 us with this branch and 1266 without.)
    const float again = f < 0x1p-126 ? 0x1p-126f : 1.0f;
    const float factor = (float)(f < 0x1p-126 ? f * 0x1p126 : f);
    const int e = __builtin_amdgcn_readfirstlane(entry_of(t, blockIdx.x, threadIdx.x & 63));
    // nothing changes in place
    if (factor == 1.0f && again == 1.0f && t.in[e] == t.out[e]) return;
    const int es = t.dtype[e] == F32 ? 4 : 2, chunk = kGradScaleBytes / es;
    const uint32_t at = (blockIdx.x - t.first[e]) * chunk, left = t.size[e] - at;
    const int n = left < (uint32_t)chunk ? (int)left : chunk;
    const char *in = t.in[e] + (long long)at * es;
    char *out = t.out[e] + (long long)at * es;
    switch (t.dtype[e]) {
    case F32: scale_chunk<F32>(in, out, n, factor, again); break;
    case BF16: scale_chunk<BF16>(in, out, n, factor, again); break;
    default: scale_chunk<F16>(in, out, n, factor, again); break;
    }
}

}  // namespace

hipError_t launch_grad_sum(const GradTable &t, int groups, hipStream_t s) {
    return launch(t.again ? grad_sum_kernel<false> : grad_sum_kernel<true>, dim3((unsigned)groups), dim3(kThreads), 0, s, t);
}
hipError_t launch_grad_finish(const GradTable &t, hipStream_t s) {
    return launch(grad_finish_kernel, dim3(1), dim3(64 * kFinishWaves), 0, s, t);
}
hipError_t launch_grad_scale(const GradTable &t, uint32_t groups, hipStream_t s) {
    return launch(grad_scale_kernel, dim3(groups), dim3(kThreads), 0, s, t);
}

}  // namespace ar
