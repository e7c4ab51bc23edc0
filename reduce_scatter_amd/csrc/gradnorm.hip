// gradnorm.hip -- the global norm of many gradient buffers, and clipping.
//
//   norm = scale sqrt(sum g^2),   out = g scale f,   f = min(1, max_norm / (norm + eps))
//
// A launch takes a table of buffers by value; its workgroups deal out chunks of
// them.  Squares are added up in 64 bits (their range and their number are the
// lists', not one row's), a partial sum to a workgroup; the partial sums are few,
// so every workgroup of the scaling launch adds them up by itself instead of
// waiting for a launch that does nothing else.  Bounded by HBM bytes: everything
// is read once for the norm and, where it does not stay in the cache, again for the scaling.
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

__device__ __forceinline__ double block_sum(double v, double *lds) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    v = lanes_sum<64>(v, lane);
    if (lane == 0) lds[wave] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += lds[w];
    return v;
}

template <int DT> __device__ __forceinline__ void add_squares(const char *p, int n, double &sum) {
    constexpr int U = DT == F32 ? 4 : 8;
    int i = threadIdx.x * 8;
    for (; i + (U - 1) * kThreads * 8 + 8 <= n; i += U * kThreads * 8) {
        Oct<DT> o[U];
#pragma unroll
        for (int u = 0; u < U; ++u) o[u] = load_oct<DT, false>(p + (long long)(i + u * kThreads * 8) * elem_bytes<DT>());
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float v[8];
            widen<DT>(o[u], v);
#pragma unroll
            for (int k = 0; k < 8; ++k) sum = __builtin_fma((double)v[k], (double)v[k], sum);
        }
    }
    for (; i < n; i += kThreads * 8) {
        float v[8];
        const char *q = p + (long long)i * elem_bytes<DT>();
        if (n - i >= 8) widen<DT>(load_oct<DT, false>(q), v);
        else widen<DT>(load_short<DT>(q, n - i), v);
#pragma unroll
        for (int k = 0; k < 8; ++k) sum = __builtin_fma((double)v[k], (double)v[k], sum);
    }
}

__global__ __launch_bounds__(kThreads) void grad_sum_kernel(const GradTable t) {
    __shared__ double lds[kWaves];
    const int lane = threadIdx.x & 63;
    const uint32_t chunks = t.first[t.n];
    double sum = 0.0;
    for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int e = __builtin_amdgcn_readfirstlane(entry_of(t, c, lane));
        const uint32_t at = (c - t.first[e]) * kGradChunk, left = t.size[e] - at;
        const int n = left < kGradChunk ? (int)left : kGradChunk;
        switch (t.dtype[e]) {
        case F32: add_squares<F32>(t.in[e] + (long long)at * 4, n, sum); break;
        case BF16: add_squares<BF16>(t.in[e] + (long long)at * 2, n, sum); break;
        default: add_squares<F16>(t.in[e] + (long long)at * 2, n, sum); break;
        }
    }
    sum = block_sum(sum, lds);
    if (threadIdx.x == 0) t.part[blockIdx.x] = sum;
}

// scale * sqrt of all partial sums, in 64 bits.
__device__ __forceinline__ double whole_norm(const GradTable &t, double *lds) {
    double sum = 0.0;
    for (int i = threadIdx.x; i < t.parts; i += kThreads) sum += t.part[i];
    return (double)t.scale * __builtin_sqrt(block_sum(sum, lds));
}

__global__ __launch_bounds__(kThreads) void grad_finish_kernel(const GradTable t) {
    __shared__ double lds[kWaves];
    const double norm = whole_norm(t, lds);
    if (threadIdx.x == 0) *t.norm = (float)norm;
}

template <int DT> __device__ __forceinline__ void scale_chunk(const char *in, char *out, int n, float f) {
    constexpr int U = DT == F32 ? 2 : 4;
    int i = threadIdx.x * 8;
    for (; i + (U - 1) * kThreads * 8 + 8 <= n; i += U * kThreads * 8) {
        Oct<DT> o[U];
#pragma unroll
        for (int u = 0; u < U; ++u) o[u] = load_oct<DT>(in + (long long)(i + u * kThreads * 8) * elem_bytes<DT>());
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float v[8];
            widen<DT>(o[u], v);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] *= f;
            store_oct<DT>(out + (long long)(i + u * kThreads * 8) * elem_bytes<DT>(), narrow<DT>(v), 8);
        }
    }
    for (; i < n; i += kThreads * 8) {
        float v[8];
        const char *q = in + (long long)i * elem_bytes<DT>();
        if (n - i >= 8) widen<DT>(load_oct<DT>(q), v);
        else widen<DT>(load_short<DT>(q, n - i), v);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] *= f;
        store_oct<DT>(out + (long long)i * elem_bytes<DT>(), narrow<DT>(v), n - i);
    }
}

__global__ __launch_bounds__(kThreads) void grad_scale_kernel(const GradTable t) {
    __shared__ double lds[kWaves];
    const int lane = threadIdx.x & 63;
    const double norm = whole_norm(t, lds);
    if (t.norm && blockIdx.x == 0 && threadIdx.x == 0) *t.norm = (float)norm;
    double f = (double)t.max_norm / (norm + (double)t.eps);
    if (!(f < 1.0)) f = norm != norm ? norm : 1.0;
    const float factor = (float)(f * (double)t.scale);
    const uint32_t chunks = t.first[t.n];
    for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int e = __builtin_amdgcn_readfirstlane(entry_of(t, c, lane));
        // nothing changes in place (a NaN keeps its bits, too)
        if (factor == 1.0f && t.in[e] == t.out[e]) continue;
        const uint32_t at = (c - t.first[e]) * kGradChunk, left = t.size[e] - at;
        const int n = left < kGradChunk ? (int)left : kGradChunk;
        switch (t.dtype[e]) {
        case F32: scale_chunk<F32>(t.in[e] + (long long)at * 4, t.out[e] + (long long)at * 4, n, factor); break;
        case BF16: scale_chunk<BF16>(t.in[e] + (long long)at * 2, t.out[e] + (long long)at * 2, n, factor); break;
        default: scale_chunk<F16>(t.in[e] + (long long)at * 2, t.out[e] + (long long)at * 2, n, factor); break;
        }
    }
}

}  // namespace

hipError_t launch_grad_sum(const GradTable &t, int groups, hipStream_t s) {
    return launch(grad_sum_kernel, dim3((unsigned)groups), dim3(kThreads), 0, s, t);
}
hipError_t launch_grad_finish(const GradTable &t, hipStream_t s) {
    return launch(grad_finish_kernel, dim3(1), dim3(kThreads), 0, s, t);
}
hipError_t launch_grad_scale(const GradTable &t, int groups, hipStream_t s) {
    return launch(grad_scale_kernel, dim3((unsigned)groups), dim3(kThreads), 0, s, t);
}

}  // namespace ar
