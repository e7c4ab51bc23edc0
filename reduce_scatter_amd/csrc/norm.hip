// norm.hip -- the sum of n ranks' partial results with the residual, its RMS
// norm and 8-bit output, and the backward pass.
//
//   s = residual + sum_r partial_r,  rstd = 1/sqrt(mean(s^2) + eps),
//   y = s rstd (offset + w),         out8 = e4m3(y / scale)
//   h = x rstd, u = g (offset + w),  dx = rstd (u - h mean(u h)) + g_s,  dw = sum over rows of g h
//
// Both are bounded by HBM bytes: a row is read once, stays in registers between
// its sum and its results, and is written once.  A row of up to 128 columns
// belongs to 16 lanes, one of up to 512 to a wave, a longer one to a workgroup
// of as many waves as it needs.
#include "dispatch.hpp"
#include "layer_device.hpp"

namespace ar {
namespace {

constexpr int kNormWaves = 16;
constexpr int kShortThreads = 256;     // of a workgroup with several rows

template <int LANES> constexpr int kWaveLanes = LANES == 16 ? 16 : 64;

// Sum over the row's lanes; `lds` (one entry per wave) is not used again.
template <int LANES, typename T> __device__ __forceinline__ T row_sum(T v, T *lds, int waves, int wave, int lane) {
    v = lanes_sum<kWaveLanes<LANES>>(v, lane);
    if constexpr (LANES == 0) {
        if (lane == 0) lds[wave] = v;
        __syncthreads();
        v = (lane & 15) < waves ? lds[lane & 15] : T(0);
        v = lanes_sum<16>(v, lane);
    }
    return v;
}
template <int LANES> __device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t *lds, int waves, int wave, int lane) {
    v = lanes_max<kWaveLanes<LANES>>(v, lane);
    if constexpr (LANES == 0) {
        if (lane == 0) lds[wave] = v;
        __syncthreads();
        v = (lane & 15) < waves ? lds[lane & 15] : 0u;
        v = lanes_max<16>(v, lane);
    }
    return v;
}

// offset + weight of a lane's columns.
template <int DT, bool TINY> __device__ __forceinline__ void load_weight(const NormRow &r, const ColPlace &p, float *w) {
    if (r.weight32) widen<F32>(load_at<F32, TINY, false>((const char *)r.weight, p), w);
    else widen<DT>(load_at<DT, TINY, false>((const char *)r.weight, p), w);
    settle<TINY>(w, p);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] += r.offset;
}

// Adds ranks r, ..., r + B - 1, their loads issued together.
template <int B, int DT, int U, bool TINY, int NR>
__device__ __forceinline__ void add_ranks(const NormArgs<NR> &a, int r, long long row, const ColPlace *p, float (*s)[8]) {
    Oct<DT> o[B][U];
#pragma unroll
    for (int b = 0; b < B; ++b) {
        const char *x = a.x[r + b] + row * (long long)a.pitch[r + b] * elem_bytes<DT>();
#pragma unroll
        for (int u = 0; u < U; ++u) o[b][u] = load_at<DT, TINY>(x, p[u]);
    }
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float v[8];
            widen<DT>(o[b][u], v);
#pragma unroll
            for (int i = 0; i < 8; ++i) s[u][i] += v[i];
        }
}

template <int DT, int U, int LANES, bool TINY, int NR>
__global__ __launch_bounds__(LANES ? kShortThreads : 64 * kNormWaves) void reduce_norm_kernel(const NormArgs<NR> a) {
    __shared__ float lds_sum[kNormWaves];
    __shared__ double lds_wide[kNormWaves];
    __shared__ uint32_t lds_max[kNormWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int threads = LANES ? LANES : blockDim.x, t = LANES ? threadIdx.x % (LANES ? LANES : 1) : threadIdx.x;
    const int width = a.r.width;
    const long long row = a.r.row0 + (LANES ? (long long)blockIdx.x * (kShortThreads / (LANES ? LANES : 1)) + threadIdx.x / (LANES ? LANES : 1)
                                            : (long long)blockIdx.x);
    if (LANES && row >= a.r.rows) return;

    ColPlace p[U];
    float s[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) p[u] = col_place<TINY>(u * threads + t, width);
    const long long packed = row * width;          // of the tensors without a pitch
    if (a.residual) {
#pragma unroll
        for (int u = 0; u < U; ++u) widen<DT>(load_at<DT, TINY>(a.residual + packed * elem_bytes<DT>(), p[u]), s[u]);
    } else {
        // -0 + x is x for every x, a negative zero included
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 8; ++i) s[u][i] = -0.0f;
    }
    constexpr int B = (DT == F32 ? 4 : 8) / U;
    int r = 0;
    for (; r + B <= a.n; r += B) add_ranks<B, DT, U, TINY>(a, r, row, p, s);
    if constexpr (B > 4)
        if (r + 4 <= a.n) add_ranks<4, DT, U, TINY>(a, r, row, p, s), r += 4;
    if constexpr (B > 2)
        if (r + 2 <= a.n) add_ranks<2, DT, U, TINY>(a, r, row, p, s), r += 2;
    if constexpr (B > 1)
        if (r < a.n) add_ranks<1, DT, U, TINY>(a, r, row, p, s);

    float sq = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        settle<TINY>(s[u], p[u]);
#pragma unroll
        for (int i = 0; i < 8; ++i) sq = __builtin_fmaf(s[u][i], s[u][i], sq);
    }
    sq = row_sum<LANES>(sq, lds_sum, waves, wave, lane);
    float rstd;
    if (sq >= 1e-30f && sq <= 1e30f) {
        rstd = __builtin_amdgcn_rsqf(sq / (float)width + a.r.eps);
    } else {
        // squares out of fp32's range, or a row of zeros, infinities or NaN
        double wide = 0.0;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 8; ++i) wide = __builtin_fma((double)s[u][i], (double)s[u][i], wide);
        wide = row_sum<LANES>(wide, lds_wide, waves, wave, lane);
        rstd = (float)(1.0 / __builtin_sqrt(wide / width + (double)a.r.eps));
    }
    if (a.rstd && t == 0) a.rstd[row] = rstd;

    if (a.summed) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            store_oct<DT>(a.summed + (packed + p[u].col) * elem_bytes<DT>(), narrow<DT>(s[u]), p[u].left);
    }
    if (!a.out && !a.out8) return;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float w[8];
        load_weight<DT, TINY>(a.r, p[u], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[u][i] = p[u].left > i ? s[u][i] * rstd * w[i] : 0.0f;
    }
    if (a.out) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            store_oct<DT>(a.out + (packed + p[u].col) * elem_bytes<DT>(), narrow<DT>(s[u]), p[u].left);
    }
    if (!a.out8) return;

    // The largest |y| by its bits, so that a NaN is larger than everything else.
    uint32_t most[U];
    uint32_t all = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        most[u] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t b = f32_bits(s[u][i]) & 0x7fffffffu;
            most[u] = b > most[u] ? b : most[u];
        }
        all = most[u] > all ? most[u] : all;
    }
    if (a.group == 0) all = row_max<LANES>(all, lds_max, waves, wave, lane);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (a.group == 0) {
            most[u] = all;
        } else {
            row_bits<kWaveLanes<LANES>>([&](auto m) {
                if (m.value < a.group) {
                    const uint32_t o = lane_xor<m.value>(most[u], lane);
                    most[u] = o > most[u] ? o : most[u];
                }
            });
        }
        const float amax = bits_f32(most[u]);
        const bool fine = finite(amax);
        const float scale = fine ? __builtin_fmaxf(amax / kE4m3Max, kLeastScale) : bits_f32(0x7fc00000u);
        const float inv = 1.0f / scale;
        const bool first = a.group ? t % a.group == 0 : (t == 0 && u == 0);
        if (first && p[u].left > 0) a.scales[row * a.groups + (a.group ? p[u].col / (8 * a.group) : 0)] = scale;
        uint32_t q[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            int v = __builtin_amdgcn_cvt_pk_fp8_f32(s[u][4 * i] * inv, s[u][4 * i + 1] * inv, 0, false);
            v = __builtin_amdgcn_cvt_pk_fp8_f32(s[u][4 * i + 2] * inv, s[u][4 * i + 3] * inv, v, true);
            q[i] = fine ? (uint32_t)v : 0x7f7f7f7fu;
        }
        uint8_t *to = a.out8 + packed + p[u].col;
        if (p[u].left >= 8) {
            __builtin_nontemporal_store(u32x2e{q[0], q[1]}, (u32x2e *)to);
        } else {
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (i < p[u].left) to[i] = (uint8_t)(q[i / 4] >> (8 * (i % 4)));
        }
    }
}

// h = x rstd and u = g (offset + w) of a lane's columns; g as it came.
template <int DT, bool TINY>
__device__ __forceinline__ void back_terms(const Oct<DT> &xo, const Oct<DT> &go, const ColPlace &p, const float *w,
                                           float rstd, float *h, float *g, float *u) {
    widen<DT>(xo, h);
    widen<DT>(go, g);
    settle<TINY>(h, p);
    settle<TINY>(g, p);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        h[i] *= rstd;
        u[i] = g[i] * w[i];
    }
}

// A workgroup takes every gridDim.x-th set of rows and keeps its part of the
// weight's gradient in registers throughout, and the weight too while that is
// eight columns to a lane.
template <int DT, int U, int LANES, bool TINY>
__global__ __launch_bounds__(LANES ? kShortThreads : 64 * kNormWaves) void norm_back_kernel(const NormBackArgs a) {
    constexpr int kSets = LANES ? kShortThreads / (LANES ? LANES : 1) : 1;     // rows at a time
    __shared__ float lds_sum[2][kNormWaves];
    __shared__ float lds_part[LANES ? kShortThreads / 64 : 1][LANES ? 512 : 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int threads = LANES ? LANES : blockDim.x, t = LANES ? threadIdx.x % (LANES ? LANES : 1) : threadIdx.x;
    const int width = a.r.width;
    ColPlace p[U];
    float w[8], dw[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        p[u] = col_place<TINY>(u * threads + t, width);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[u][i] = 0.0f;
    }
    if constexpr (U == 1) load_weight<DT, TINY>(a.r, p[0], w);
    int flip = 0;
    for (long long row = (long long)blockIdx.x * kSets + (LANES ? threadIdx.x / (LANES ? LANES : 1) : 0); row < a.r.rows;
         row += (long long)gridDim.x * kSets, flip ^= 1) {
        const long long packed = row * width * elem_bytes<DT>();
        const char *xr = a.x + row * a.x_pitch * elem_bytes<DT>();
        Oct<DT> xo[U], go[U], so[U];
#pragma unroll
        for (int u = 0; u < U; ++u) xo[u] = load_at<DT, TINY>(xr, p[u]), go[u] = load_at<DT, TINY>(a.grad_out + packed, p[u]);
        if (a.grad_summed) {
#pragma unroll
            for (int u = 0; u < U; ++u) so[u] = load_at<DT, TINY>(a.grad_summed + packed, p[u]);
        }
        const float rstd = a.rstd[row];
        float h[8], g[8], uv[8], dot = 0.0f;
        NormRow again = a.r;           // longer rows: read where it is used, not kept across rows
        if constexpr (U > 1) asm volatile("" : "+s"(again.weight));
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if constexpr (U > 1) {
                __builtin_amdgcn_sched_barrier(0);     // one oct's terms at a time
                load_weight<DT, TINY>(again, p[u], w);
            }
            back_terms<DT, TINY>(xo[u], go[u], p[u], w, rstd, h, g, uv);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dw[u][i] = __builtin_fmaf(g[i], h[i], dw[u][i]);
                if (p[u].left > i) dot = __builtin_fmaf(uv[i], h[i], dot);
            }
        }
        if (a.grad_summed) {
            // grad_x may be one of the inputs, and a short oct is read from columns that another lane writes:
            // everything has been read before the sum's barrier
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < (DT == F32 ? 2 : 1); ++j) asm volatile("" : "+v"(so[u].w[j]));
        }
        const float c = row_sum<LANES>(dot, lds_sum[flip], waves, wave, lane) / (float)width;
        if constexpr (U > 1) {
            // longer rows: the terms are worked out again from the values as stored, which take half the registers
            asm volatile("" : "+s"(again.weight));
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < (DT == F32 ? 2 : 1); ++j) asm volatile("" : "+v"(xo[u].w[j]), "+v"(go[u].w[j]));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if constexpr (U > 1) {
                __builtin_amdgcn_sched_barrier(0);
                load_weight<DT, TINY>(again, p[u], w);
                back_terms<DT, TINY>(xo[u], go[u], p[u], w, rstd, h, g, uv);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) uv[i] = rstd * __builtin_fmaf(-h[i], c, uv[i]);
            if (a.grad_summed) {
                widen<DT>(so[u], g);
                settle<TINY>(g, p[u]);
#pragma unroll
                for (int i = 0; i < 8; ++i) uv[i] += g[i];
            }
            store_oct<DT>(a.grad_x + packed + (long long)p[u].col * elem_bytes<DT>(), narrow<DT>(uv), p[u].left);
        }
    }
    if (!a.part) return;
    float *part = a.part + (long long)blockIdx.x * width;
    if constexpr (LANES == 0) {
#pragma unroll
        for (int u = 0; u < U; ++u) store_oct<F32, false>((char *)(part + p[u].col), narrow<F32>(dw[u]), p[u].left);
    } else {
        // rows of one workgroup, first within a wave (LANES 16), then over its waves
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (LANES == 16) {
                dw[0][i] += bits_f32(lane_xor<16>(f32_bits(dw[0][i]), lane));
                dw[0][i] += bits_f32(lane_xor<32>(f32_bits(dw[0][i]), lane));
            }
            if (lane < LANES) lds_part[wave][lane * 8 + i] = dw[0][i];
        }
        __syncthreads();
        for (int col = threadIdx.x; col < width; col += kShortThreads) {
            float v = 0.0f;
            for (int k = 0; k < kShortThreads / 64; ++k) v += lds_part[k][col];
            part[col] = v;
        }
    }
}

// Sum of the workgroups' partial weight gradients: 16 columns by 16 slices of the workgroups.
__global__ __launch_bounds__(256) void norm_weight_kernel(const float *part, int groups, int width, float *out) {
    __shared__ float lds[16][17];
    const int c = threadIdx.x & 15, k = threadIdx.x >> 4, col = blockIdx.x * 16 + c;
    float v = 0.0f;
    if (col < width)
        for (int g = k; g < groups; g += 16) v += part[(long long)g * width + col];
    lds[k][c] = v;
    __syncthreads();
    if (k == 0 && col < width) {
        v = 0.0f;
        for (int i = 0; i < 16; ++i) v += lds[i][c];
        out[col] = v;
    }
}

// Lanes, octs per lane and waves of a row.
struct RowPlan {
    int lanes, u, threads;
};
RowPlan plan_row(int width) {
    const int octs = (width + 7) / 8;
    if (octs <= 16) return {16, 1, kShortThreads};
    if (octs <= 64) return {64, 1, kShortThreads};
    int u = 1;
    while (octs > 64 * kNormWaves * u) u *= 2;
    return {0, u, (octs + 64 * u - 1) / (64 * u) * 64};
}

// f(dtype, octs per lane, lanes of a row, whether rows are shorter than an oct)
template <typename F> hipError_t dispatch_rows(int dtype, const RowPlan &p, int width, F &&f) {
    auto by_dt = [&](auto dt) {
        constexpr std::integral_constant<int, 1> one{};
        if (width < 8) return f(dt, one, std::integral_constant<int, 16>{}, std::true_type{});
        if (p.lanes == 16) return f(dt, one, std::integral_constant<int, 16>{}, std::false_type{});
        if (p.lanes == 64) return f(dt, one, std::integral_constant<int, 64>{}, std::false_type{});
        constexpr std::integral_constant<int, 0> block{};
        switch (p.u) {
        case 1: return f(dt, one, block, std::false_type{});
        case 2: return f(dt, std::integral_constant<int, 2>{}, block, std::false_type{});
        default: return hipErrorInvalidValue;
        }
    };
    switch (dtype) {
    case F32: return by_dt(std::integral_constant<int, F32>{});
    case BF16: return by_dt(std::integral_constant<int, BF16>{});
    case F16: return by_dt(std::integral_constant<int, F16>{});
    default: return hipErrorInvalidValue;
    }
}

template <int NR, typename DT, typename U, typename L, typename T>
hipError_t launch_forward(const NormCall &c, const RowPlan &p, DT, U, L, T, hipStream_t s) {
    NormArgs<NR> a;
    for (int r = 0; r < NR; ++r) {
        a.x[r] = r < c.n ? (const char *)c.x[r] : nullptr;
        a.pitch[r] = r < c.n ? (uint32_t)c.pitches[r] : 0;
    }
    a.n = c.n;
    a.group = c.a.group;
    a.groups = c.a.groups;
    a.r = c.a.r;
    a.residual = c.a.residual;
    a.summed = c.a.summed;
    a.out = c.a.out;
    a.rstd = c.a.rstd;
    a.out8 = c.a.out8;
    a.scales = c.a.scales;
    const long long sets = p.lanes ? kShortThreads / p.lanes : 1;
    const long long most = ((1LL << 31) / p.threads) * sets;       // a grid's threads stay below 2^32
    for (long long row = 0; row < c.a.r.rows; row += most) {
        a.r.row0 = row;
        const long long n = c.a.r.rows - row < most ? c.a.r.rows - row : most;
        const hipError_t e = launch(reduce_norm_kernel<DT::value, U::value, L::value, T::value, NR>,
                                    dim3((unsigned)((n + sets - 1) / sets)), dim3((unsigned)p.threads), 0, s, a);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_reduce_norm(const NormCall &c, hipStream_t s) {
    const RowPlan p = plan_row(c.a.r.width);
    return dispatch_rows(c.dtype, p, c.a.r.width, [&](auto dt, auto u, auto l, auto tiny) {
        return c.n <= kLayerFew ? launch_forward<kLayerFew>(c, p, dt, u, l, tiny, s)
                                : launch_forward<kLayerMany>(c, p, dt, u, l, tiny, s);
    });
}

int norm_back_groups(long long rows, int width) {
    const RowPlan p = plan_row(width);
    const long long sets = p.lanes ? kShortThreads / p.lanes : 1;
    const long long groups = (rows + sets - 1) / sets, most = 256LL * (2048 / p.threads);
    return (int)(groups < most ? groups : most);
}

hipError_t launch_norm_back(int dtype, const NormBackArgs &a, int groups, float *grad_weight, hipStream_t s) {
    const RowPlan p = plan_row(a.r.width);
    hipError_t e = hipSuccess;
    if (groups)
        e = dispatch_rows(dtype, p, a.r.width, [&](auto dt, auto u, auto l, auto tiny) {
            return launch(norm_back_kernel<dt.value, u.value, l.value, tiny.value>, dim3((unsigned)groups),
                          dim3((unsigned)p.threads), 0, s, a);
        });
    if (e == hipSuccess && grad_weight)
        e = launch(norm_weight_kernel, dim3((unsigned)((a.r.width + 15) / 16)), dim3(256), 0, s, (const float *)a.part, groups,
                   a.r.width, grad_weight);
    return e;
}

}  // namespace ar
