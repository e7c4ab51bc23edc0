// norm.hip -- the sum of n ranks' partial results with the residual, its RMS
// norm and 8-bit output, and the backward pass.
//
//   s = residual + sum_r partial_r,  rstd = 1/sqrt(mean(s^2) + eps),
//   y = s rstd (offset + w),         out8 = e4m3(y / scale)
//   h = x rstd, u = g (offset + w),  dx = rstd (u - h mean(u h)) + g_s,  dw = sum over rows of g h
//
// Both are bounded by HBM bytes: a row is read once, stays in registers between
// its sum and its results, and is written once.  A row of up to 16 runs (16
// bytes each) belongs to 16 lanes, one of up to 64 to a wave, a longer one to a
// workgroup of as many waves as it needs.
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
template <int DT, int K, bool TINY> __device__ __forceinline__ void load_weight(const NormRow &r, const ColPlace &p, float *w) {
    if (r.weight32) widen<F32, K>(load_at<F32, K, TINY, false>((const char *)r.weight, p), w);
    else widen<DT, K>(load_at<DT, K, TINY, false>((const char *)r.weight, p), w);
    settle<K, TINY>(w, p);
#pragma unroll
    for (int i = 0; i < K; ++i) w[i] += r.offset;
}

// Adds ranks r, ..., r + B - 1, their loads issued together.
template <int B, int DT, int K, int U, bool TINY, int NR>
__device__ __forceinline__ void add_ranks(const NormArgs<NR> &a, int r, long long row, const ColPlace *p, float (*s)[K]) {
    Run<DT, K> o[B][U];
#pragma unroll
    for (int b = 0; b < B; ++b) {
        const char *x = a.x[r + b] + row * (long long)a.pitch[r + b] * elem_bytes<DT>();
#pragma unroll
        for (int u = 0; u < U; ++u) o[b][u] = load_at<DT, K, TINY>(x, p[u]);
    }
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float v[K];
            widen<DT, K>(o[b][u], v);
#pragma unroll
            for (int i = 0; i < K; ++i) s[u][i] += v[i];
        }
}

// y / scale to nearest, the reciprocal taken in two parts (inv and what it lacks):
// off only where the quotient is within 2^-22 of a step of a border between two
// numbers.  y * inv alone is off by up to 1.5 steps, which put one value in a few
// million on the neighbouring e4m3 number.  us of y * inv, of this, of two steps
// of correction by the remainder, of a division: 16384 x 8192 fp32, a scale to a
// row 139, 143, 148, 154; bf16 from 2 ranks, 128 columns to a scale 193, 194, 195, 207.
__device__ __forceinline__ float quotient(float y, float inv, float rest) { return __builtin_fmaf(y, inv, y * rest); }

// 16384 x 8192 bf16 from 8 ranks with the residual: 481 us, 6.1 TB/s of 2.95 GB, the
// same with 4, 8 or 16 waves to a row; 3001 x 5003 fp16 from 4 with both outputs 45
// us, 5.0 TB/s (rows off 16-byte boundaries); one row of 4096 from 8 ranks 3.2 us.
template <int DT, int U, int LANES, bool TINY, int NR>
__global__ __launch_bounds__(LANES ? kShortThreads : 64 * kNormWaves) void reduce_norm_kernel(const NormArgs<NR> a) {
    __shared__ float lds_sum[kNormWaves];
    __shared__ double lds_wide[kNormWaves];
    __shared__ uint32_t lds_max[kNormWaves * U];
    constexpr int K = Lanes<DT>::value;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int threads = LANES ? LANES : blockDim.x, t = LANES ? threadIdx.x % (LANES ? LANES : 1) : threadIdx.x;
    const int width = a.r.width;
    const long long row = a.r.row0 + (LANES ? (long long)blockIdx.x * (kShortThreads / (LANES ? LANES : 1)) + threadIdx.x / (LANES ? LANES : 1)
                                            : (long long)blockIdx.x);
    if (LANES && row >= a.r.rows) return;

    ColPlace p[U];
    float s[U][K];
#pragma unroll
    for (int u = 0; u < U; ++u) p[u] = col_place<K, TINY>(u * threads + t, width);
    const long long packed = row * width;          // of the tensors without a pitch
    if (a.residual) {
#pragma unroll
        for (int u = 0; u < U; ++u) widen<DT, K>(load_at<DT, K, TINY>(a.residual + packed * elem_bytes<DT>(), p[u]), s[u]);
    } else {
        // -0 + x is x for every x, a negative zero included
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < K; ++i) s[u][i] = -0.0f;
    }
    constexpr int B = 8 / U;
    int r = 0;
    for (; r + B <= a.n; r += B) add_ranks<B, DT, K, U, TINY>(a, r, row, p, s);
    if constexpr (B > 4)
        if (r + 4 <= a.n) add_ranks<4, DT, K, U, TINY>(a, r, row, p, s), r += 4;
    if constexpr (B > 2)
        if (r + 2 <= a.n) add_ranks<2, DT, K, U, TINY>(a, r, row, p, s), r += 2;
    if constexpr (B > 1)
        if (r < a.n) add_ranks<1, DT, K, U, TINY>(a, r, row, p, s);

    float sq = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        settle<K, TINY>(s[u], p[u]);
#pragma unroll
        for (int i = 0; i < K; ++i) sq = __builtin_fmaf(s[u][i], s[u][i], sq);
    }
    sq = row_sum<LANES>(sq, lds_sum, waves, wave, lane);
    float rstd, root;                  // what is stored, and what s is multiplied with
    bool lift = false;                 // rstd may be past fp32, which takes eps = 0 and subnormal numbers: s 2^64, root 2^-64
    if (sq >= 1e-30f && sq <= 1e30f) {
        root = rstd = __builtin_amdgcn_rsqf(sq / (float)width + a.r.eps);
    } else {
        // squares out of fp32's range, or a row of zeros, infinities or NaN
        double wide = 0.0;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < K; ++i) wide = __builtin_fma((double)s[u][i], (double)s[u][i], wide);
        wide = row_sum<LANES>(wide, lds_wide, waves, wave, lane);
        const double r = 1.0 / __builtin_sqrt(wide / width + (double)a.r.eps);
        rstd = (float)r;
        lift = r > 0x1p127 && r < 0x1p300;
        if (lift) root = (float)(r * 0x1p-64);
        else root = rstd;
    }
    if (a.rstd && t == 0) a.rstd[row] = rstd;

    if (a.summed) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            store_run<DT, K>(a.summed + (packed + p[u].col) * elem_bytes<DT>(), narrow<DT, K>(s[u]), p[u].left);
    }
    if (!a.out && !a.out8) return;
    if (lift) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < K; ++i) s[u][i] *= 0x1p64f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float w[K];
        load_weight<DT, K, TINY>(a.r, p[u], w);
#pragma unroll
        for (int i = 0; i < K; ++i) s[u][i] = p[u].left > i ? s[u][i] * root * w[i] : 0.0f;
    }
    if (a.out) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            store_run<DT, K>(a.out + (packed + p[u].col) * elem_bytes<DT>(), narrow<DT, K>(s[u]), p[u].left);
    }
    if (!a.out8) return;

    // The largest |y| by its bits, so that a NaN is larger than everything else.
    uint32_t most[U];
    uint32_t all = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        most[u] = 0;
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const uint32_t b = f32_bits(s[u][i]) & 0x7fffffffu;
            most[u] = b > most[u] ? b : most[u];
        }
        all = most[u] > all ? most[u] : all;
    }
    if (a.group == 0) {
        all = row_max<LANES>(all, lds_max, waves, wave, lane);
#pragma unroll
        for (int u = 0; u < U; ++u) most[u] = all;
    } else {
#pragma unroll
        for (int u = 0; u < U; ++u)
            row_bits<kWaveLanes<LANES>>([&](auto m) {
                if (m.value < a.group) {
                    const uint32_t o = lane_xor<m.value>(most[u], lane);
                    most[u] = o > most[u] ? o : most[u];
                }
            });
        if (LANES == 0 && a.group > 64) {
            // a group of 512 columns in fp32: those of two neighbouring waves, in the order of the row
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (lane == 0) lds_max[u * waves + wave] = most[u];
            __syncthreads();
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int other = (u * waves + wave) ^ 1;
                if (other < U * waves) most[u] = lds_max[other] > most[u] ? lds_max[other] : most[u];
            }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const float amax = bits_f32(most[u]);
        const bool fine = finite(amax);
        const float scale = fine ? __builtin_fmaxf(amax / kE4m3Max, kLeastScale) : bits_f32(0x7fc00000u);
        const float inv = 1.0f / scale;
        const float rest = __builtin_fmaf(-inv, scale, 1.0f) * inv;        // the two make 1 / scale but for 2^-47 of it
        const int run = u * threads + t;
        if (p[u].left > 0 && (a.group ? run % a.group == 0 : run == 0)) a.scales[row * a.groups + (a.group ? run / a.group : 0)] = scale;
        uint32_t q[K / 4];
#pragma unroll
        for (int i = 0; i < K / 4; ++i) {
            float y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = quotient(s[u][4 * i + j], inv, rest);
            int v = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
            v = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], v, true);
            q[i] = fine ? (uint32_t)v : 0x7f7f7f7fu;
        }
        uint8_t *to = a.out8 + packed + p[u].col;
        if (p[u].left >= K) {
            if constexpr (K == 8) __builtin_nontemporal_store(u32x2e{q[0], q[1]}, (u32x2e *)to);
            else __builtin_nontemporal_store(q[0], (u32e *)to);
        } else {
#pragma unroll
            for (int i = 0; i < K - 1; ++i)
                if (i < p[u].left) to[i] = (uint8_t)(q[i / 4] >> (8 * (i % 4)));
        }
    }
}

// h = x rstd and u = g (offset + w) of a lane's columns; g as it came.
template <int DT, int K, bool TINY>
__device__ __forceinline__ void back_terms(const Run<DT, K> &xo, const Run<DT, K> &go, const ColPlace &p, const float *w,
                                           float rstd, float *h, float *g, float *u) {
    widen<DT, K>(xo, h);
    widen<DT, K>(go, g);
    settle<K, TINY>(h, p);
    settle<K, TINY>(g, p);
#pragma unroll
    for (int i = 0; i < K; ++i) {
        h[i] *= rstd;
        u[i] = g[i] * w[i];
    }
}

template <int DT, int K, int U> struct BackRow {       // a row as stored
    Run<DT, K> x[U], g[U], s[U];
    float rstd;
};
template <int DT, int K, int U, bool TINY>
__device__ __forceinline__ void load_back(const NormBackArgs &a, long long row, const ColPlace *p, BackRow<DT, K, U> &o) {
    const long long packed = row * a.r.width * elem_bytes<DT>();
    const char *x = a.x + row * a.x_pitch * elem_bytes<DT>();
#pragma unroll
    for (int u = 0; u < U; ++u) {
        o.x[u] = load_at<DT, K, TINY>(x, p[u]);
        o.g[u] = load_at<DT, K, TINY>(a.grad_out + packed, p[u]);
        if (a.grad_summed) o.s[u] = load_at<DT, K, TINY>(a.grad_summed + packed, p[u]);
    }
    o.rstd = a.rstd[row];
}

// A workgroup takes every gridDim.x-th set of rows, the next one's loads in
// flight while it works on one, and keeps its part of the weight's gradient in
// registers throughout.  16384 x 8192 bf16 with the residual's gradient: 170 us,
// 6.3 TB/s of its 1.07 GB, and 5 for the weight's gradient (512 workgroups
// without the next row in flight: 185 and 10).
template <int DT, int U, int LANES, bool TINY>
__global__ __launch_bounds__(LANES ? kShortThreads : 64 * kNormWaves) void norm_back_kernel(const NormBackArgs a) {
    constexpr int K = Lanes<DT>::value;
    constexpr int kSets = LANES ? kShortThreads / (LANES ? LANES : 1) : 1;     // rows at a time
    __shared__ float lds_sum[2][kNormWaves];
    __shared__ float lds_part[LANES ? kShortThreads / 64 : 1][LANES ? 64 * K : 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int threads = LANES ? LANES : blockDim.x, t = LANES ? threadIdx.x % (LANES ? LANES : 1) : threadIdx.x;
    const int width = a.r.width;
    // Up to 8 columns to a lane: the weight stays in registers, and a row's terms stay there from its sum to its results.
    constexpr bool kLong = U * K > 8;
    constexpr int kKept = kLong ? 1 : U;
    ColPlace p[U];
    float w[kKept][K], dw[U][K];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        p[u] = col_place<K, TINY>(u * threads + t, width);
        if constexpr (!kLong) load_weight<DT, K, TINY>(a.r, p[u], w[u]);
#pragma unroll
        for (int i = 0; i < K; ++i) dw[u][i] = 0.0f;
    }
    const long long step = (long long)gridDim.x * kSets;
    long long row = (long long)blockIdx.x * kSets + (LANES ? threadIdx.x / (LANES ? LANES : 1) : 0);
    BackRow<DT, K, U> next;            // longer rows have no registers for a second one
    if (!kLong && row < a.r.rows) load_back<DT, K, U, TINY>(a, row, p, next);
    for (int flip = 0; row < a.r.rows; row += step, flip ^= 1) {
        BackRow<DT, K, U> o;
        if constexpr (kLong) {
            load_back<DT, K, U, TINY>(a, row, p, o);
        } else {
            o = next;
            if (row + step < a.r.rows) load_back<DT, K, U, TINY>(a, row + step, p, next);
        }
        float h[kKept][K], uv[kKept][K], g[K], dot = 0.0f;
        NormRow again = a.r;           // longer rows: the weight is read where it is used, not kept across rows
        if constexpr (kLong) asm volatile("" : "+s"(again.weight));
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = kLong ? 0 : u;
            if constexpr (kLong) load_weight<DT, K, TINY>(again, p[u], w[k]);
            back_terms<DT, K, TINY>(o.x[u], o.g[u], p[u], w[k], o.rstd, h[k], g, uv[k]);
#pragma unroll
            for (int i = 0; i < K; ++i) {
                dw[u][i] = __builtin_fmaf(g[i], h[k][i], dw[u][i]);
                if (p[u].left > i) dot = __builtin_fmaf(uv[k][i], h[k][i], dot);
            }
        }
        // grad_x may be one of the inputs, and a short run is read from columns that another lane writes: everything of
        // the row has been read before the sum's barrier.
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < o.x[u].W; ++j) {
                if (a.grad_summed) asm volatile("" : "+v"(o.s[u].w[j]));
            }
        const float c = row_sum<LANES>(dot, lds_sum[flip], waves, wave, lane) / (float)width;
        if constexpr (kLong) {
            // the terms are worked out again from the values as stored, which take half the registers
            asm volatile("" : "+s"(again.weight));
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < o.x[u].W; ++j) asm volatile("" : "+v"(o.x[u].w[j]), "+v"(o.g[u].w[j]));
        }
        char *to = a.grad_x + row * width * elem_bytes<DT>();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = kLong ? 0 : u;
            if constexpr (kLong) {
                load_weight<DT, K, TINY>(again, p[u], w[k]);
                back_terms<DT, K, TINY>(o.x[u], o.g[u], p[u], w[k], o.rstd, h[k], g, uv[k]);
            }
            float d[K];
#pragma unroll
            for (int i = 0; i < K; ++i) d[i] = o.rstd * __builtin_fmaf(-h[k][i], c, uv[k][i]);
            if (a.grad_summed) {
                widen<DT, K>(o.s[u], g);
                settle<K, TINY>(g, p[u]);
#pragma unroll
                for (int i = 0; i < K; ++i) d[i] += g[i];
            }
            store_run<DT, K>(to + (long long)p[u].col * elem_bytes<DT>(), narrow<DT, K>(d), p[u].left);
        }
    }
    if (!a.part) return;
    float *part = a.part + (long long)blockIdx.x * a.part_width;
    if constexpr (LANES == 0) {
        // four columns of every lane after the other, so that a store's lanes fill whole lines
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < K / 4; ++j)
                store_run<F32, 4, false>((char *)(part + ((u * (K / 4) + j) * threads + t) * 4), narrow<F32, 4>(dw[u] + 4 * j), 4);
    } else {
        // rows of one workgroup, first within a wave (LANES 16), then over its waves
#pragma unroll
        for (int i = 0; i < K; ++i) {
            if constexpr (LANES == 16) {
                dw[0][i] += bits_f32(lane_xor<16>(f32_bits(dw[0][i]), lane));
                dw[0][i] += bits_f32(lane_xor<32>(f32_bits(dw[0][i]), lane));
            }
            if (lane < LANES) lds_part[wave][lane * K + i] = dw[0][i];
        }
        __syncthreads();
        for (int col = threadIdx.x; col < width; col += kShortThreads) {
            float v = 0.0f;
            for (int k = 0; k < kShortThreads / 64; ++k) v += lds_part[k][col];
            part[col] = v;
        }
    }
}

// Sum of the workgroups' partial weight gradients: 64 places by 16 slices of the
// workgroups.  `quads` is the number of lanes whose four columns follow one
// another in a partial gradient, `per` how many fours a lane has in a row (0:
// the columns are in order).
constexpr int kWeightSlices = 16;
__global__ __launch_bounds__(64 * kWeightSlices) void norm_weight_kernel(const float *part, int groups, int part_width, int quads,
                                                                         int per, int width, float *out) {
    __shared__ float lds[kWeightSlices][64];
    const int c = threadIdx.x & 63, k = threadIdx.x >> 6, at = blockIdx.x * 64 + c;
    float v = 0.0f;
    if (at < part_width) {
        constexpr int B = 8;
        int g = k;
        for (; g + (B - 1) * kWeightSlices < groups; g += B * kWeightSlices) {
            float f[B];
#pragma unroll
            for (int b = 0; b < B; ++b) f[b] = part[(long long)(g + b * kWeightSlices) * part_width + at];
#pragma unroll
            for (int b = 0; b < B; ++b) v += f[b];
        }
        for (; g < groups; g += kWeightSlices) v += part[(long long)g * part_width + at];
    }
    lds[k][c] = v;
    __syncthreads();
    if (k != 0 || at >= part_width) return;
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < kWeightSlices; ++i) v += lds[i][c];
    int col = at;
    if (per) {
        const int four = at / 4 / quads, lane = at / 4 % quads;
        col = ((four / per * quads + lane) * per + four % per) * 4 + at % 4;
    }
    if (col < width) out[col] = v;
}

// Lanes, runs per lane and threads of a row.
struct RowPlan {
    int lanes, u, threads;
};
RowPlan plan_row(int dtype, int width) {
    const int k = dtype == F32 ? 4 : 8, runs = (width + k - 1) / k;
    if (runs <= 16) return {16, 1, kShortThreads};
    if (runs <= 64) return {64, 1, kShortThreads};
    int u = 1;
    while (runs > 64 * kNormWaves * u) u *= 2;
    return {0, u, (runs + 64 * u - 1) / (64 * u) * 64};
}

// f(dtype, runs per lane, lanes of a row, whether rows are shorter than eight columns)
template <typename F> hipError_t dispatch_rows(int dtype, const RowPlan &p, int width, F &&f) {
    auto by_dt = [&](auto dt) {
        constexpr std::integral_constant<int, 1> one{};
        if (width < 8) return f(dt, one, std::integral_constant<int, 16>{}, std::true_type{});
        if (p.lanes == 16) return f(dt, one, std::integral_constant<int, 16>{}, std::false_type{});
        if (p.lanes == 64) return f(dt, one, std::integral_constant<int, 64>{}, std::false_type{});
        constexpr std::integral_constant<int, 0> block{};
        if (p.u == 1) return f(dt, one, block, std::false_type{});
        if (p.u == 2) return f(dt, std::integral_constant<int, 2>{}, block, std::false_type{});
        if constexpr (dt.value == F32) return f(dt, std::integral_constant<int, 4>{}, block, std::false_type{});
        return hipErrorInvalidValue;
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
    const RowPlan p = plan_row(c.dtype, c.a.r.width);
    return dispatch_rows(c.dtype, p, c.a.r.width, [&](auto dt, auto u, auto l, auto tiny) {
        return c.n <= kLayerFew ? launch_forward<kLayerFew>(c, p, dt, u, l, tiny, s)
                                : launch_forward<kLayerMany>(c, p, dt, u, l, tiny, s);
    });
}

NormBackPlan norm_back_plan(int dtype, long long rows, int width) {
    const RowPlan p = plan_row(dtype, width);
    const long long sets = p.lanes ? kShortThreads / p.lanes : 1;
    // Workgroups to a compute unit, up to 16 waves of them; each leaves a partial weight gradient that is written and
    // read once more.  us with 1, 2, 3, 4, 8 to a unit: 777 x 5003 fp32 (10 waves) 19, 21, 24, 25, 25; 2048 x 4096
    // bf16 (8) 15.2, 16.9, 19.0, 22.5, 27.8; 16384 x 2048 (4) 55, 42, 39, 42, 49; 8192 x 1024 (2) 27, 20, 18, 18, 21;
    // 65536 x 256 (a wave to a row, 4 rows) 55, 36, 33, 32, 36.  The rule takes the best of three of these; 2048 x 4096
    // would be 1.7 us faster with one, 16384 x 2048 3 us with three.
    const long long groups = (rows + sets - 1) / sets, most = 256LL * (1024 / p.threads < 4 ? 1024 / p.threads : 4);
    return {(int)(groups < most ? groups : most), p.lanes ? width : p.u * (dtype == F32 ? 4 : 8) * p.threads};
}

hipError_t launch_norm_back(int dtype, const NormBackArgs &a, const NormBackPlan &plan, float *grad_weight, hipStream_t s) {
    const RowPlan p = plan_row(dtype, a.r.width);
    hipError_t e = hipSuccess;
    if (plan.groups)
        e = dispatch_rows(dtype, p, a.r.width, [&](auto dt, auto u, auto l, auto tiny) {
            return launch(norm_back_kernel<dt.value, u.value, l.value, tiny.value>, dim3((unsigned)plan.groups),
                          dim3((unsigned)p.threads), 0, s, a);
        });
    if (e == hipSuccess && grad_weight)
        e = launch(norm_weight_kernel, dim3((unsigned)((plan.width + 63) / 64)), dim3(64 * kWeightSlices), 0, s, (const float *)a.part,
                   plan.groups, plan.width, p.threads, p.lanes ? 0 : dtype == F32 ? 1 : 2, a.r.width, grad_weight);
    return e;
}

}  // namespace ar
