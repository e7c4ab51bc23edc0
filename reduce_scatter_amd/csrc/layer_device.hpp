// layer_device.hpp -- device-side building blocks of the operators around a
// step's collectives: runs of K columns per lane, in fp32, read and written as
// vectors at any element alignment, and sums over the lanes that share a row.
//
// A run is the 16 bytes that one lane's store of the widest type involved takes
// (8 columns of 16-bit elements, 4 where fp32 is written), so that the lanes of
// a store instruction fill whole lines: with 8 fp32 columns to a lane, in two
// stores that leave every other 16 bytes out, zeros were written at 2.2 TB/s
// instead of 5.0.
#pragma once

#include "layer_kernels.hpp"
#include "vocab_device.hpp"

namespace ar {

typedef unsigned int u32x2e __attribute__((ext_vector_type(2), aligned(1)));   // 8 bytes at any alignment
typedef unsigned int u32e __attribute__((aligned(1)));                         // 4 bytes at any alignment

// K elements as stored.
template <int DT, int K> struct Run {
    static constexpr int W = K * elem_bytes<DT>() / 4;
    static_assert(W == 2 || W == 4 || W == 8, "8, 16 or 32 bytes");
    uint32_t w[W];
};

template <int DT, int K, bool STREAM = true> __device__ __forceinline__ Run<DT, K> load_run(const char *p) {
    Run<DT, K> o;
    if constexpr (o.W == 2) {
        const u32x2e v = STREAM ? __builtin_nontemporal_load((const u32x2e *)p) : *(const u32x2e *)p;
        o.w[0] = v[0], o.w[1] = v[1];
    } else {
#pragma unroll
        for (int i = 0; i < o.W; i += 4) {
            const u32x4e *q = (const u32x4e *)p + i / 4;
            const u32x4e v = STREAM ? __builtin_nontemporal_load(q) : *q;
#pragma unroll
            for (int j = 0; j < 4; ++j) o.w[i + j] = v[j];
        }
    }
    return o;
}

// Fewer than K elements (`left`), zeros behind them.
template <int DT, int K> __device__ __forceinline__ Run<DT, K> load_short(const char *p, int left) {
    Run<DT, K> o;
#pragma unroll
    for (int i = 0; i < o.W; ++i) o.w[i] = 0;
#pragma unroll
    for (int i = 0; i < K; ++i)
        if (i < left) {
            if constexpr (DT == F32) o.w[i] = ((const uint32_t *)p)[i];
            else o.w[i / 2] |= (uint32_t)((const uint16_t *)p)[i] << (16 * (i % 2));
        }
    return o;
}

template <int DT, int K> __device__ __forceinline__ void widen(const Run<DT, K> &o, float *v) {
#pragma unroll
    for (int i = 0; i < o.W; ++i) {
        if constexpr (DT == F32) {
            v[i] = bits_f32(o.w[i]);
        } else if constexpr (DT == BF16) {
            v[2 * i] = bits_f32(o.w[i] << 16);
            v[2 * i + 1] = bits_f32(o.w[i] & 0xffff0000u);
        } else {
            v[2 * i] = (float)__builtin_bit_cast(_Float16, (uint16_t)(o.w[i] & 0xffffu));
            v[2 * i + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(o.w[i] >> 16));
        }
    }
}

// K values rounded once, to nearest even, to the storage type.
template <int DT, int K> __device__ __forceinline__ Run<DT, K> narrow(const float *v) {
    Run<DT, K> o;
#pragma unroll
    for (int i = 0; i < o.W; ++i) {
        if constexpr (DT == F32) {
            o.w[i] = f32_bits(v[i]);
        } else {
            const f32x2 f = {fence_value(v[2 * i]), fence_value(v[2 * i + 1])};
            if constexpr (DT == BF16) o.w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
            else o.w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, f16x2));
        }
    }
    return o;
}

// The first `left` elements (all from K on, none up to 0).
template <int DT, int K, bool STREAM = true> __device__ __forceinline__ void store_run(char *p, const Run<DT, K> &o, int left) {
    if (left >= K) {
        if constexpr (Run<DT, K>::W == 2) {
            const u32x2e v = {o.w[0], o.w[1]};
            if constexpr (STREAM) __builtin_nontemporal_store(v, (u32x2e *)p);
            else *(u32x2e *)p = v;
        } else {
#pragma unroll
            for (int i = 0; i < o.W; i += 4) {
                const u32x4e v = {o.w[i], o.w[i + 1], o.w[i + 2], o.w[i + 3]};
                if constexpr (STREAM) __builtin_nontemporal_store(v, (u32x4e *)p + i / 4);
                else *((u32x4e *)p + i / 4) = v;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < K - 1; ++i)
            if (i < left) {
                if constexpr (DT == F32) ((uint32_t *)p)[i] = o.w[i];
                else ((uint16_t *)p)[i] = (uint16_t)(o.w[i / 2] >> (16 * (i % 2)));
            }
    }
}

// v[i] = v[i + k], zeros from the end on (k >= 0).
template <int K> __device__ __forceinline__ void shift_down(float *v, int k) {
#pragma unroll
    for (int b = K / 2; b >= 1; b /= 2) {
        const bool on = k & b;
#pragma unroll
        for (int i = 0; i < K; ++i) v[i] = on ? (i + b < K ? v[i + b] : 0.0f) : v[i];
    }
    if (k >= K) {
#pragma unroll
        for (int i = 0; i < K; ++i) v[i] = 0.0f;
    }
}

// Where a lane's run stands in its row.  A short last run, and one behind the
// row's end, is read as the row's last K columns and moved into place, so that
// no lane leaves the vector path; rows of fewer than eight columns (TINY) are
// read by the element.
struct ColPlace {
    int col, at, left;                 // first column, the column read from, columns from col on
};
template <int K, bool TINY> __device__ __forceinline__ ColPlace col_place(int run, int width) {
    ColPlace p;
    p.col = run * K;
    p.left = width - p.col;
    p.at = TINY ? 0 : (p.left >= K ? p.col : width - K);
    return p;
}
template <int DT, int K, bool TINY, bool STREAM = true>
__device__ __forceinline__ Run<DT, K> load_at(const char *row, const ColPlace &p) {
    if constexpr (TINY) return load_short<DT, K>(row + (p.left > 0 ? p.col * elem_bytes<DT>() : 0), p.left);
    else return load_run<DT, K, STREAM>(row + (long long)p.at * elem_bytes<DT>());
}
// Into place, and zeros behind the row's end.
template <int K, bool TINY> __device__ __forceinline__ void settle(float *v, const ColPlace &p) {
    if constexpr (!TINY)
        if (p.left < K) shift_down<K>(v, p.col - p.at);
}

// Sum (largest bits) over the LANES lanes of a row within a wave.
template <int LANES, typename F> __device__ __forceinline__ void row_bits(F f) {
    f(std::integral_constant<int, 1>{});
    f(std::integral_constant<int, 2>{});
    f(std::integral_constant<int, 4>{});
    f(std::integral_constant<int, 8>{});
    if constexpr (LANES >= 64) {
        f(std::integral_constant<int, 16>{});
        f(std::integral_constant<int, 32>{});
    }
}
template <int LANES> __device__ __forceinline__ float lanes_sum(float v, int lane) {
    row_bits<LANES>([&](auto m) { v += bits_f32(lane_xor<m.value>(f32_bits(v), lane)); });
    return v;
}
template <int LANES> __device__ __forceinline__ double lanes_sum(double v, int lane) {
    row_bits<LANES>([&](auto m) {
        const uint64_t u = __builtin_bit_cast(uint64_t, v);
        const uint64_t o = (uint64_t)lane_xor<m.value>((uint32_t)(u >> 32), lane) << 32 | lane_xor<m.value>((uint32_t)u, lane);
        v += __builtin_bit_cast(double, o);
    });
    return v;
}
template <int LANES> __device__ __forceinline__ uint32_t lanes_max(uint32_t v, int lane) {
    row_bits<LANES>([&](auto m) {
        const uint32_t o = lane_xor<m.value>(v, lane);
        v = o > v ? o : v;
    });
    return v;
}

}  // namespace ar
