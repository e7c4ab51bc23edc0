// layer_device.hpp -- device-side building blocks of the operators around a
// step's collectives: runs of eight columns ("octs") in fp32, read and written
// as 16-byte vectors at any element alignment, and sums over the lanes that
// share a row.
#pragma once

#include "layer_kernels.hpp"
#include "vocab_device.hpp"

namespace ar {

typedef unsigned int u32x2e __attribute__((ext_vector_type(2), aligned(1)));   // 8 bytes at any alignment

// Eight elements as stored.
template <int DT> struct Oct {
    u32x4 w[DT == F32 ? 2 : 1];
};

template <int DT, bool STREAM = true> __device__ __forceinline__ Oct<DT> load_oct(const char *p) {
    Oct<DT> o;
    const u32x4e *q = (const u32x4e *)p;
#pragma unroll
    for (int i = 0; i < (DT == F32 ? 2 : 1); ++i) o.w[i] = STREAM ? __builtin_nontemporal_load(q + i) : q[i];
    return o;
}

// Fewer than eight elements (`left`), zeros behind them.
template <int DT> __device__ __forceinline__ Oct<DT> load_short(const char *p, int left) {
    Oct<DT> o;
#pragma unroll
    for (int i = 0; i < (DT == F32 ? 2 : 1); ++i) o.w[i] = u32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) {
            if constexpr (DT == F32) o.w[i / 4][i % 4] = ((const uint32_t *)p)[i];
            else o.w[0][i / 2] |= (uint32_t)((const uint16_t *)p)[i] << (16 * (i % 2));
        }
    return o;
}

template <int DT> __device__ __forceinline__ void widen(const Oct<DT> &o, float *v) {
    constexpr int K = Pack<DT>::K;
#pragma unroll
    for (int j = 0; j < 8 / K; ++j) {
        const Pack<DT> p = unpack<DT>(o.w[j]);
#pragma unroll
        for (int i = 0; i < K; ++i) v[j * K + i] = p.v[i];
    }
}

// Eight values rounded once, to nearest even, to the storage type.
template <int DT> __device__ __forceinline__ Oct<DT> narrow(const float *v) {
    Oct<DT> o;
    constexpr int K = Pack<DT>::K;
#pragma unroll
    for (int j = 0; j < 8 / K; ++j) {
        if constexpr (DT == F32) {
#pragma unroll
            for (int i = 0; i < 4; ++i) o.w[j][i] = f32_bits(v[4 * j + i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x2 f = {fence_value(v[2 * i]), fence_value(v[2 * i + 1])};
                if constexpr (DT == BF16) o.w[j][i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
                else o.w[j][i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, f16x2));
            }
        }
    }
    return o;
}

// The first `left` elements (all eight from 8 on, none up to 0).
template <int DT, bool STREAM = true> __device__ __forceinline__ void store_oct(char *p, const Oct<DT> &o, int left) {
    if (left >= 8) {
        u32x4e *q = (u32x4e *)p;
#pragma unroll
        for (int i = 0; i < (DT == F32 ? 2 : 1); ++i) {
            if constexpr (STREAM) __builtin_nontemporal_store((u32x4e)o.w[i], q + i);
            else q[i] = o.w[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < left) {
                if constexpr (DT == F32) ((uint32_t *)p)[i] = o.w[i / 4][i % 4];
                else ((uint16_t *)p)[i] = (uint16_t)(o.w[0][i / 2] >> (16 * (i % 2)));
            }
    }
}

// v[i] = v[i + k], zeros from the end on (k >= 0).
__device__ __forceinline__ void shift_down(float *v, int k) {
#pragma unroll
    for (int b = 4; b >= 1; b /= 2) {
        const bool on = k & b;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = on ? (i + b < 8 ? v[i + b] : 0.0f) : v[i];
    }
    if (k >= 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    }
}

// Where a lane's oct stands in its row.  A short last oct, and one behind the
// row's end, is read as the row's last eight columns and moved into place, so
// that no lane leaves the vector path; rows of fewer than eight columns (TINY)
// are read by the element.
struct ColPlace {
    int col, at, left;                 // first column, the column read from, columns from col on
};
template <bool TINY> __device__ __forceinline__ ColPlace col_place(int oct, int width) {
    ColPlace p;
    p.col = oct * 8;
    p.left = width - p.col;
    p.at = TINY ? 0 : (p.left >= 8 ? p.col : width - 8);
    return p;
}
template <int DT, bool TINY, bool STREAM = true>
__device__ __forceinline__ Oct<DT> load_at(const char *row, const ColPlace &p) {
    if constexpr (TINY) return load_short<DT>(row, p.col == 0 ? p.left : 0);
    else return load_oct<DT, STREAM>(row + (long long)p.at * elem_bytes<DT>());
}
// Into place, and zeros behind the row's end.
template <bool TINY> __device__ __forceinline__ void settle(float *v, const ColPlace &p) {
    if constexpr (!TINY)
        if (p.left < 8) shift_down(v, p.col - p.at);
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
