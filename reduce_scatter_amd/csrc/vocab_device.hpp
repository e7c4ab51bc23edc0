// vocab_device.hpp -- device-side building blocks of the vocabulary-split
// reductions: the tile walk over a row's rank buffers, the running softmax
// statistics, their merge across lanes, waves and workgroups, and the top-k
// selection.
//
// Statistics are kept in units of log2: with c = log2(e) / T and a reference
// logit m, t = x*c - y, y = m*c rounded once, is one fused multiply-add per
// logit and 2^t one instruction; the rounding of y is the same for every
// logit and cancels in every result, because results only use t and the sum
// relative to the same y.  A lane's reference moves only when a tile's
// maximum exceeds it by more than 8 / c (a factor 2^8, far from overflow in
// fp32), so the rescaling multiply is rare and the sums lose nothing.
#pragma once

#include "ar_device.hpp"
#include "vocab_kernels.hpp"

namespace ar {

typedef unsigned int u32x4e __attribute__((ext_vector_type(4), aligned(2)));   // 16 bytes at element alignment
typedef unsigned long long u64;

constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kTLow = -1e6f;         // stands for lower t (2^t = 0 far above it) where t multiplies 2^t: 0 * -inf is NaN

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ bool finite(float x) { return __builtin_fabsf(x) < __builtin_huge_valf(); }

// The reference of a set of logits.  y stands for m*c; m = -inf (nothing but
// masked logits so far) counts from 0.  Where m is so large that m*c
// overflows, t is computed from x - m instead (`wide`).
struct Ref {
    float m, y;
    bool wide;
};
__device__ __forceinline__ Ref make_ref(float m, float c) {
    Ref r;
    r.m = m;
    r.y = m == kNegInf ? 0.0f : m * c;
    r.wide = finite(m) && !finite(r.y);
    return r;
}
__device__ __forceinline__ float rel(float x, const Ref &r, float c) {
    return r.wide ? (x - r.m) * c : __builtin_fmaf(x, c, -r.y);
}
// (x - m) / T in natural units, also where the larger number in units of log2 overflows.
__device__ __forceinline__ float rel_ln(float x, const Ref &r, float c, float inv_t) {
    const float t = rel(x, r, c);
    return finite(t) ? kLn2 * t : (x - r.m) * inv_t;
}
// log2 of the factor that takes sums relative to `from` to reference `to` (to.m >= from.m).
__device__ __forceinline__ float ref_shift(const Ref &from, const Ref &to, float c) {
    if (from.m == to.m) return 0.0f;
    if (from.m == kNegInf) return kNegInf;
    return (from.wide || to.wide) ? (from.m - to.m) * c : from.y - to.y;
}

// Sums of 2^t and t*2^t, and where the sums stand.
struct Stats {
    float m, s, s1;
};
__device__ __forceinline__ void shift_stats(Stats &a, float to, float c) {
    const float d = ref_shift(make_ref(a.m, c), make_ref(to, c), c);
    const float f = exp2_fast(d);
    a.s1 = f == 0.0f ? 0.0f : f * __builtin_fmaf(a.s, d, a.s1);
    a.s *= f;
    a.m = to;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int o = 32; o; o >>= 1) v = __builtin_fmaxf(v, __shfl_xor(v, o));
    return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// Every lane's statistics joined over the wave (all lanes get the result).
template <bool S1> __device__ __forceinline__ void wave_stats(Stats &a, float c) {
    shift_stats(a, wave_max(a.m), c);
    a.s = wave_sum(a.s);
    if constexpr (S1) a.s1 = wave_sum(a.s1);
}

// Joined over the workgroup's waves, in wave order; `lds` holds kVocabWaves
// entries and may be reused after the next barrier.
template <bool S1> __device__ __forceinline__ void block_stats(Stats &a, Stats *lds, int waves, int wave, int lane, float c) {
    wave_stats<S1>(a, c);
    if (waves == 1) return;
    if (lane == 0) lds[wave] = a;
    __syncthreads();
    Stats r = lds[0];
    float m = r.m;
    for (int w = 1; w < waves; ++w) m = __builtin_fmaxf(m, lds[w].m);
    shift_stats(r, m, c);
    for (int w = 1; w < waves; ++w) {
        Stats b = lds[w];
        shift_stats(b, m, c);
        r.s += b.s;
        r.s1 += b.s1;
    }
    a = r;
}

// ---- the tile walk --------------------------------------------------------
template <int DT> constexpr int elem_bytes() { return DT == F32 ? 4 : 2; }
template <int DT> constexpr int kTileElems = 64 * kVocabU * Lanes<DT>::value;

template <int DT, int NR> __device__ __forceinline__ int width_of(const VocabGeom<NR> &g, int s) {
    return g.col0[s + 1] - g.col0[s];
}
template <int DT, int NR> __device__ __forceinline__ int tiles_of(const VocabGeom<NR> &g, int s) {
    return (width_of<DT>(g, s) + kTileElems<DT> - 1) / kTileElems<DT>;
}

// Tile t as a rank and a tile within it; s == n past the last tile.
struct TileWalk {
    int s, j;
    template <int DT, int NR> __device__ __forceinline__ void settle(const VocabGeom<NR> &g) {
        while (s < g.n) {
            const int k = tiles_of<DT>(g, s);
            if (j < k) break;
            j -= k;
            ++s;
        }
    }
};

template <int DT, int NR> __device__ __forceinline__ const char *row_of(const VocabGeom<NR> &g, int s, long long row) {
    return g.x[s] + row * (long long)g.pitch[s] * elem_bytes<DT>();
}
template <int DT, int NR> __device__ __forceinline__ char *grad_row_of(const VocabGeom<NR> &g, int s, long long row) {
    return g.g[s] + row * (long long)g.gpitch[s] * elem_bytes<DT>();
}

// First element (within the rank) of vector u of this lane in tile j.
template <int DT> __device__ __forceinline__ int elem0(int j, int u, int lane) {
    return ((j * kVocabU + u) * 64 + lane) * Lanes<DT>::value;
}

// A tile's logits; past the rank's width -inf.  `w` is the rank's width.
template <int DT> struct Tile {
    Pack<DT> v[kVocabU];
};
template <int DT> __device__ __forceinline__ void load_tile(Tile<DT> &t, const char *x, int j, int w, int lane) {
    constexpr int K = Lanes<DT>::value;
    if ((j + 1) * kTileElems<DT> <= w) {
        u32x4 raw[kVocabU];
#pragma unroll
        for (int u = 0; u < kVocabU; ++u)
            raw[u] = *(const u32x4e *)(x + (uint32_t)elem0<DT>(j, u, lane) * elem_bytes<DT>());
#pragma unroll
        for (int u = 0; u < kVocabU; ++u) t.v[u] = unpack<DT>(raw[u]);
    } else {
#pragma unroll
        for (int u = 0; u < kVocabU; ++u) {
            const int e0 = elem0<DT>(j, u, lane);
            if (e0 + K <= w) t.v[u] = unpack<DT>(*(const u32x4e *)(x + (uint32_t)e0 * elem_bytes<DT>()));
            else {
#pragma unroll
                for (int i = 0; i < K; ++i) t.v[u].v[i] = e0 + i < w ? load1<DT>(x, e0 + i) : kNegInf;
            }
        }
    }
}

// A vector of gradients, rounded to the logits' type.
template <int DT> __device__ __forceinline__ u32x4 round_pack(const Pack<DT> &p) {
    u32x4 w;
    if constexpr (DT == F32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = f32_bits(p.v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x2 v = {fence_value(p.v[2 * i]), fence_value(p.v[2 * i + 1])};
            if constexpr (DT == BF16) w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
            else w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
        }
    }
    return w;
}
template <int DT> __device__ __forceinline__ void store_vec(char *g, const Pack<DT> &p, int e0, int w) {
    constexpr int K = Lanes<DT>::value;
    if (e0 + K <= w) {
        __builtin_nontemporal_store(round_pack<DT>(p), (u32x4e *)(g + (uint32_t)e0 * elem_bytes<DT>()));
    } else {
#pragma unroll
        for (int i = 0; i < K; ++i)
            if (e0 + i < w) store1<DT>(g, e0 + i, round_to<DT>(p.v[i]));
    }
}

// Column id's rank: ranks of no columns are passed over.
template <int NR> __device__ __forceinline__ int rank_of(const VocabGeom<NR> &g, int id) {
    int s = 0;
    for (int r = 0; r + 1 < g.n; ++r) s += id >= g.col0[r + 1];
    return s;
}
template <int DT, int NR> __device__ __forceinline__ float logit_at(const VocabGeom<NR> &g, long long row, int id) {
    const int s = rank_of(g, id);
    return load1<DT>(row_of<DT>(g, s, row), id - g.col0[s]);
}

// The tile, vector, lane and element that hold column id.
struct Place {
    int t, u, lane, i;
};
template <int DT, int NR> __device__ __forceinline__ Place place_of(const VocabGeom<NR> &g, int id) {
    constexpr int K = Lanes<DT>::value;
    int s = 0, t = 0;
    for (int r = 0; r + 1 < g.n; ++r) {
        const bool past = id >= g.col0[r + 1];
        s += past;
        t += past ? tiles_of<DT>(g, r) : 0;
    }
    const int e = id - g.col0[s], c = e / K;
    return {t + c / (64 * kVocabU), (c / 64) % kVocabU, c % 64, e % K};
}

// Move a lane's reference to cover a tile whose maximum is tm.
__device__ __forceinline__ void rebase(Stats &a, Ref &r, float &limit, float tm, float c, float slack) {
    if (tm > limit) {
        shift_stats(a, tm, c);
        r = make_ref(tm, c);
        limit = tm + slack;
    }
}

// Add one vector's logits to a lane's sums.
template <int DT, bool S1> __device__ __forceinline__ void add_vec(Stats &a, const Ref &r, const Pack<DT> &v, float c) {
#pragma unroll
    for (int i = 0; i < Lanes<DT>::value; ++i) {
        const float t = __builtin_fmaf(v.v[i], c, -r.y);
        const float e = exp2_fast(t);
        a.s += e;
        if constexpr (S1) a.s1 = __builtin_fmaf(e, __builtin_fmaxf(t, kTLow), a.s1);
    }
}
template <int DT, bool S1> __device__ __forceinline__ void add_vec_wide(Stats &a, const Ref &r, const Pack<DT> &v, float c) {
#pragma unroll
    for (int i = 0; i < Lanes<DT>::value; ++i) {
        const float t = rel(v.v[i], r, c);
        const float e = exp2_fast(t);
        a.s += e;
        if constexpr (S1) a.s1 = __builtin_fmaf(e, __builtin_fmaxf(t, kTLow), a.s1);
    }
}
template <int DT> __device__ __forceinline__ float vec_max(const Pack<DT> &v) {
    float m = v.v[0];
#pragma unroll
    for (int i = 1; i < Lanes<DT>::value; ++i) m = __builtin_fmaxf(m, v.v[i]);
    return m;
}
template <int DT, bool S1> __device__ __forceinline__ void add_tile(Stats &a, Ref &r, float &limit, const Tile<DT> &t,
                                                                    float tm, float c, float slack) {
    if (__any(tm > limit)) rebase(a, r, limit, tm, c, slack);
    if (__any(r.wide)) {
#pragma unroll
        for (int u = 0; u < kVocabU; ++u) add_vec_wide<DT, S1>(a, r, t.v[u], c);
    } else {
#pragma unroll
        for (int u = 0; u < kVocabU; ++u) add_vec<DT, S1>(a, r, t.v[u], c);
    }
}

// ---- top-k ----------------------------------------------------------------
// Logits are ordered by 64-bit keys: the value's order-preserving bits, then
// the complement of the column (equal values: lowest column first).  -0
// counts as +0 and NaN as -inf; key 0 is "nothing".
__device__ __forceinline__ uint32_t order_bits(float x) {
    x = x == x ? x + 0.0f : kNegInf;
    const uint32_t u = f32_bits(x);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t o) {
    return bits_f32(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ u64 top_key(float x, int col) { return (u64)order_bits(x) << 32 | (uint32_t)~col; }
__device__ __forceinline__ int key_col(u64 k) { return (int)~(uint32_t)k; }

__device__ __forceinline__ u64 shfl_xor64(u64 v, int mask) {
    const uint32_t lo = __shfl_xor((uint32_t)v, mask), hi = __shfl_xor((uint32_t)(v >> 32), mask);
    return (u64)hi << 32 | lo;
}
__device__ __forceinline__ u64 cmp_exchange(u64 v, int mask, bool keep_max) {
    const u64 o = shfl_xor64(v, mask);
    return (o > v) == keep_max ? o : v;
}
// A bitonic sequence over the 64 lanes into descending order.
__device__ __forceinline__ u64 merge_down(u64 v, int lane) {
#pragma unroll
    for (int j = 32; j; j >>= 1) v = cmp_exchange(v, j, !(lane & j));
    return v;
}
__device__ __forceinline__ u64 sort_down(u64 v, int lane) {
#pragma unroll
    for (int k = 2; k < 64; k <<= 1)
#pragma unroll
        for (int j = k >> 1; j; j >>= 1) v = cmp_exchange(v, j, !(lane & j) == !(lane & k));
    return merge_down(v, lane);
}
// The 64 largest of two descending lists, descending: lane i keeps the larger
// of a[i] and b[63 - i], which is a bitonic sequence.
__device__ __forceinline__ u64 merge_lists(u64 a, u64 b_reversed, int lane) {
    return merge_down(a > b_reversed ? a : b_reversed, lane);
}
__device__ __forceinline__ u64 reversed(u64 v, int lane) { return shfl_xor64(v, 63); }

// The 64 largest of every wave's descending list, in all waves.  `lds` holds
// waves * 64 keys.
__device__ __forceinline__ u64 block_lists(u64 v, u64 *lds, int waves, int wave, int lane) {
    if (waves == 1) return v;
    __syncthreads();                                          // earlier readers of lds are done
    lds[wave * 64 + lane] = v;
    __syncthreads();
    for (int r = waves >> 1; r; r >>= 1) {
        if (wave < r) {
            v = merge_lists(v, lds[(wave + r) * 64 + 63 - lane], lane);
            lds[wave * 64 + lane] = v;
        }
        __syncthreads();
    }
    return lds[lane];
}

}  // namespace ar
