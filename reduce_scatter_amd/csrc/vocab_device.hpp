// vocab_device.hpp -- device-side building blocks of the vocabulary-split
// reductions: the tile walk over a row's rank buffers, the running softmax
// statistics, their merge across lanes, waves and workgroups, and the top-k
// selection.
//
// Statistics are kept in units of log2: with c = log2(e) / T and a reference
// logit m, t = x*c - y, y = m*c rounded once, is one fused multiply-add per
// logit and 2^t one instruction; the rounding of y is the same for every
// logit, so sums stand against y as they are joined, and a row's whole sums are
// taken to m itself (settled) before any result or gradient uses them.  The
// reference need not be the maximum: a lane takes its first vector's and keeps
// it while a tile's sum stays below 2^16, so the stream takes no maxima; a
// vector that carries the sum past that is added again after moving the
// reference.
#pragma once

#include "ar_device.hpp"
#include "vocab_kernels.hpp"

namespace ar {

typedef unsigned int u32x4e __attribute__((ext_vector_type(4), aligned(2)));   // 16 bytes at element alignment
typedef unsigned long long u64;

constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kTLow = -1e6f;         // stands for lower t (2^t = 0 far above it) where t multiplies 2^t: 0 * -inf is NaN
constexpr float kWide = 0x1p30f;       // see make_ref

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ bool finite(float x) { return __builtin_fabsf(x) < __builtin_huge_valf(); }

// The reference of a set of logits: t = x*c - y.  m = -inf (nothing but masked
// logits) counts from 0.  For x = m that leaves t = residue(), what rounding y
// took away: up to half a unit in the last place of m*c.  That is no more than
// 32 while |m*c| is below 2^30, but hundreds and more beyond (masks of -1e10,
// or any logit at a temperature near 0), infinity or zero to 2^t.  From 2^30 on
// c therefore is the power of two that puts |m| c into [2^30, 2^31): the
// product is exact, t = 0 at x = m, and any other number is a unit in m's last
// place away, 2^6 at least in t under either scale, where 2^t counts for
// nothing beside 1 (2^20 columns of it are 2^-44).
struct Ref {
    float m, y, c;
    bool wide;                         // c is that power of two instead of log2(e) / T
};
__device__ __forceinline__ Ref make_ref(float m, float c) {
    Ref r;
    r.m = m;
    r.c = c;
    r.y = m == kNegInf ? 0.0f : m * c;
    r.wide = finite(m) && __builtin_fabsf(r.y) >= kWide;
    if (r.wide) {
        r.c = __builtin_amdgcn_ldexpf(1.0f, 31 - __builtin_amdgcn_frexp_expf(m));
        r.y = m * r.c;
    }
    return r;
}
__device__ __forceinline__ float rel(float x, const Ref &r) { return __builtin_fmaf(x, r.c, -r.y); }
// t at x = m: what rounding y took away, exactly.
__device__ __forceinline__ float residue(const Ref &r) {
    return r.wide || r.m == kNegInf ? 0.0f : __builtin_fmaf(r.m, r.c, -r.y);
}
// (x - m) / T in natural units and in units of log2, also where t overflows or has the other scale.
__device__ __forceinline__ float rel_ln(float x, const Ref &r, float inv_t) {
    const float t = rel(x, r);
    return finite(t) && !r.wide ? kLn2 * (t - residue(r)) : (x - r.m) * inv_t;
}
__device__ __forceinline__ float rel_log2(float x, const Ref &r, float c) {
    const float t = rel(x, r);
    return finite(t) && !r.wide ? t - residue(r) : (x - r.m) * c;
}
// log2 of the factor that takes sums relative to `from` to reference `to` (to.m >= from.m).
__device__ __forceinline__ float ref_shift(const Ref &from, const Ref &to, float c) {
    if (from.m == to.m) return 0.0f;
    if (from.m == kNegInf) return kNegInf;
    return from.wide || to.wide ? (from.m - to.m) * c + (residue(to) - residue(from)) : from.y - to.y;
}

// Sums of 2^t and t*2^t, and where the sums stand.
struct Stats {
    float m, s, s1;
};
// To the reference logit `to`, d = log2 of the factor f.
__device__ __forceinline__ void shift_by(Stats &a, float to, float d, float f) {
    a.s1 = f == 0.0f ? 0.0f : f * __builtin_fmaf(a.s, d, a.s1);
    a.s *= f;
    a.m = to;
}
// ref_shift without making the references, unless some lane's is wide.
__device__ __forceinline__ void shift_stats(Stats &a, float to, float c) {
    const float from_y = a.m * c, to_y = to * c;
    const bool wide = (finite(a.m) && __builtin_fabsf(from_y) >= kWide) ||
                      (finite(to) && __builtin_fabsf(to_y) >= kWide);
    float d = a.m == to ? 0.0f : from_y - to_y;
    if (__builtin_expect(__any(wide), 0)) d = ref_shift(make_ref(a.m, c), make_ref(to, c), c);
    shift_by(a, to, d, exp2_fast(d));
}

// A row's whole sums relative to its reference logit m instead of y: what rel_ln
// and the fp32 terms (term) count from, and what a caller is given.
__device__ __forceinline__ Stats settled(const Stats &a, float c) {
    const float r = residue(make_ref(a.m, c)), f = exp2_fast(-r);
    return Stats{a.m, a.s * f, __builtin_fmaf(a.s, -r, a.s1) * f};
}

// The value of lane (lane ^ M): data-parallel moves within rows of 16 lanes,
// gfx950's row swaps across them; none goes through LDS.
template <int CTRL> __device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
template <int M> __device__ __forceinline__ uint32_t lane_xor(uint32_t v, int lane) {
    static_assert(M == 1 || M == 2 || M == 4 || M == 8 || M == 16 || M == 32, "one bit");
    if constexpr (M == 1) return dpp<0xB1>(v);                          // quad_perm 1 0 3 2
    else if constexpr (M == 2) return dpp<0x4E>(v);                     // quad_perm 2 3 0 1
    else if constexpr (M == 4) return dpp<0x1B>(dpp<0x141>(v));         // half-row mirror (^7), then ^3
    else if constexpr (M == 8) return dpp<0x128>(v);                    // row rotate by 8
    else {
        // the swaps exchange odd rows (halves) of one register with even rows (halves) of the other
        if constexpr (M == 16) {
            const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
            return lane & 16 ? r[0] : r[1];
        } else {
            const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
            return lane & 32 ? r[0] : r[1];
        }
    }
}
// The bits 1, 2, ..., 32 in turn, as compile-time constants.
template <typename F> __device__ __forceinline__ void each_bit(F f) {
    f(std::integral_constant<int, 1>{});
    f(std::integral_constant<int, 2>{});
    f(std::integral_constant<int, 4>{});
    f(std::integral_constant<int, 8>{});
    f(std::integral_constant<int, 16>{});
    f(std::integral_constant<int, 32>{});
}
__device__ __forceinline__ float wave_max(float v, int lane) {
    each_bit([&](auto m) { v = __builtin_fmaxf(v, bits_f32(lane_xor<m.value>(f32_bits(v), lane))); });
    return v;
}
__device__ __forceinline__ float wave_sum(float v, int lane) {
    each_bit([&](auto m) { v += bits_f32(lane_xor<m.value>(f32_bits(v), lane)); });
    return v;
}

// Every lane's statistics joined over the wave (all lanes get the result).
template <bool S1> __device__ __forceinline__ void wave_stats(Stats &a, int lane, float c) {
    shift_stats(a, wave_max(a.m, lane), c);
    a.s = wave_sum(a.s, lane);
    if constexpr (S1) a.s1 = wave_sum(a.s1, lane);
}

// Joined over the workgroup's waves; `lds` holds kVocabWaves entries and may
// be reused after the next barrier.
template <bool S1> __device__ __forceinline__ void block_stats(Stats &a, Stats *lds, int waves, int wave, int lane, float c) {
    wave_stats<S1>(a, lane, c);
    if (waves == 1) return;
    if (lane == 0) lds[wave] = a;
    __syncthreads();
    a = lane < waves ? lds[lane] : Stats{kNegInf, 0.0f, 0.0f};
    wave_stats<S1>(a, lane, c);
}

// ---- the tile walk --------------------------------------------------------
template <int DT> constexpr int elem_bytes() { return DT == F32 ? 4 : 2; }
template <int DT> constexpr int kTileElems = 64 * kVocabU * Lanes<DT>::value;

template <int DT, int NR> __device__ __forceinline__ int width_of(const VocabGeom<NR> &g, int s) {
    return g.col0[s + 1] - g.col0[s];
}
template <int DT, int NR> __device__ __forceinline__ int tiles_of(const VocabGeom<NR> &g, int s) {
    const int w = width_of<DT>(g, s);
    return w ? (w + g.skew + kTileElems<DT> - 1) / kTileElems<DT> : 0;
}

template <int DT, int NR> __device__ __forceinline__ const char *row_of(const VocabGeom<NR> &g, int s, long long row) {
    return g.x[s] + row * (long long)g.pitch[s] * elem_bytes<DT>();
}
template <int DT, int NR> __device__ __forceinline__ char *grad_row_of(const VocabGeom<NR> &g, int s, long long row) {
    return g.g[s] + row * (long long)g.gpitch[s] * elem_bytes<DT>();
}

template <int NR> constexpr bool kTiny = NR > kVocabFew;
// Vectors lie on 16-byte boundaries of memory: a row that begins `phase`
// elements after one has its first vector cut short.  (Ranks of fewer columns
// than a vector, TINY, are read by the element.)
template <int DT, bool TINY> __device__ __forceinline__ int phase_of(const char *x, int w) {
    if (TINY && w < Lanes<DT>::value) return 0;
    return (int)((uintptr_t)x / elem_bytes<DT>() % Lanes<DT>::value);
}

// A wave's way through its tiles: the tile (numbered over all ranks), its
// rank, its number within the rank, and what the rank's tiles have in common.
struct TileWalk {
    int at, s, j;
    int w, tiles, col;                 // the rank's width, tiles and first column
    int phase;                         // elements from the 16-byte boundary below to the row's first
    const char *x;                     // its logits of the row

    // To the tile `by` further on; false past the last.
    template <int DT, int NR> __device__ __forceinline__ bool move(const VocabGeom<NR> &g, long long row, int by) {
        at += by;
        j += by;
        if (j < tiles) return true;
        do {
            j -= tiles;
            if (++s >= g.n) return false;
            tiles = tiles_of<DT>(g, s);
        } while (j >= tiles);
        load_rank<DT>(g, row);
        return true;
    }
    template <int DT, int NR> __device__ __forceinline__ bool start(const VocabGeom<NR> &g, long long row, int first) {
        at = s = j = 0;
        tiles = tiles_of<DT>(g, 0);
        load_rank<DT>(g, row);
        return move<DT>(g, row, first);
    }
    template <int DT, int NR> __device__ __forceinline__ void load_rank(const VocabGeom<NR> &g, long long row) {
        w = width_of<DT>(g, s);
        col = g.col0[s];
        x = row_of<DT>(g, s, row);
        phase = phase_of<DT, kTiny<NR>>(x, w);
    }
    // First element (within the rank) of vector u of a lane: below 0 where the
    // rank's first vector begins before the row does.
    template <int DT> __device__ __forceinline__ int elem0(int u, int lane) const {
        return ((j * kVocabU + u) * 64 + lane) * Lanes<DT>::value - phase;
    }
    template <int DT> __device__ __forceinline__ bool full() const {
        return j * kTileElems<DT> >= phase && (j + 1) * kTileElems<DT> - phase <= w;
    }
};

// Where register element 0 of that vector stands.  The vector covers those of
// [e0, e0 + K) that the rank has; where that is not all, its registers hold
// the rank's first or last K elements, of which some are another vector's, so
// that one unconditional in-bounds 16-byte load serves every lane of a rank of
// at least K columns.  Ranks of fewer (TINY) are served by the kernels with
// the large pointer table alone.
template <int DT, bool TINY> __device__ __forceinline__ int held0(int e0, int w) {
    constexpr int K = Lanes<DT>::value;
    if (TINY && w < K) return e0;
    return min(max(e0, 0), w - K);
}

template <int DT> __device__ __forceinline__ uint32_t neg_inf_bits() {
    return DT == F32 ? 0xff800000u : DT == BF16 ? 0xff80u : 0xfc00u;
}
// Vector u of a tile.  STREAM: the logits are not read again (non-temporal).
template <int DT, bool STREAM, bool TINY>
__device__ __forceinline__ u32x4 load_vec(const TileWalk &t, int u, int lane) {
    constexpr int K = Lanes<DT>::value;
    if constexpr (TINY) {
        if (t.w < K) {                                         // all in vector 0 of lane 0
            u32x4 v{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < K; ++i) {
                if (lane == 0 && u == 0 && i < t.w) {
                    if constexpr (DT == F32) v[i] = ((const uint32_t *)t.x)[i];
                    else v[i / 2] |= (uint32_t)((const uint16_t *)t.x)[i] << (i & 1) * 16;
                }
            }
            return v;
        }
    }
    // in bytes, from the lane's part and the wave's, so that two instructions make the address
    const int at = lane * 16 + t.elem0<DT>(u, 0) * elem_bytes<DT>();
    const u32x4e *p = (const u32x4e *)(t.x + (uint32_t)min(max(at, 0), (t.w - K) * elem_bytes<DT>()));
    if constexpr (STREAM) return __builtin_nontemporal_load(p);
    else return *p;
}
// Registers of a vector at a rank's ends that hold no element of it become -inf.
template <int DT> __device__ __forceinline__ void mask_vec(u32x4 &v, int e0, int held, int w) {
    constexpr int K = Lanes<DT>::value;
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const bool out = held + i < e0 || held + i >= e0 + K || held + i >= w;
        if constexpr (DT == F32) v[i] = out ? neg_inf_bits<DT>() : v[i];
        else {
            const uint32_t part = 0xffffu << (i & 1) * 16, ninf = neg_inf_bits<DT>() << (i & 1) * 16;
            v[i / 2] = out ? (v[i / 2] & ~part) | ninf : v[i / 2];
        }
    }
}

// A wave's vectors in order.  start() issues the loads of the first tile, so
// that what else a kernel has to read and work out runs meanwhile; run() calls
// f(walk, u, e0, held, raw) for every vector and loads one of the next tile as
// soon as the one in its registers is used up: a tile's loads stay in flight.
template <int DT, bool STREAM, int NR> struct VectorStream {
    static constexpr bool TINY = kTiny<NR>;
    TileWalk t;
    u32x4 v[kVocabU];
    bool any;
    __device__ __forceinline__ void start(const VocabGeom<NR> &g, long long row, int first, int lane) {
        any = t.start<DT>(g, row, first);
        if (!any) return;
#pragma unroll
        for (int u = 0; u < kVocabU; ++u) v[u] = load_vec<DT, STREAM, TINY>(t, u, lane);
    }
    template <typename F>
    __device__ __forceinline__ void run(const VocabGeom<NR> &g, long long row, int step, int lane, F f) {
        // The last round loads its own tile again, into registers that nothing
        // reads: without a branch around the loads the compiler knows how many
        // are in flight and waits for the oldest only.
        for (bool more = any; more;) {
            TileWalk n = t;
            more = n.move<DT>(g, row, step);
            if (!more) n = t;
#pragma unroll
            for (int u = 0; u < kVocabU; ++u) {
                const int e0 = t.elem0<DT>(u, lane);
                f(t, u, e0, held0<DT, TINY>(e0, t.w), v[u]);
                v[u] = load_vec<DT, STREAM, TINY>(n, u, lane);
            }
            t = n;
        }
    }
};

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
// Store a vector whose register 0 stands at element `held`: whole, or at a
// rank's ends only the elements that are its own.
template <int DT>
__device__ __forceinline__ void store_vec(char *g, const Pack<DT> &p, const TileWalk &t, int e0, int held) {
    constexpr int K = Lanes<DT>::value;
    if (t.full<DT>() || (e0 >= 0 && e0 + K <= t.w)) {
        __builtin_nontemporal_store(round_pack<DT>(p), (u32x4e *)(g + (uint32_t)e0 * elem_bytes<DT>()));
    } else {
#pragma unroll
        for (int i = 0; i < K; ++i)
            if (held + i >= e0 && held + i < e0 + K && held + i < t.w) store1<DT>(g, held + i, round_to<DT>(p.v[i]));
    }
}

template <int DT, int NR>
__device__ __forceinline__ void zero_tiles(const VocabGeom<NR> &g, long long row, int first, int step, int lane) {
    Pack<DT> zero;
#pragma unroll
    for (int i = 0; i < Lanes<DT>::value; ++i) zero.v[i] = 0.0f;
    TileWalk t;
    for (bool more = t.start<DT>(g, row, first); more; more = t.move<DT>(g, row, step)) {
#pragma unroll
        for (int u = 0; u < kVocabU; ++u) {
            const int e0 = t.elem0<DT>(u, lane);
            store_vec<DT>(grad_row_of<DT>(g, t.s, row), zero, t, e0, held0<DT, kTiny<NR>>(e0, t.w));
        }
    }
}

// f(r) for every rank but the first, without a loop in the kernels with the
// small table (their first columns are then loaded together).
template <int NR, typename F> __device__ __forceinline__ void each_later_rank(const VocabGeom<NR> &g, F f) {
    if constexpr (NR <= kVocabFew) {
#pragma unroll
        for (int r = 1; r < NR; ++r) f(r);
    } else {
        for (int r = 1; r < g.n; ++r) f(r);
    }
}
// Column id's rank: ranks of no columns are passed over.
template <int NR> __device__ __forceinline__ int rank_of(const VocabGeom<NR> &g, int id) {
    int s = 0;
    each_later_rank(g, [&](int r) { s += id >= g.col0[r]; });
    return s;
}
template <int DT, int NR> __device__ __forceinline__ float logit_at(const VocabGeom<NR> &g, long long row, int id) {
    const int s = rank_of(g, id);
    return load1<DT>(row_of<DT>(g, s, row), id - g.col0[s]);
}

// Column id's rank and its element there; its tile, and its element within that.
struct Place {
    int s, e, t, et;
};
template <int DT, int NR>
__device__ __forceinline__ Place place_of(const VocabGeom<NR> &g, long long row, int id) {
    int s = 0, first = 0, t = 0;
    each_later_rank(g, [&](int r) {
        const bool past = id >= g.col0[r];
        s = past ? r : s;
        first = past ? g.col0[r] : first;
        t += past ? tiles_of<DT>(g, r - 1) : 0;
    });
    const int e = id - first, at = e + phase_of<DT, kTiny<NR>>(row_of<DT>(g, s, row), width_of<DT>(g, s));
    return {s, e, t + at / kTileElems<DT>, at % kTileElems<DT>};
}

// t and 2^t of a logit for its gradient.  In units of log2 a logit far below
// the reference carries |t| 2^-24 of rounding into 2^t.  In the sums that
// averages out, and gradients of 16-bit logits are rounded to 2^-8 or 2^-11,
// so these take t relative to y (term_shift() of the reference off); for
// those of fp32 the product (x - m) c is carried in two parts (c too), which
// leaves the rounding of x - m itself.  Where x - m overflows the low
// part is no number and left out (2^t is 0 or infinity then).
struct Term {
    float t, e;
};
__device__ __forceinline__ float hold_up(float t, float least) {
    // one instruction: the builtin first quiets a signalling NaN, which no result of arithmetic is
    float r;
    asm("v_max_f32 %0, %1, %2" : "=v"(r) : "s"(least), "v"(t));
    return r;
}
template <int DT, int NR> __device__ __forceinline__ Term term(float x, const Ref &r, const VocabGeom<NR> &g) {
    Term a;
    if constexpr (DT == F32) {
        const float d = x - (r.m == kNegInf ? 0.0f : r.m);
        a.t = d * g.c;
        const float lo = __builtin_fmaf(d, g.c_low, __builtin_fmaf(d, g.c, -a.t));
        a.e = exp2_fast(a.t) * __builtin_fmaf(kLn2, __builtin_fabsf(lo) < 1.0f ? lo : 0.0f, 1.0f);
    } else {
        a.t = rel(x, r);
        a.e = exp2_fast(a.t);
    }
    return a;
}

// What t in term() is too large by: a row's factors take it away, not each logit.
template <int DT> __device__ __forceinline__ float term_shift(const Ref &r) { return DT == F32 ? 0.0f : residue(r); }

// A lane's running sums and reference: those of the tile at hand, and of the
// tiles done, which are only added up tile by tile (a lane sees thousands of
// terms, and each addition to the large sum would round it).
struct Running {
    Stats st{kNegInf, 0.0f, 0.0f};
    float done = 0.0f, done1 = 0.0f;
    Ref ref{kNegInf, 0.0f, 1.0f, false};
    int fresh = 1;                     // some lane has met no logit above -inf yet
};
__device__ __forceinline__ void end_tile(Running &a) {
    a.done += a.st.s;
    a.done1 += a.st.s1;
    a.st.s = a.st.s1 = 0.0f;
}
__device__ __forceinline__ Stats total(const Running &a) {
    return Stats{a.st.m, a.done + a.st.s, a.done1 + a.st.s1};
}
// Add one vector's logits to a lane's sums.  2^t = 0 where t = -inf, but
// 0 * -inf is NaN: t is held above kTLow in the weighted sum.
template <int DT, bool S1> __device__ __forceinline__ void add_terms(Running &a, const Pack<DT> &v) {
    constexpr int K = Lanes<DT>::value;
    float e[K], s1 = 0.0f;
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const float t = rel(v.v[i], a.ref);
        e[i] = exp2_fast(t);
        if constexpr (S1) {
            const float h = hold_up(t, kTLow);
            s1 = i ? __builtin_fmaf(e[i], h, s1) : e[i] * h;
        }
    }
#pragma unroll
    for (int h = K / 2; h; h /= 2)
#pragma unroll
        for (int i = 0; i < h; ++i) e[i] += e[i + h];
    a.st.s += e[0];
    if constexpr (S1) a.st.s1 += s1;
}
// The same after moving the references of lanes whose vector has a larger maximum.
template <int DT, bool S1, int NR>
__device__ __forceinline__ void add_with_care(Running &a, Pack<DT> v, const VocabGeom<NR> &g) {
    // other values to the compiler, which would otherwise take the first steps below for every vector
#pragma unroll
    for (int i = 0; i < Lanes<DT>::value; ++i) asm volatile("" : "+v"(v.v[i]));
    float m = v.v[0];
#pragma unroll
    for (int i = 1; i < Lanes<DT>::value; ++i) m = __builtin_fmaxf(m, v.v[i]);
    if (m > a.st.m) {
        const Ref to = make_ref(m, g.c);
        const float d = ref_shift(a.ref, to, g.c), f = exp2_fast(d);
        Stats done{a.st.m, a.done, a.done1};
        shift_by(a.st, m, d, f);
        shift_by(done, m, d, f);
        a.done = done.s;
        a.done1 = done.s1;
        a.ref = to;
    }
    a.fresh = __builtin_amdgcn_readfirstlane(__any(a.st.m == kNegInf));
    add_terms<DT, S1>(a, v);
}
// Whether what has just been added has to be added again, with care: the
// first vectors, and seldom later.
__device__ __forceinline__ bool sums_off(const Running &a) { return (__ballot(a.st.s > 65536.0f) | (u64)a.fresh) != 0; }
template <int DT, bool S1, int NR>
__device__ __forceinline__ void add_vec(Running &a, const Pack<DT> &x, const VocabGeom<NR> &g) {
    const Stats before = a.st;
    add_terms<DT, S1>(a, x);
    if (sums_off(a)) {
        a.st = before;
        add_with_care<DT, S1>(a, x, g);
    }
}

// ---- rows held in registers -------------------------------------------------
// A wave's tiles, all of them (at most T): read once for sums and gradient
// together.  Missing tiles are loaded as copies of the last one and never
// used, so that the number of loads in flight is known (see VectorStream).
template <int DT, int NR, int T> struct HeldTiles {
    static constexpr bool TINY = kTiny<NR>;
    TileWalk t[T];
    int n;
    u32x4 v[T * kVocabU];
    __device__ __forceinline__ void start(const VocabGeom<NR> &g, long long row, int first, int step, int lane) {
        t[0].template start<DT>(g, row, first);                        // a workgroup has no more waves than a row has tiles
        n = 1;
#pragma unroll
        for (int k = 0; k < T; ++k) {
            if (k) {
                t[k] = t[k - 1];
                TileWalk next = t[k];
                if (n == k && next.template move<DT>(g, row, step)) {
                    t[k] = next;
                    n = k + 1;
                }
            }
#pragma unroll
            for (int u = 0; u < kVocabU; ++u) v[k * kVocabU + u] = load_vec<DT, true, TINY>(t[k], u, lane);
        }
    }
    // f for every vector, after(k) at the end of every tile
    template <typename F, typename G> __device__ __forceinline__ void each(int lane, F f, G after) {
#pragma unroll
        for (int k = 0; k < T; ++k) {
            if (k < n) {
#pragma unroll
                for (int u = 0; u < kVocabU; ++u) {
                    // another number to the compiler, which would otherwise keep every vector's bounds from one
                    // walk to the next, in more registers than there are
                    int here = lane;
                    asm volatile("" : "+v"(here));
                    const int e0 = t[k].template elem0<DT>(u, here);
                    f(t[k], k, u, e0, held0<DT, TINY>(e0, t[k].w), v[k * kVocabU + u]);
                }
                after(k);
            }
        }
    }
    template <typename F> __device__ __forceinline__ void each(int lane, F f) {
        each(lane, f, [](int) {});
    }
};

// Sums of a wave's held tiles; prepare(k, u, e0, held, raw) may change a vector before it is first used.
template <int DT, bool S1, int NR, int T, typename F>
__device__ __forceinline__ Stats held_sums(const VocabGeom<NR> &g, HeldTiles<DT, NR, T> &h, int lane, F prepare) {
    Running a;
    h.each(
        lane,
        [&](const TileWalk &t, int k, int u, int e0, int held, u32x4 &raw) {
            asm volatile("" : "+v"(raw), "+v"(a.st.s), "+v"(a.st.s1));         // after the vector before: few values live
            if (!t.template full<DT>()) mask_vec<DT>(raw, e0, held, t.w);
            prepare(k, u, e0, held, raw);
            add_terms<DT, S1>(a, unpack<DT>(raw));
        },
        [&](int k) {
            if (sums_off(a)) {
                a.st.s = a.st.s1 = 0.0f;                       // as at the tile's start
#pragma unroll
                for (int u = 0; u < kVocabU; ++u) add_with_care<DT, S1>(a, unpack<DT>(h.v[k * kVocabU + u]), g);
            }
            end_tile(a);
        });
    return total(a);
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

template <int M> __device__ __forceinline__ u64 cmp_exchange(u64 v, int lane, bool keep_max) {
    const uint32_t lo = lane_xor<M>((uint32_t)v, lane), hi = lane_xor<M>((uint32_t)(v >> 32), lane);
    const u64 o = (u64)hi << 32 | lo;
    return (o > v) == keep_max ? o : v;
}
// A bitonic sequence over blocks of 2 * M lanes into order: descending in
// lanes where `down`.
template <int M> __device__ __forceinline__ u64 merge_steps(u64 v, int lane, bool down) {
    v = cmp_exchange<M>(v, lane, !(lane & M) == down);
    if constexpr (M > 1) v = merge_steps<M / 2>(v, lane, down);
    return v;
}
// The 64 lanes' keys in descending order.
__device__ __forceinline__ u64 sort_down(u64 v, int lane) {
    v = merge_steps<1>(v, lane, !(lane & 2));
    v = merge_steps<2>(v, lane, !(lane & 4));
    v = merge_steps<4>(v, lane, !(lane & 8));
    v = merge_steps<8>(v, lane, !(lane & 16));
    v = merge_steps<16>(v, lane, !(lane & 32));
    return merge_steps<32>(v, lane, true);
}
// The reverse of the lanes' order.
__device__ __forceinline__ u64 reversed(u64 v, int lane) {
    uint32_t lo = (uint32_t)v, hi = (uint32_t)(v >> 32);
    lo = lane_xor<32>(lane_xor<16>(dpp<0x140>(lo), lane), lane);        // row mirror (^15), ^16, ^32
    hi = lane_xor<32>(lane_xor<16>(dpp<0x140>(hi), lane), lane);
    return (u64)hi << 32 | lo;
}
// The 64 largest of a descending and an ascending list, descending: lane i
// keeps the larger of the two, which makes a bitonic sequence.
__device__ __forceinline__ u64 merge_lists(u64 down, u64 up, int lane) {
    return merge_steps<32>(down > up ? down : up, lane, true);
}

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

// How many keys of N descending lists of 64 in LDS are larger than v: a binary
// search in each, all at once, because every step waits for LDS.
template <int N> __device__ __forceinline__ int count_larger(const u64 *lists, u64 v) {
    int n[N], all = 0;
#pragma unroll
    for (int w = 0; w < N; ++w) n[w] = 0;
#pragma unroll
    for (int b = 32; b; b >>= 1)
#pragma unroll
        for (int w = 0; w < N; ++w) n[w] += lists[w * 64 + n[w] + b - 1] > v ? b : 0;
#pragma unroll
    for (int w = 0; w < N; ++w) all += n[w] + (lists[w * 64 + n[w]] > v);
    return all;
}

}  // namespace ar
