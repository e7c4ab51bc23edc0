// distill.hip -- distillation from a teacher's top logits over
// vocabulary-split rows: the loss and its gradient.
//
// One pass over the logits as in logprobs.hip.  Where the teacher leaves mass
// to the unlisted entries, the student's mass on them is summed directly:
// the sum of everything less the listed terms would lose it to cancellation
// wherever the student is sure of a listed token.  The list is worked out
// once per workgroup, an entry to a thread, and kept in LDS; each wave makes of
// the entries in a tile of its own one bit per logit in the lanes that hold
// them, and only vectors with a bit look at single logits.
#include "dispatch.hpp"
#include "vocab_device.hpp"
#include "vocab_launch.hpp"

namespace ar {

constexpr float kTailLeast = 0x1p-20f;             // a remaining mass below this is the values' rounding
constexpr int kPer = kTeacherMax / 64;             // entries per lane, where a wave holds them all

// A row's list in LDS.
struct ListScratch {
    alignas(16) int place[kTeacherMax];            // tile * kTileElems + element there; -1: padding, also to a
                                                   // multiple of 4 entries
    int s[kTeacherMax], e[kTeacherMax];            // rank and element there
    float v[kTeacherMax];                          // the teacher's value
    float z[kTeacherMax];                          // the student's logit, read before any gradient is stored
    int repeats;                                   // some id stands more than once
};
// Places by hash, to find out whether any repeats: slots for k entries, a power
// of two, four times as many (looks are then short) but no more than twice the
// longest list.  The launch asks for this LDS, because the longest list's
// would keep workgroups of one wave from filling a compute unit.
__host__ __device__ inline int slot_bits(int k) {
    static_assert(kTeacherMax == 256, "9 bits");
    const int bits = 32 - __builtin_clz(4 * k - 1);
    return bits < 6 ? 6 : bits > 9 ? 9 : bits;
}
__device__ __forceinline__ int *place_table() {
    extern __shared__ int table[];
    return table;
}

// The teacher's distribution (uniform over the workgroup): ln q = (v - m) * scale - ls.
struct Teacher {
    float m, scale, ls;
    float qt, total;                               // remaining mass, sum of everything
    bool live;                                     // has entries
};
__device__ __forceinline__ float ln_q(const Teacher &t, float v) { return (v - t.m) * t.scale - t.ls; }

// f(k) for this thread's entries.
template <typename F> __device__ __forceinline__ void each_entry(const DistillArgs &a, F f) {
    for (int k = threadIdx.x; k < a.k; k += blockDim.x) f(k);
}

// Fill the list (all threads; the row's logits may not be overwritten before
// the barrier in here has been passed).
template <int DT, bool TAIL, int NR>
__device__ __forceinline__ Teacher load_teacher(const VocabGeom<NR> &g, const DistillArgs &a, ListScratch &l,
                                                long long row, int lane) {
    const int vocab = g.col0[g.n];
    each_entry(a, [&](int k) {
        const int64_t id = a.ids[row * a.k + k];
        const float v = a.values[row * a.k + k];
        const bool in = id >= 0 && id < vocab;
        const Place p = place_of<DT>(g, row, in ? (int)id : 0);
        l.place[k] = in ? p.t * kTileElems<DT> + p.et : -1;
        l.s[k] = p.s;
        l.e[k] = p.e;
        l.v[k] = in ? v : kNegInf;
        l.z[k] = in ? load1<DT>(row_of<DT>(g, p.s, row), p.e) : kNegInf;
    });
    if (threadIdx.x < (unsigned)(-a.k & 3)) l.place[a.k + threadIdx.x] = -1;
    for (int i = threadIdx.x; i < 1 << slot_bits(a.k); i += blockDim.x) place_table()[i] = -1;
    if (threadIdx.x == 0) l.repeats = 0;
    __syncthreads();
    Teacher t;
    float sum = 0.0f, m = kNegInf;
    if constexpr (TAIL) {
        bool any = false;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (i * 64 >= a.k) break;
            const int k = i * 64 + lane;
            if (k < a.k) {
                any |= l.place[k] >= 0;
                sum += expf(l.v[k]);
            }
        }
        sum = wave_sum(sum, lane);
        t.live = __any(any);
        t.m = t.ls = 0.0f;
        t.scale = 1.0f;
        t.qt = 1.0f - sum;
        t.qt = t.qt < kTailLeast ? 0.0f : t.qt;
        t.total = sum + t.qt;
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (i * 64 >= a.k) break;
            const int k = i * 64 + lane;
            if (k < a.k) m = __builtin_fmaxf(m, l.v[k]);
        }
        m = wave_max(m, lane);
        t.live = m != kNegInf;
        t.m = t.live ? m : 0.0f;
        t.scale = g.inv_t;
        t.ls = 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (i * 64 >= a.k) break;
            const int k = i * 64 + lane;
            if (k < a.k) sum += expf(ln_q(t, l.v[k]));
        }
        sum = wave_sum(sum, lane);
        t.ls = t.live ? logf(sum) : 0.0f;
        t.qt = 0.0f;
        t.total = !t.live ? 0.0f : sum == sum ? 1.0f : sum;
    }
    return t;
}

// Sums of a row, each relative to its own reference logit: every entry's and
// the unlisted entries'.  The unlisted ones keep theirs, because they may lie
// any distance below the row's: one number for both would lose their count.
struct RowSums {
    float m, s;
    float tm, ts;
};
// Unlisted and listed sums (each with its own reference) put together.
__device__ __forceinline__ RowSums join_sums(Stats tail, Stats listed, float c) {
    const Stats rest = settled(tail, c);
    const float m = __builtin_fmaxf(tail.m, listed.m);
    shift_stats(tail, m, c);
    shift_stats(listed, m, c);
    const Stats all = settled(Stats{m, tail.s + listed.s, 0.0f}, c);
    return {all.m, all.s, rest.m, rest.s};
}

// Whether any id repeats, in l.repeats past the next barrier (all threads,
// after load_teacher): every entry looks for its place in the table, which
// takes a look or two; comparing each with the whole list is left to those
// rows where it says so.
__device__ __forceinline__ void note_repeats(const DistillArgs &a, ListScratch &l) {
    const int bits = slot_bits(a.k);
    each_entry(a, [&](int k) {
        const int place = l.place[k];
        if (place < 0) return;
        for (unsigned h = (unsigned)place * 2654435761u >> (32 - bits);; h = (h + 1) & ((1u << bits) - 1)) {
            const int there = atomicCAS(&place_table()[h], -1, place);
            if (there == place) l.repeats = 1;
            if (there == place || there == -1) return;         // there are free slots always
        }
    });
}
// f(i) for every entry i of the list that stands at `place`, in order.
template <typename F> __device__ __forceinline__ void each_at(const ListScratch &l, int n, int place, F f) {
    for (int i = 0; i < n; i += 4) {
        const int4 p = *(const int4 *)(l.place + i);
        if (p.x == place) f(i);
        if (p.y == place) f(i + 1);
        if (p.z == place) f(i + 2);
        if (p.w == place) f(i + 3);
    }
}
// ln q of entry k's id: a repeated one's entries are added up.
__device__ __forceinline__ float ln_q_of_id(const DistillArgs &a, const Teacher &t, const ListScratch &l, int k) {
    const int place = l.place[k];
    const float lq = ln_q(t, l.v[k]);
    if (!l.repeats || place < 0) return lq;
    float q = 0.0f;
    int same = 0;
    each_at(l, a.k, place, [&](int i) { q += expf(ln_q(t, l.v[i])), ++same; });
    return same > 1 ? logf(q) : lq;
}

// The row's loss, in all lanes of the wave.  An entry counts its own q times
// the logarithm of its id's.
template <bool TAIL, int NR>
__device__ __forceinline__ float row_loss(const VocabGeom<NR> &g, const DistillArgs &a, const Teacher &t,
                                          const ListScratch &l, const RowSums &r, int lane) {
    const Ref ref = make_ref(r.m, g.c);
    const bool empty = r.m == kNegInf && r.s == 0.0f;
    const float lse = logf(r.s);
    float sum = 0.0f;
    for (int k = lane; k < a.k; k += 64) {
        const float lq = ln_q_of_id(a, t, l, k), q = expf(ln_q(t, l.v[k]));
        const float lp = empty ? kNegInf : rel_ln(l.z[k], ref, g.inv_t) - lse;
        if (l.place[k] >= 0 && q != 0.0f) sum += q * (lq - lp);
    }
    sum = wave_sum(sum, lane);
    if constexpr (TAIL) {
        const float lt = empty ? kNegInf : rel_ln(r.tm, ref, g.inv_t) + (logf(r.ts) - lse);
        if (t.qt != 0.0f) sum += t.qt * (logf(t.qt) - lt);
    }
    return t.live ? sum : 0.0f;
}

__device__ __forceinline__ void write_row(const DistillArgs &a, long long row, const RowSums &r, float loss) {
    if (a.loss) a.loss[row] = loss;
    if (a.saved) {
        float *o = a.saved + row * 4;
        o[0] = r.m;
        o[1] = r.s;
        o[2] = r.tm;
        o[3] = r.ts;
    }
}

// Bit u*K + i of a lane: its logit i in vector u of tile `at` is listed.
// place: the wave's copy of the list's places, entry k in lane k % 64.
struct Places {
    int at[kPer];
};
__device__ __forceinline__ Places load_places(const ListScratch &l, int k, int lane) {
    Places p;
#pragma unroll
    for (int i = 0; i < kPer; ++i) p.at[i] = i * 64 + lane < k ? l.place[i * 64 + lane] : -1;
    return p;
}
template <int DT>
__device__ __forceinline__ uint32_t tile_bits(const Places &p, int k, int at, int lane) {
    constexpr int K = Lanes<DT>::value;
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (i * 64 >= k) break;
        const int lo = at * kTileElems<DT>;
        for (u64 in = __ballot((unsigned)(p.at[i] - lo) < (unsigned)kTileElems<DT>); in; in &= in - 1) {
            const int el = __builtin_amdgcn_readlane(p.at[i], __builtin_ctzll(in)) - lo;
            const uint32_t bit = 1u << (el / (64 * K) * K + el % K);
            bits |= lane == el / K % 64 ? bit : 0;
        }
    }
    return bits;
}
// The listed logits of vector u become -inf.
template <int DT>
__device__ __forceinline__ void drop_listed(u32x4 &v, uint32_t bits, int u, int e0, int held) {
    constexpr int K = Lanes<DT>::value;
    asm volatile("" : "+v"(bits));                             // nothing here is worked out for all vectors beforehand
    uint32_t m = bits >> u * K & ((1u << K) - 1);
    if (!__any(m)) return;
    m = e0 < held ? m >> (held - e0) : m << (e0 - held < K ? e0 - held : 0);       // at a rank's ends register 0 is not e0
#pragma unroll
    for (int i = 0; i < K; ++i) {
        if constexpr (DT == F32) {
            v[i] = m >> i & 1 ? neg_inf_bits<DT>() : v[i];
        } else {
            const uint32_t part = 0xffffu << (i & 1) * 16, ninf = neg_inf_bits<DT>() << (i & 1) * 16;
            v[i / 2] = m >> i & 1 ? (v[i / 2] & ~part) | ninf : v[i / 2];
        }
    }
}

// Gradient of a row, t relative to m (listed) or to the unlisted entries' m_t:
//   unlisted  2^t * cu,  listed  (Q 2^t / S - q_v) * g / T,
// with cu = (Q p_t - q_t) g / (T S_t), p_t = 2^((m_t - m) c) S_t / S (TAIL), or,
// both against the whole row, cu = Q g / (T S).  Referred to their own sum, the
// unlisted terms keep their precision however small their share is.  The
// first form is stored everywhere; then, past a barrier, the workgroup stores
// its listed columns once more, an entry to a thread.
struct RowGradient {
    Ref ref, all;                                  // of the unlisted terms, of the row's sum
    float gs, total, lse2, cu;
    bool zero;
};
template <int DT, bool TAIL, int NR>
__device__ __forceinline__ RowGradient row_gradient(const VocabGeom<NR> &g, const DistillArgs &a, const Teacher &t,
                                                    const RowSums &r, long long row) {
    RowGradient d;
    d.gs = (a.grad_loss ? a.grad_loss[row] : 1.0f) * g.inv_t;
    d.zero = !t.live || d.gs == 0.0f || (r.m == kNegInf && r.s == 0.0f);
    d.ref = d.all = make_ref(r.m, g.c);
    d.total = t.total;
    d.lse2 = __builtin_log2f(r.s);
    if constexpr (TAIL) {
        const float pt = exp2_fast(rel_log2(r.tm, d.all, g.c)) * (r.ts / r.s);
        d.ref = make_ref(r.tm, g.c);
        d.cu = r.ts == 0.0f ? 0.0f : (t.total * pt - t.qt) * d.gs / r.ts;          // no unlisted mass: nothing to scale
    } else {
        d.cu = t.total * d.gs / r.s;
    }
    d.cu *= exp2_fast(-term_shift<DT>(d.ref));
    return d;
}
template <int DT, int NR>
__device__ __forceinline__ void gradient_vec(const VocabGeom<NR> &g, const RowGradient &d, long long row,
                                             const TileWalk &w, int e0, int held, u32x4 raw) {
    Pack<DT> v = unpack<DT>(raw);
#pragma unroll
    for (int i = 0; i < Lanes<DT>::value; ++i) v.v[i] = term<DT>(v.v[i], d.ref, g).e * d.cu;
    store_vec<DT>(grad_row_of<DT>(g, w.s, row), v, w, e0, held);
}
// The listed columns among the workgroup's tiles; an id's entries all store
// the same.
template <int DT, int NR>
__device__ __forceinline__ void store_listed(const VocabGeom<NR> &g, const DistillArgs &a, const RowGradient &d,
                                             const Teacher &t, const ListScratch &l, long long row, int part) {
    __syncthreads();
    each_entry(a, [&](int k) {
        const int place = l.place[k], waves = blockDim.x >> 6;
        if (place < 0 || place / kTileElems<DT> / waves % g.parts != part) return;
        const float q = expf(ln_q_of_id(a, t, l, k));
        const float p = d.total * exp2_fast(rel_log2(l.z[k], d.all, g.c) - d.lse2);
        store1<DT>(grad_row_of<DT>(g, l.s[k], row), l.e[k], round_to<DT>((p - q) * d.gs));
    });
}
template <int DT, int NR>
__device__ __forceinline__ void gradient_tiles(const VocabGeom<NR> &g, const DistillArgs &a, const RowGradient &d,
                                               const Teacher &t, const ListScratch &l, long long row, int part,
                                               int first, int step, int lane) {
    if (d.zero) {
        zero_tiles<DT>(g, row, first, step, lane);
        return;
    }
    VectorStream<DT, true, NR> stream;
    stream.start(g, row, first, lane);
    stream.run(g, row, step, lane, [&](const TileWalk &w, int, int e0, int held, u32x4 raw) {
        gradient_vec<DT>(g, d, row, w, e0, held, raw);
    });
    store_listed<DT>(g, a, d, t, l, row, part);
}

// Sums over this thread's listed logits in the workgroup's part of the row, each id once.
template <int DT, int NR>
__device__ __forceinline__ Stats listed_sums(const VocabGeom<NR> &g, const DistillArgs &a, const ListScratch &l, int part) {
    Stats li{kNegInf, 0.0f, 0.0f};
    each_entry(a, [&](int k) {
        const int place = l.place[k], waves = blockDim.x >> 6;
        if (place < 0 || place / kTileElems<DT> / waves % g.parts != part) return;
        bool first = true;
        if (l.repeats) each_at(l, k, place, [&](int i) { first &= i >= k; });
        if (!first) return;
        const float z = l.z[k];
        if (z > li.m) shift_stats(li, z, g.c);
        li.s += exp2_fast(rel(z, make_ref(li.m, g.c)));
    });
    return li;
}
// Both sums over the workgroup.
struct SumScratch {
    Stats tail[kHeldWaves], listed[kHeldWaves];
};
template <bool TAIL>
__device__ __forceinline__ void block_sums(Stats &st, Stats &li, SumScratch &lds, int waves, int wave, int lane, float c) {
    wave_stats<false>(st, lane, c);
    if constexpr (TAIL) wave_stats<false>(li, lane, c);
    if (waves == 1) return;
    if (lane == 0) {
        lds.tail[wave] = st;
        if constexpr (TAIL) lds.listed[wave] = li;
    }
    __syncthreads();
    const Stats none{kNegInf, 0.0f, 0.0f};
    st = lane < waves ? lds.tail[lane] : none;
    wave_stats<false>(st, lane, c);
    if constexpr (TAIL) {
        li = lane < waves ? lds.listed[lane] : none;
        wave_stats<false>(li, lane, c);
    }
}

// Sums of a row (or of one part of it), the loss where the row is whole, and
// with BOTH its gradient by the same workgroup.  AGAIN: the logits will be
// read again soon and are left in the caches.
// Bound by HBM where rows are many: with BOTH 8192 x 131072 bf16, 64 entries
// and a tail 909 us, 7.0 TB/s for two reads and one write.  With fewer it goes
// by rounds: scalar registers allow seven waves to a SIMD, three workgroups to
// a compute unit, 768 rows at once.  With 100 entries 768 x 50021 bf16 take 34
// us, 780 rows 41 (the bytes 11): list, stream and joining once more.
template <int DT, int NR, bool TAIL, bool BOTH, bool AGAIN>
__global__ __launch_bounds__(64 * kVocabWaves) void distill_kernel(const VocabGeom<NR> g, const DistillArgs a) {
    __shared__ SumScratch lds;
    __shared__ ListScratch list;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int waves = blockDim.x >> 6, step = waves * g.parts;
    const int local = blockIdx.x / g.parts, part = blockIdx.x - local * g.parts;
    const long long row = g.row0 + local;
    const int first = part * waves + wave;
    VectorStream<DT, !AGAIN, NR> stream;
    stream.start(g, row, first, lane);
    const Teacher t = load_teacher<DT, TAIL>(g, a, list, row, lane);
    Running run;
    Stats li{kNegInf, 0.0f, 0.0f};
    if (t.live) {                                              // a row without a teacher is not read further
        note_repeats(a, list);
        Places places;
        if constexpr (TAIL) {
            __syncthreads();
            places = load_places(list, a.k, lane);
            li = listed_sums<DT>(g, a, list, part);
        }
        uint32_t bits = 0;
        stream.run(g, row, step, lane, [&](const TileWalk &w, int u, int e0, int held, u32x4 raw) {
            if (!w.template full<DT>()) mask_vec<DT>(raw, e0, held, w.w);
            if constexpr (TAIL) {
                if (u == 0) bits = tile_bits<DT>(places, a.k, w.at, lane);
                drop_listed<DT>(raw, bits, u, e0, held);
            }
            if (u == 0) end_tile(run);
            add_vec<DT, false>(run, unpack<DT>(raw), g);
        });
    }
    Stats st = total(run);
    block_sums<TAIL>(st, li, lds, waves, wave, lane, g.c);
    if (g.parts > 1) {
        // a sum's sign, which it does not need, says whether the list repeats an id
        if (threadIdx.x == 0)
            a.part[row * g.parts + part] =
                make_float4(st.m, __builtin_copysignf(st.s, t.live && list.repeats ? -1.0f : 1.0f), li.m, li.s);
        return;
    }
    const RowSums r = join_sums(st, li, g.c);
    if (wave == 0) {
        const float loss = row_loss<TAIL>(g, a, t, list, r, lane);
        if (lane == 0) write_row(a, row, r, loss);
    }
    if constexpr (BOTH)
        gradient_tiles<DT>(g, a, row_gradient<DT, TAIL>(g, a, t, r, row), t, list, row, part, first, step, lane);
}

// Loss and gradient of a row held in the workgroup's registers: 8192 x 32768
// bf16, 64 entries and a tail 229 us (read twice: 257).
template <int DT, int NR, bool TAIL, int T>
__global__ __launch_bounds__(64 * kHeldWaves) void distill_held_kernel(const VocabGeom<NR> g, const DistillArgs a) {
    __shared__ SumScratch lds;
    __shared__ ListScratch list;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int waves = blockDim.x >> 6;
    const long long row = g.row0 + blockIdx.x;
    HeldTiles<DT, NR, T> tiles;
    tiles.start(g, row, wave, waves, lane);
    const Teacher t = load_teacher<DT, TAIL>(g, a, list, row, lane);
    Stats st{kNegInf, 0.0f, 0.0f}, li = st;
    if (t.live) {
        note_repeats(a, list);
        uint32_t bits[T];
        if constexpr (TAIL) {
            __syncthreads();
            li = listed_sums<DT>(g, a, list, 0);
            const Places places = load_places(list, a.k, lane);
#pragma unroll
            for (int k = 0; k < T; ++k) bits[k] = tile_bits<DT>(places, a.k, wave + k * waves, lane);
        }
        st = held_sums<DT, false>(g, tiles, lane, [&](int k, int u, int e0, int held, u32x4 &raw) {
            if constexpr (TAIL) drop_listed<DT>(raw, bits[k], u, e0, held);
        });
    }
    block_sums<TAIL>(st, li, lds, waves, wave, lane, g.c);
    const RowSums r = join_sums(st, li, g.c);
    if (wave == 0) {
        const float loss = row_loss<TAIL>(g, a, t, list, r, lane);
        if (lane == 0) write_row(a, row, r, loss);
    }
    const RowGradient d = row_gradient<DT, TAIL>(g, a, t, r, row);
    if (d.zero) {
        zero_tiles<DT>(g, row, wave, waves, lane);
        return;
    }
    tiles.each(lane, [&](const TileWalk &w, int, int, int e0, int held, u32x4 raw) {
        gradient_vec<DT>(g, d, row, w, e0, held, raw);
    });
    store_listed<DT>(g, a, d, t, list, row, 0);
}

// A row's loss from its parts: one wave, one lane per part.
template <int DT, int NR, bool TAIL>
__global__ __launch_bounds__(64) void distill_join_kernel(const VocabGeom<NR> g, const DistillArgs a) {
    __shared__ ListScratch list;
    const int lane = threadIdx.x;
    const long long row = g.row0 + blockIdx.x;
    const Teacher t = load_teacher<DT, TAIL>(g, a, list, row, lane);
    Stats st{kNegInf, 0.0f, 0.0f}, li{kNegInf, 0.0f, 0.0f};
    if (lane < g.parts) {
        const float4 p = a.part[row * g.parts + lane];
        st.m = p.x, st.s = __builtin_fabsf(p.y), li.m = p.z, li.s = p.w;
        if (lane == 0) list.repeats = f32_bits(p.y) >> 31;
    }
    wave_stats<false>(st, lane, g.c);
    wave_stats<false>(li, lane, g.c);
    const RowSums r = join_sums(st, li, g.c);
    __syncthreads();
    const float loss = row_loss<TAIL>(g, a, t, list, r, lane);
    if (lane == 0) write_row(a, row, r, loss);
}

template <int DT, int NR, bool TAIL>
__global__ __launch_bounds__(64 * kVocabWaves) void distill_backward_kernel(const VocabGeom<NR> g, const DistillArgs a) {
    __shared__ ListScratch list;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int waves = blockDim.x >> 6, step = waves * g.parts;
    const int local = blockIdx.x / g.parts, part = blockIdx.x - local * g.parts;
    const long long row = g.row0 + local;
    const Teacher t = load_teacher<DT, TAIL>(g, a, list, row, lane);
    note_repeats(a, list);
    const float *o = a.saved + row * 4;
    const RowGradient d = row_gradient<DT, TAIL>(g, a, t, RowSums{o[0], o[1], o[2], o[3]}, row);
    gradient_tiles<DT>(g, a, d, t, list, row, part, part * waves + wave, step, lane);
}

template <int DT, int NR, bool TAIL>
hipError_t run_distill(const VocabCall &c, const DistillArgs &a, VocabStage stage, hipStream_t s) {
    const size_t lds = sizeof(int) << slot_bits(a.k);
    switch (stage) {
    case kForward:
        if (c.again) return launch_rows<NR>(c, a, distill_kernel<DT, NR, TAIL, false, true>, c.parts, c.waves, s, lds);
        return launch_rows<NR>(c, a, distill_kernel<DT, NR, TAIL, false, false>, c.parts, c.waves, s, lds);
    case kBoth:
        if (c.held == 1) return launch_rows<NR>(c, a, distill_held_kernel<DT, NR, TAIL, 1>, 1, c.waves, s, lds);
        if (c.held == 2) return launch_rows<NR>(c, a, distill_held_kernel<DT, NR, TAIL, 2>, 1, c.waves, s, lds);
        if constexpr (!TAIL || DT == BF16)                     // the others are never chosen (vocab_api.cpp)
            if (c.held) return launch_rows<NR>(c, a, distill_held_kernel<DT, NR, TAIL, kHeldTiles>, 1, c.waves, s, lds);
        return launch_rows<NR>(c, a, distill_kernel<DT, NR, TAIL, true, true>, 1, c.waves, s, lds);
    case kBackward: return launch_rows<NR>(c, a, distill_backward_kernel<DT, NR, TAIL>, c.parts, c.waves, s, lds);
    default: return launch_rows<NR>(c, a, distill_join_kernel<DT, NR, TAIL>, 1, 1, s, lds);
    }
}

hipError_t launch_distill(const VocabCall &c, const DistillArgs &a, bool tail, VocabStage stage, hipStream_t s) {
    return dispatch_vocab(c, [&](auto dt, auto nr) {
        return tail ? run_distill<dt.value, nr.value, true>(c, a, stage, s)
                    : run_distill<dt.value, nr.value, false>(c, a, stage, s);
    });
}

}  // namespace ar
