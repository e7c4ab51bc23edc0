// distill.hip -- distillation from a teacher's top logits over
// vocabulary-split rows: the loss and its gradient.
//
// One pass over the logits as in logprobs.hip.  Where the teacher leaves mass
// to the unlisted entries, the student's mass on them is summed directly:
// the sum of everything less the listed terms would lose it to cancellation
// wherever the student is sure of a listed token.  Every wave holds the whole
// list, one entry to a lane (four past 64 entries), with the place of each in
// the row's tiles, and makes of those in a tile of its own one bit per logit
// in the lanes that hold them; only vectors with a bit look at single logits.
#include "dispatch.hpp"
#include "vocab_device.hpp"
#include "vocab_launch.hpp"

namespace ar {

constexpr float kTailLeast = 0x1p-20f;             // a remaining mass below this is the values' rounding

// The teacher's distribution of a row, entry k of it in lane k % 64.
template <int PER> struct Teacher {
    int id[PER];                                   // -1: padding
    float q[PER], lq[PER];                         // probability and its logarithm
    float qt, total;                               // remaining mass, sum of everything
    bool live;                                     // has entries
};
template <bool TAIL, int PER>
__device__ __forceinline__ Teacher<PER> load_teacher(const DistillArgs &a, long long row, int vocab, float inv_t, int lane) {
    Teacher<PER> t;
    float m = kNegInf;
    bool any = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int k = i * 64 + lane;
        t.id[i] = -1;
        t.lq[i] = kNegInf;
        if (k < a.k) {
            const int64_t id = a.ids[row * a.k + k];
            if (id >= 0 && id < vocab) {
                t.id[i] = (int)id;
                t.lq[i] = a.values[row * a.k + k];
                any = true;
            }
        }
        m = __builtin_fmaxf(m, t.lq[i]);
    }
    float sum = 0.0f;
    if constexpr (TAIL) {
        t.live = __any(any);
#pragma unroll
        for (int i = 0; i < PER; ++i) sum += t.q[i] = expf(t.lq[i]);
        sum = wave_sum(sum, lane);
        t.qt = 1.0f - sum;
        t.qt = t.qt < kTailLeast ? 0.0f : t.qt;
        t.total = sum + t.qt;
    } else {
        m = wave_max(m, lane);
        t.live = m != kNegInf;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            t.lq[i] = t.live ? (t.lq[i] - m) * inv_t : kNegInf;
            sum += expf(t.lq[i]);
        }
        sum = wave_sum(sum, lane);
        const float ls = logf(sum);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            t.lq[i] = t.live ? t.lq[i] - ls : kNegInf;
            t.q[i] = expf(t.lq[i]);
        }
        t.qt = 0.0f;
        t.total = t.live ? 1.0f : 0.0f;
        if (sum != sum) t.total = sum;
    }
    return t;
}

// Sums of a row: every entry's, and the unlisted entries' as a logarithm.
struct RowSums {
    float m, s;                                    // reference, sum of 2^t
    float tail2;                                   // log2 of the unlisted part of the sum
};
// Unlisted and listed sums (each with its own reference) put together.
__device__ __forceinline__ RowSums join_sums(Stats tail, Stats listed, float c) {
    const float m = __builtin_fmaxf(tail.m, listed.m);
    const Ref to = make_ref(m, c);
    RowSums r;
    r.m = m;
    r.tail2 = ref_shift(make_ref(tail.m, c), to, c) + __builtin_log2f(tail.s);
    shift_stats(tail, m, c);
    shift_stats(listed, m, c);
    r.s = tail.s + listed.s;
    return r;
}

// The row's loss, in all lanes of the wave.
template <bool TAIL, int NR, int PER>
__device__ __forceinline__ float row_loss(const VocabGeom<NR> &g, const Teacher<PER> &t, const float *z,
                                          const RowSums &r, int lane) {
    const Ref ref = make_ref(r.m, g.c);
    const bool empty = r.m == kNegInf && r.s == 0.0f;
    const float lse = logf(r.s);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const float lp = empty ? kNegInf : rel_ln(z[i], ref, g.inv_t) - lse;
        if (t.id[i] >= 0 && t.q[i] != 0.0f) sum += t.q[i] * (t.lq[i] - lp);
    }
    sum = wave_sum(sum, lane);
    if constexpr (TAIL) {
        if (t.qt != 0.0f) sum += t.qt * (logf(t.qt) - (empty ? kNegInf : kLn2 * r.tail2 - lse));
    }
    return t.live ? sum : 0.0f;
}

template <int NR>
__device__ __forceinline__ void write_row(const DistillArgs &a, long long row, const RowSums &r, float loss) {
    if (a.loss) a.loss[row] = loss;
    if (a.saved) {
        float *o = a.saved + row * 4;
        o[0] = r.m;
        o[1] = r.s;
        o[2] = r.tail2;
        o[3] = 0.0f;
    }
}

// The entries in the row: where they stand, and the student's logits there
// (read before any gradient is stored, which may take the logits' place).
template <int PER> struct Entries {
    int place[PER];                                // tile * kTileElems + element (-1: padding)
    int s[PER], e[PER];                            // rank and element there
    float z[PER];
};
template <int DT, int NR, int PER>
__device__ __forceinline__ Entries<PER> place_entries(const VocabGeom<NR> &g, const Teacher<PER> &t, long long row) {
    Entries<PER> e;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        e.place[i] = -1;
        e.s[i] = e.e[i] = 0;
        e.z[i] = kNegInf;
        if (t.id[i] >= 0) {
            const Place p = place_of<DT>(g, row, t.id[i]);
            e.place[i] = p.t * kTileElems<DT> + p.et;
            e.s[i] = p.s;
            e.e[i] = p.e;
            e.z[i] = load1<DT>(row_of<DT>(g, p.s, row), p.e);
        }
    }
    return e;
}
// Whether an entry stands in this wave's tiles.
template <int DT> __device__ __forceinline__ bool owned(int place, int first, int step) {
    return place >= 0 && (unsigned)place / kTileElems<DT> % (unsigned)step == (unsigned)first;
}

// What this wave does for the entries in its tiles: the probability on each
// one's id (its own, and those of other entries of the same id, if there are
// any), and whether it is the id's first.
template <int PER> struct Own {
    float q[PER];
    bool mine[PER], lead[PER];
};
template <int DT, int PER>
__device__ __forceinline__ Own<PER> own_entries(const Entries<PER> &e, const Teacher<PER> &t, int first, int step,
                                                int lane) {
    Own<PER> o;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        o.q[i] = t.q[i];
        o.mine[i] = o.lead[i] = owned<DT>(e.place[i], first, step);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        for (u64 in = __ballot(o.mine[i]); in; in &= in - 1) {
            const int b = __builtin_ctzll(in), place = __builtin_amdgcn_readlane(e.place[i], b);
            int entries = 0;
#pragma unroll
            for (int k = 0; k < PER; ++k) entries += __builtin_popcountll(__ballot(e.place[k] == place));
            if (entries == 1) continue;
            float sum = 0.0f;
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                for (u64 same = __ballot(e.place[k] == place); same; same &= same - 1)
                    sum += bits_f32((uint32_t)__builtin_amdgcn_readlane((int)f32_bits(t.q[k]), __builtin_ctzll(same)));
            }
            const bool again = __builtin_amdgcn_readlane((int)o.lead[i], b) == 0;
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                if (e.place[k] != place) continue;
                o.q[k] = sum;
                if (!again) o.lead[k] = k == i && lane == b;
            }
        }
    }
    return o;
}

// Bit u*K + i of a lane: its logit i in vector u of tile `at` is listed.
template <int DT, int PER>
__device__ __forceinline__ uint32_t tile_bits(const Entries<PER> &e, int at, int lane) {
    constexpr int K = Lanes<DT>::value;
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        for (u64 in = __ballot(e.place[i] >= 0 && e.place[i] / kTileElems<DT> == at); in; in &= in - 1) {
            const int el = __builtin_amdgcn_readlane(e.place[i], __builtin_ctzll(in)) % kTileElems<DT>;
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

// Gradient of a row:
//   unlisted  2^(t - r2) * cu,  listed  (Q 2^(t - lse2) - q_v) * g / T,
// where r2 is the log2 of the unlisted sum and cu = (Q tail / S - q_t) g / T
// (TAIL), or of the whole sum and cu = Q g / T.  Referred to their own sum,
// the unlisted terms keep their precision however small their share is.  The
// first form is stored everywhere; then the wave stores its listed columns
// once more, an entry to a lane.
struct RowGradient {
    Ref ref;
    float gs, total, lse2, r2, cu;
    bool zero;
};
template <bool TAIL, int NR, int PER>
__device__ __forceinline__ RowGradient row_gradient(const VocabGeom<NR> &g, const DistillArgs &a,
                                                    const Teacher<PER> &t, const RowSums &r, long long row) {
    RowGradient d;
    d.gs = (a.grad_loss ? a.grad_loss[row] : 1.0f) * g.inv_t;
    d.zero = !t.live || d.gs == 0.0f || (r.m == kNegInf && r.s == 0.0f);
    d.ref = make_ref(r.m, g.c);
    d.total = t.total;
    d.lse2 = __builtin_log2f(r.s);
    d.r2 = d.lse2;
    d.cu = t.total * d.gs;
    if constexpr (TAIL) {
        const bool none = r.tail2 == kNegInf;                  // no unlisted mass: nothing to scale
        d.r2 = none ? 0.0f : r.tail2;
        d.cu = none ? 0.0f : (t.total * exp2_fast(r.tail2 - d.lse2) - t.qt) * d.gs;
    }
    return d;
}
template <int DT, int NR>
__device__ __forceinline__ void gradient_vec(const VocabGeom<NR> &g, const RowGradient &d, long long row,
                                             const TileWalk &w, int e0, int held, u32x4 raw) {
    Pack<DT> v = unpack<DT>(raw);
#pragma unroll
    for (int i = 0; i < Lanes<DT>::value; ++i) v.v[i] = exp2_fast(rel(v.v[i], d.ref) - d.r2) * d.cu;
    store_vec<DT>(grad_row_of<DT>(g, w.s, row), v, w, e0, held);
}
template <int DT, int NR, int PER>
__device__ __forceinline__ void store_listed(const VocabGeom<NR> &g, const RowGradient &d, const Entries<PER> &e,
                                             const Own<PER> &o, long long row) {
    // after the vectors' stores, which other lanes of this wave have issued
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (o.mine[i]) {
            const float p = d.total * exp2_fast(rel(e.z[i], d.ref) - d.lse2);
            store1<DT>(grad_row_of<DT>(g, e.s[i], row), e.e[i], round_to<DT>((p - o.q[i]) * d.gs));
        }
    }
}
template <int DT, int NR, int PER>
__device__ __forceinline__ void gradient_tiles(const VocabGeom<NR> &g, const RowGradient &d, const Entries<PER> &e,
                                               const Own<PER> &o, long long row, int first, int step, int lane) {
    if (d.zero) {
        zero_tiles<DT>(g, row, first, step, lane);
        return;
    }
    VectorStream<DT, true, NR> stream;
    stream.start(g, row, first, lane);
    stream.run(g, row, step, lane, [&](const TileWalk &w, int, int e0, int held, u32x4 raw) {
        gradient_vec<DT>(g, d, row, w, e0, held, raw);
    });
    store_listed<DT>(g, d, e, o, row);
}

// Sums over this wave's listed logits, each id once.
template <int PER> __device__ __forceinline__ Stats listed_sums(const Entries<PER> &e, const Own<PER> &o, float c) {
    Stats li{kNegInf, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < PER; ++i) li.m = __builtin_fmaxf(li.m, o.lead[i] ? e.z[i] : kNegInf);
    const Ref ref = make_ref(li.m, c);
#pragma unroll
    for (int i = 0; i < PER; ++i) li.s += o.lead[i] ? exp2_fast(rel(e.z[i], ref)) : 0.0f;
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
// with BOTH its gradient by the same workgroup.
template <int DT, int NR, bool TAIL, bool BOTH, int PER>
__global__ __launch_bounds__(64 * kVocabWaves) void distill_kernel(const VocabGeom<NR> g, const DistillArgs a) {
    __shared__ SumScratch lds;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int waves = blockDim.x >> 6, step = waves * g.parts;
    const int local = blockIdx.x / g.parts, part = blockIdx.x - local * g.parts;
    const long long row = g.row0 + local;
    const int first = part * waves + wave;
    VectorStream<DT, !BOTH, NR> stream;
    stream.start(g, row, first, lane);
    const Teacher<PER> t = load_teacher<TAIL, PER>(a, row, g.col0[g.n], g.inv_t, lane);
    const Entries<PER> e = place_entries<DT>(g, t, row);
    Running run;
    if (t.live) {                                              // a row without a teacher is not read further
        uint32_t bits = 0;
        stream.run(g, row, step, lane, [&](const TileWalk &w, int u, int e0, int held, u32x4 raw) {
            if (!w.template full<DT>()) mask_vec<DT>(raw, e0, held, w.w);
            if constexpr (TAIL) {
                if (u == 0) bits = tile_bits<DT>(e, w.at, lane);
                drop_listed<DT>(raw, bits, u, e0, held);
            }
            add_vec<DT, false>(run, unpack<DT>(raw), g.c);
        });
    }
    Own<PER> o;
    if constexpr (TAIL || BOTH) o = own_entries<DT>(e, t, first, step, lane);
    Stats st = run.st, li{kNegInf, 0.0f, 0.0f};
    if constexpr (TAIL) li = listed_sums(e, o, g.c);
    block_sums<TAIL>(st, li, lds, waves, wave, lane, g.c);
    if (g.parts > 1) {
        if (threadIdx.x == 0) a.part[row * g.parts + part] = make_float4(st.m, st.s, li.m, li.s);
        return;
    }
    const RowSums r = join_sums(st, li, g.c);
    if (wave == 0) {
        const float loss = row_loss<TAIL>(g, t, e.z, r, lane);
        if (lane == 0) write_row<NR>(a, row, r, loss);
    }
    if constexpr (BOTH) gradient_tiles<DT>(g, row_gradient<TAIL>(g, a, t, r, row), e, o, row, first, step, lane);
}

// Loss and gradient of a row held in the workgroup's registers.
template <int DT, int NR, bool TAIL, int PER, int T>
__global__ __launch_bounds__(64 * kHeldWaves) void distill_held_kernel(const VocabGeom<NR> g, const DistillArgs a) {
    __shared__ SumScratch lds;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int waves = blockDim.x >> 6;
    const long long row = g.row0 + blockIdx.x;
    HeldTiles<DT, NR, T> tiles;
    tiles.start(g, row, wave, waves, lane);
    const Teacher<PER> t = load_teacher<TAIL, PER>(a, row, g.col0[g.n], g.inv_t, lane);
    const Entries<PER> e = place_entries<DT>(g, t, row);
    const Own<PER> o = own_entries<DT>(e, t, wave, waves, lane);
    Stats st{kNegInf, 0.0f, 0.0f}, li = st;
    if (t.live) {
        uint32_t bits[T];
#pragma unroll
        for (int k = 0; k < T; ++k) bits[k] = TAIL ? tile_bits<DT>(e, wave + k * waves, lane) : 0;
        st = held_sums<DT, false>(g, tiles, lane, [&](int k, int u, int e0, int held, u32x4 &raw) {
            if constexpr (TAIL) drop_listed<DT>(raw, bits[k], u, e0, held);
        });
    }
    if constexpr (TAIL) li = listed_sums(e, o, g.c);
    block_sums<TAIL>(st, li, lds, waves, wave, lane, g.c);
    const RowSums r = join_sums(st, li, g.c);
    if (wave == 0) {
        const float loss = row_loss<TAIL>(g, t, e.z, r, lane);
        if (lane == 0) write_row<NR>(a, row, r, loss);
    }
    const RowGradient d = row_gradient<TAIL>(g, a, t, r, row);
    if (d.zero) {
        zero_tiles<DT>(g, row, wave, waves, lane);
        return;
    }
    tiles.each(lane, [&](const TileWalk &w, int, int, int e0, int held, u32x4 raw) {
        gradient_vec<DT>(g, d, row, w, e0, held, raw);
    });
    store_listed<DT>(g, d, e, o, row);
}

// A row's loss from its parts: one wave, one lane per part.
template <int DT, int NR, bool TAIL, int PER>
__global__ __launch_bounds__(64) void distill_join_kernel(const VocabGeom<NR> g, const DistillArgs a) {
    const int lane = threadIdx.x;
    const long long row = g.row0 + blockIdx.x;
    const Teacher<PER> t = load_teacher<TAIL, PER>(a, row, g.col0[g.n], g.inv_t, lane);
    const Entries<PER> e = place_entries<DT>(g, t, row);
    Stats st{kNegInf, 0.0f, 0.0f}, li{kNegInf, 0.0f, 0.0f};
    if (lane < g.parts) {
        const float4 p = a.part[row * g.parts + lane];
        st.m = p.x, st.s = p.y, li.m = p.z, li.s = p.w;
    }
    wave_stats<false>(st, lane, g.c);
    wave_stats<false>(li, lane, g.c);
    const RowSums r = join_sums(st, li, g.c);
    const float loss = row_loss<TAIL>(g, t, e.z, r, lane);
    if (lane == 0) write_row<NR>(a, row, r, loss);
}

template <int DT, int NR, bool TAIL, int PER>
__global__ __launch_bounds__(64 * kVocabWaves) void distill_backward_kernel(const VocabGeom<NR> g, const DistillArgs a) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int waves = blockDim.x >> 6, step = waves * g.parts;
    const int local = blockIdx.x / g.parts, part = blockIdx.x - local * g.parts;
    const long long row = g.row0 + local;
    const int first = part * waves + wave;
    const Teacher<PER> t = load_teacher<TAIL, PER>(a, row, g.col0[g.n], g.inv_t, lane);
    const Entries<PER> e = place_entries<DT>(g, t, row);
    const float *o = a.saved + row * 4;
    const RowGradient d = row_gradient<TAIL>(g, a, t, RowSums{o[0], o[1], o[2]}, row);
    gradient_tiles<DT>(g, d, e, own_entries<DT>(e, t, first, step, lane), row, first, step, lane);
}

template <int DT, int NR, bool TAIL, int PER>
hipError_t run_distill(const VocabCall &c, const DistillArgs &a, VocabStage stage, hipStream_t s) {
    switch (stage) {
    case kForward: return launch_rows<NR>(c, a, distill_kernel<DT, NR, TAIL, false, PER>, c.parts, c.waves, s);
    case kBoth:
        if constexpr (PER == 1) {
            if (c.held == 1) return launch_rows<NR>(c, a, distill_held_kernel<DT, NR, TAIL, 1, 1>, 1, c.waves, s);
            if (c.held) return launch_rows<NR>(c, a, distill_held_kernel<DT, NR, TAIL, 1, kHeldTiles>, 1, c.waves, s);
        }
        return launch_rows<NR>(c, a, distill_kernel<DT, NR, TAIL, true, PER>, 1, c.waves, s);
    case kBackward: return launch_rows<NR>(c, a, distill_backward_kernel<DT, NR, TAIL, PER>, c.parts, c.waves, s);
    default: return launch_rows<NR>(c, a, distill_join_kernel<DT, NR, TAIL, PER>, 1, 1, s);
    }
}

hipError_t launch_distill(const VocabCall &c, const DistillArgs &a, bool tail, VocabStage stage, hipStream_t s) {
    return dispatch_vocab(c, [&](auto dt, auto nr) {
        constexpr int DT = dt.value, NR = nr.value;
        if (a.k <= 64) return tail ? run_distill<DT, NR, true, 1>(c, a, stage, s) : run_distill<DT, NR, false, 1>(c, a, stage, s);
        return tail ? run_distill<DT, NR, true, kTeacherMax / 64>(c, a, stage, s)
                    : run_distill<DT, NR, false, kTeacherMax / 64>(c, a, stage, s);
    });
}

}  // namespace ar
