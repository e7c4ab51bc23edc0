// distill.hip -- distillation from a teacher's top logits over
// vocabulary-split rows: the loss and its gradient.
//
// One pass over the logits as in logprobs.hip.  Where the teacher leaves mass
// to the unlisted entries, the student's mass on them is summed directly:
// the sum of everything less the listed terms would lose it to cancellation
// wherever the student is sure of a listed token.  Every wave holds the whole
// list, one entry to a lane (four past 64 entries), with the place of each in
// the row's tiles; a vector that holds some is found by one ballot, and each
// is taken out of it (set to -inf) before it is added or its gradient formed.
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

// The listed logits, entry k in lane k % 64.
template <int DT, int NR, int PER>
__device__ __forceinline__ void listed_logits(const VocabGeom<NR> &g, const Teacher<PER> &t, long long row, float *z) {
#pragma unroll
    for (int i = 0; i < PER; ++i) z[i] = t.id[i] >= 0 ? logit_at<DT>(g, row, t.id[i]) : kNegInf;
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

// Where the entries stand: tile * kTileElems + element (-1: padding).
template <int PER> struct Entries {
    int place[PER];
    float z[PER];                                  // the logit, once taken out of its vector
};
template <int DT, int NR, int PER>
__device__ __forceinline__ Entries<PER> place_entries(const VocabGeom<NR> &g, const Teacher<PER> &t) {
    Entries<PER> e;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const Place p = t.id[i] >= 0 ? place_of<DT>(g, t.id[i]) : Place{0, 0};
        e.place[i] = t.id[i] >= 0 ? p.t * kTileElems<DT> + p.e : -1;
        e.z[i] = kNegInf;
    }
    return e;
}

// f(i, lane of the entry, lane of the vector, register element) for every
// entry in vector u of tile `at`; all but the wave's own lane are uniform.
template <int DT, bool TINY, int PER, typename F>
__device__ __forceinline__ void each_listed(const Entries<PER> &e, const TileWalk &t, int u, F f) {
    constexpr int K = Lanes<DT>::value;
    const int lo = t.at * kTileElems<DT> + u * 64 * K;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        u64 in = __ballot((unsigned)(e.place[i] - lo) < 64u * K);
        while (in) {
            const int b = __builtin_ctzll(in);
            in &= in - 1;
            const int d = __builtin_amdgcn_readlane(e.place[i], b) - lo, owner = d / K;
            const int e0 = elem0<DT>(t.j, u, owner);
            f(i, b, owner, d % K + e0 - held0<DT, TINY>(e0, t.w));
        }
    }
}
// Take the listed logits out of vector u: -inf in the vector, the value in the
// entry's lane.  An id's second entry finds -inf, so it counts its share of
// the student's mass as nothing and only its own probability.
template <int DT, bool TINY, int PER>
__device__ __forceinline__ void take_listed(Entries<PER> &e, u32x4 &v, const TileWalk &t, int u, int lane) {
    each_listed<DT, TINY>(e, t, u, [&](int i, int entry, int owner, int r) {
        const int word = DT == F32 ? r : r / 2, sh = DT == F32 ? 0 : (r & 1) * 16;
        uint32_t x = v[0];
#pragma unroll
        for (int k = 1; k < 4; ++k) x = word == k ? v[k] : x;
        x = (uint32_t)__builtin_amdgcn_readlane((int)x, owner);
        const uint32_t part = DT == F32 ? 0xffffffffu : 0xffffu << sh;
        const uint32_t gone = (x & ~part) | neg_inf_bits<DT>() << sh;
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = word == k && lane == owner ? gone : v[k];
        const Pack<DT> z = unpack<DT>(u32x4{(x & part) >> sh, 0, 0, 0});
        e.z[i] = lane == entry ? z.v[0] : e.z[i];
    });
}

// Whether an entry stands in this wave's tiles (`step` is a power of two).
template <int DT> __device__ __forceinline__ bool owned(int place, int first, int step) {
    return place >= 0 && (place / kTileElems<DT> & (step - 1)) == first;
}
// The probability on each owned entry's id: its own, and those of other
// entries of the same id, if there are any.
template <int DT, int PER>
__device__ __forceinline__ void merge_repeats(const Entries<PER> &e, const Teacher<PER> &t, int first, int step, float *q) {
#pragma unroll
    for (int i = 0; i < PER; ++i) q[i] = t.q[i];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        u64 in = __ballot(owned<DT>(e.place[i], first, step));
        while (in) {
            const int place = __builtin_amdgcn_readlane(e.place[i], __builtin_ctzll(in));
            in &= in - 1;
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
#pragma unroll
            for (int k = 0; k < PER; ++k) q[k] = e.place[k] == place ? sum : q[k];
        }
    }
}

// Gradient of this workgroup's tiles:
//   unlisted  2^(t - r2) * cu,  listed  (Q 2^(t - lse2) - q_v) * g / T,
// where r2 is the log2 of the unlisted sum and cu = (Q tail / S - q_t) g / T
// (TAIL), or of the whole sum and cu = Q g / T.  Referred to their own sum,
// the unlisted terms keep their precision however small their share is.  The
// first form is stored everywhere; then the wave stores its listed columns
// once more, an entry to a lane.  The listed logits are read before anything
// is stored (the gradient may take the logits' place).
template <int DT, int NR, bool TAIL, int PER>
__device__ __forceinline__ void gradient_tiles(const VocabGeom<NR> &g, const DistillArgs &a, const Teacher<PER> &t,
                                               const Entries<PER> &e, const RowSums &r, long long row, int first,
                                               int step, int lane) {
    constexpr int K = Lanes<DT>::value;
    const float gs = (a.grad_loss ? a.grad_loss[row] : 1.0f) * g.inv_t;
    if (!t.live || gs == 0.0f || (r.m == kNegInf && r.s == 0.0f)) {
        zero_tiles<DT>(g, row, first, step, lane);
        return;
    }
    VectorStream<DT, true, NR> stream;
    stream.start(g, row, first, lane);
    float z[PER], q[PER];
    char *out[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        z[i] = kNegInf;
        if (owned<DT>(e.place[i], first, step)) {
            z[i] = logit_at<DT>(g, row, t.id[i]);
            out[i] = column_at<DT, true>(g, row, t.id[i]);
        }
    }
    merge_repeats<DT>(e, t, first, step, q);
    const Ref ref = make_ref(r.m, g.c);
    const float lse2 = __builtin_log2f(r.s);
    float r2 = lse2, cu = t.total * gs;
    if constexpr (TAIL) {
        const bool none = r.tail2 == kNegInf;                  // no unlisted mass: nothing to scale
        r2 = none ? 0.0f : r.tail2;
        cu = none ? 0.0f : (t.total * exp2_fast(r.tail2 - lse2) - t.qt) * gs;
    }
    stream.run(g, row, step, lane, [&](const TileWalk &w, int u, int e0, int held, u32x4 raw) {
        Pack<DT> v = unpack<DT>(raw);
#pragma unroll
        for (int i = 0; i < K; ++i) v.v[i] = rel(v.v[i], ref);
#pragma unroll
        for (int i = 0; i < K; ++i) v.v[i] = exp2_fast(v.v[i] - r2) * cu;
        store_vec<DT>(grad_row_of<DT>(g, w.s, row), v, w.j, e0, held, w.w);
    });
    // after the vectors' stores, which other lanes of this wave have issued
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (owned<DT>(e.place[i], first, step))
            store1<DT>(out[i], 0, round_to<DT>((t.total * exp2_fast(rel(z[i], ref) - lse2) - q[i]) * gs));
    }
}

// Sums of a row (or of one part of it), the loss where the row is whole, and
// with BOTH its gradient by the same workgroup.
template <int DT, int NR, bool TAIL, bool BOTH, int PER>
__global__ __launch_bounds__(64 * kVocabWaves) void distill_kernel(const VocabGeom<NR> g, const DistillArgs a) {
    __shared__ Stats lds_tail[kVocabWaves], lds_listed[TAIL ? kVocabWaves : 1];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int waves = blockDim.x >> 6, step = waves * g.parts;
    const int local = blockIdx.x / g.parts, part = blockIdx.x - local * g.parts;
    const long long row = g.row0 + local;
    const int first = part * waves + wave;
    VectorStream<DT, !BOTH, NR> stream;
    stream.start(g, row, first, lane);
    const Teacher<PER> t = load_teacher<TAIL, PER>(a, row, g.col0[g.n], g.inv_t, lane);
    float z[PER];
    if (wave == 0 && g.parts == 1) listed_logits<DT>(g, t, row, z);
    Entries<PER> e;
    if constexpr (TAIL || BOTH) e = place_entries<DT>(g, t);

    Running run;
    if (t.live) {                                              // a row without a teacher is not read further
        stream.run(g, row, step, lane, [&](const TileWalk &w, int u, int e0, int held, u32x4 raw) {
            if (!full_tile<DT>(w.j, w.w)) mask_vec<DT>(raw, e0, held, w.w);
            if constexpr (TAIL) take_listed<DT, kTiny<NR>>(e, raw, w, u, lane);
            add_vec<DT, false>(run, unpack<DT>(raw), g.c);
        });
    }
    Stats st = run.st, li{kNegInf, 0.0f, 0.0f};
    block_stats<false>(st, lds_tail, waves, wave, lane, g.c);
    if constexpr (TAIL) {
#pragma unroll
        for (int i = 0; i < PER; ++i) li.m = __builtin_fmaxf(li.m, e.z[i]);
        const Ref ref = make_ref(li.m, g.c);
#pragma unroll
        for (int i = 0; i < PER; ++i) li.s += exp2_fast(rel(e.z[i], ref));
        block_stats<false>(li, lds_listed, waves, wave, lane, g.c);
    }
    if (g.parts > 1) {
        if (threadIdx.x == 0) a.part[row * g.parts + part] = make_float4(st.m, st.s, li.m, li.s);
        return;
    }
    const RowSums r = join_sums(st, li, g.c);
    if (wave == 0) {
        const float loss = row_loss<TAIL>(g, t, z, r, lane);
        if (lane == 0) write_row<NR>(a, row, r, loss);
    }
    if constexpr (BOTH) gradient_tiles<DT, NR, TAIL>(g, a, t, place_entries<DT>(g, t), r, row, first, step, lane);
}

// A row's loss from its parts: one wave, one lane per part.
template <int DT, int NR, bool TAIL, int PER>
__global__ __launch_bounds__(64) void distill_join_kernel(const VocabGeom<NR> g, const DistillArgs a) {
    const int lane = threadIdx.x;
    const long long row = g.row0 + blockIdx.x;
    const Teacher<PER> t = load_teacher<TAIL, PER>(a, row, g.col0[g.n], g.inv_t, lane);
    float z[PER];
    listed_logits<DT>(g, t, row, z);
    Stats st{kNegInf, 0.0f, 0.0f}, li{kNegInf, 0.0f, 0.0f};
    if (lane < g.parts) {
        const float4 p = a.part[row * g.parts + lane];
        st.m = p.x, st.s = p.y, li.m = p.z, li.s = p.w;
    }
    wave_stats<false>(st, lane, g.c);
    wave_stats<false>(li, lane, g.c);
    const RowSums r = join_sums(st, li, g.c);
    const float loss = row_loss<TAIL>(g, t, z, r, lane);
    if (lane == 0) write_row<NR>(a, row, r, loss);
}

template <int DT, int NR, bool TAIL, int PER>
__global__ __launch_bounds__(64 * kVocabWaves) void distill_backward_kernel(const VocabGeom<NR> g, const DistillArgs a) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int waves = blockDim.x >> 6;
    const int local = blockIdx.x / g.parts, part = blockIdx.x - local * g.parts;
    const long long row = g.row0 + local;
    const Teacher<PER> t = load_teacher<TAIL, PER>(a, row, g.col0[g.n], g.inv_t, lane);
    const float *o = a.saved + row * 4;
    const RowSums r{o[0], o[1], o[2]};
    gradient_tiles<DT, NR, TAIL>(g, a, t, place_entries<DT>(g, t), r, row, part * waves + wave, waves * g.parts, lane);
}

template <int DT, int NR, bool TAIL, int PER>
hipError_t run_distill(const VocabCall &c, const DistillArgs &a, VocabStage stage, hipStream_t s) {
    switch (stage) {
    case kForward: return launch_rows<NR>(c, a, distill_kernel<DT, NR, TAIL, false, PER>, c.parts, c.waves, s);
    case kBoth: return launch_rows<NR>(c, a, distill_kernel<DT, NR, TAIL, true, PER>, 1, c.waves, s);
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
