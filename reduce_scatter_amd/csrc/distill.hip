// distill.hip -- distillation from a teacher's top logits over
// vocabulary-split rows: the loss and its gradient.
//
// One pass over the logits as in logprobs.hip.  Where the teacher leaves mass
// to the unlisted entries, the student's mass on them is summed directly:
// the sum of everything less the listed terms would lose it to cancellation
// wherever the student is sure of a listed token.  Listed columns are found
// by one bit per vector of the row in LDS (64 vectors, one per lane, to a
// word that the whole wave reads at once); only marked vectors compare their
// columns with the list.
#include "dispatch.hpp"
#include "vocab_device.hpp"
#include "vocab_launch.hpp"

namespace ar {

constexpr int kTeacherPer = kTeacherMax / 64;      // entries per lane
constexpr float kTailLeast = 0x1p-20f;             // a remaining mass below this is the values' rounding

// The teacher's distribution of a row, entry k of it in lane k % 64.
struct Teacher {
    int id[kTeacherPer];                           // -1: padding
    float q[kTeacherPer], lq[kTeacherPer];         // probability and its logarithm
    float qt, total;                               // remaining mass, sum of everything
    bool live;                                     // has entries
};
template <bool TAIL>
__device__ __forceinline__ Teacher load_teacher(const DistillArgs &a, long long row, int vocab, float inv_t, int lane) {
    Teacher t;
    float m = kNegInf;
    bool any = false;
#pragma unroll
    for (int i = 0; i < kTeacherPer; ++i) {
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
        for (int i = 0; i < kTeacherPer; ++i) sum += t.q[i] = expf(t.lq[i]);
        sum = wave_sum(sum);
        t.qt = 1.0f - sum;
        t.qt = t.qt < kTailLeast ? 0.0f : t.qt;
        t.total = sum + t.qt;
    } else {
        m = wave_max(m);
        t.live = m != kNegInf;
#pragma unroll
        for (int i = 0; i < kTeacherPer; ++i) {
            t.lq[i] = t.live ? (t.lq[i] - m) * inv_t : kNegInf;
            sum += expf(t.lq[i]);
        }
        sum = wave_sum(sum);
        const float ls = logf(sum);
#pragma unroll
        for (int i = 0; i < kTeacherPer; ++i) {
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
template <int DT, int NR, bool TAIL>
__device__ __forceinline__ float row_loss(const VocabGeom<NR> &g, const Teacher &t, const RowSums &r, long long row) {
    const Ref ref = make_ref(r.m, g.c);
    const bool empty = r.m == kNegInf && r.s == 0.0f;
    const float lse = logf(r.s);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kTeacherPer; ++i) {
        if (t.id[i] >= 0 && t.q[i] != 0.0f) {
            const float lp = empty ? kNegInf : rel_ln(logit_at<DT>(g, row, t.id[i]), ref, g.c, g.inv_t) - lse;
            sum += t.q[i] * (t.lq[i] - lp);
        }
    }
    sum = wave_sum(sum);
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

// The teacher's list as the tile walk needs it.
struct Listed {
    int id[kTeacherMax];
    float q[kTeacherMax];
};

// Put the list into LDS and set the bit of every vector of this workgroup
// that holds a listed column: mark[(i * U + u) * waves + wave] for the wave's
// i-th tile.  All waves call it; `words` is the length of mark.
template <int DT, int NR>
__device__ __forceinline__ void mark_listed(const VocabGeom<NR> &g, const Teacher &t, Listed &l, u64 *mark, int words,
                                            int k, int part, int waves, int wave, int lane) {
    for (int i = threadIdx.x; i < words; i += waves * 64) mark[i] = 0;
    __syncthreads();
    if (wave == 0) {
        const int step = waves * g.parts;
#pragma unroll
        for (int i = 0; i < kTeacherPer; ++i) {
            if (i * 64 >= k) break;
            l.id[i * 64 + lane] = t.id[i];
            l.q[i * 64 + lane] = t.q[i];
            if (t.id[i] >= 0) {
                const Place p = place_of<DT>(g, t.id[i]);
                const int owner = p.t % step;
                if (owner / waves == part)
                    atomicOr(mark + ((p.t / step) * kVocabU + p.u) * waves + owner % waves, 1ull << p.lane);
            }
        }
    }
    __syncthreads();
}

// For a marked vector whose first column is col: which of its columns are
// listed (bits), and with Q the teacher's probability on each.
template <int DT, bool Q>
__device__ __forceinline__ uint32_t listed_in(const Listed &l, int k, int col, float *q) {
    constexpr int K = Lanes<DT>::value;
    uint32_t bits = 0;
    if constexpr (Q) {
#pragma unroll
        for (int i = 0; i < K; ++i) q[i] = 0.0f;
    }
    for (int e = 0; e < k; ++e) {
        const int id = l.id[e], d = id - col;
        if (id >= 0 && d >= 0 && d < K) {
            bits |= 1u << d;
            if constexpr (Q) {
#pragma unroll
                for (int i = 0; i < K; ++i) q[i] += i == d ? l.q[e] : 0.0f;
            }
        }
    }
    return bits;
}

// Gradient of this workgroup's tiles:
//   unlisted  2^(t - r2) * cu,  listed  (Q 2^(t - lse2) - q_v) * g / T,
// where r2 is the log2 of the unlisted sum and cu = (Q tail / S - q_t) g / T
// (TAIL), or of the whole sum and cu = Q g / T.  Referred to their own sum,
// the unlisted terms keep their precision however small their share is.
template <int DT, int NR, bool TAIL>
__device__ __forceinline__ void gradient_tiles(const VocabGeom<NR> &g, const DistillArgs &a, const Teacher &t,
                                               const Listed &l, const u64 *mark, const RowSums &r, long long row,
                                               int part, int waves, int wave, int lane) {
    constexpr int K = Lanes<DT>::value;
    const float gs = (a.grad_loss ? a.grad_loss[row] : 1.0f) * g.inv_t;
    const bool zero = !t.live || gs == 0.0f || (r.m == kNegInf && r.s == 0.0f);
    const Ref ref = make_ref(r.m, g.c);
    const float lse2 = __builtin_log2f(r.s);
    float r2 = lse2, cu = t.total * gs;
    if constexpr (TAIL) {
        const bool none = r.tail2 == kNegInf;                  // no unlisted mass: nothing to scale
        r2 = none ? 0.0f : r.tail2;
        cu = none ? 0.0f : (t.total * exp2_fast(r.tail2 - lse2) - t.qt) * gs;
    }
    const int step = waves * g.parts, first = part * waves + wave;
    TileWalk w{0, first};
    int ord = wave;
    for (w.settle<DT>(g); w.s < g.n; w.j += step, ord += kVocabU * waves, w.settle<DT>(g)) {
        const int width = width_of<DT>(g, w.s);
        char *out = grad_row_of<DT>(g, w.s, row);
        Tile<DT> x;
        if (zero) {
#pragma unroll
            for (int u = 0; u < kVocabU; ++u)
#pragma unroll
                for (int i = 0; i < K; ++i) x.v[u].v[i] = 0.0f;
        } else {
            load_tile<DT>(x, row_of<DT>(g, w.s, row), w.j, width, lane);
#pragma unroll
            for (int u = 0; u < kVocabU; ++u) {
                const u64 word = mark[ord + u * waves];
                Pack<DT> &v = x.v[u];
                if (ref.wide) {
#pragma unroll
                    for (int i = 0; i < K; ++i) v.v[i] = rel(v.v[i], ref, g.c);
                } else {
#pragma unroll
                    for (int i = 0; i < K; ++i) v.v[i] = __builtin_fmaf(v.v[i], g.c, -ref.y);
                }
                float q[K];
                uint32_t bits = 0;
                if (word >> lane & 1) bits = listed_in<DT, true>(l, a.k, g.col0[w.s] + elem0<DT>(w.j, u, lane), q);
                if (word) {
#pragma unroll
                    for (int i = 0; i < K; ++i)
                        v.v[i] = bits >> i & 1 ? (t.total * exp2_fast(v.v[i] - lse2) - q[i]) * gs
                                               : exp2_fast(v.v[i] - r2) * cu;
                } else {
#pragma unroll
                    for (int i = 0; i < K; ++i) v.v[i] = exp2_fast(v.v[i] - r2) * cu;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kVocabU; ++u) store_vec<DT>(out, x.v[u], elem0<DT>(w.j, u, lane), width);
    }
}

// Sums of a row (or of one part of it), the loss where the row is whole, and
// with BOTH its gradient by the same workgroup.
template <int DT, int NR, bool TAIL, bool BOTH>
__global__ __launch_bounds__(64 * kVocabWaves) void distill_kernel(const VocabGeom<NR> g, const DistillArgs a,
                                                                   const int words) {
    constexpr bool MARK = TAIL || BOTH;
    constexpr int K = Lanes<DT>::value;
    __shared__ Stats lds_tail[kVocabWaves], lds_listed[TAIL ? kVocabWaves : 1];
    __shared__ Listed lds_list[1];
    extern __shared__ u64 mark[];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int waves = blockDim.x >> 6, step = waves * g.parts;
    const int local = blockIdx.x / g.parts, part = blockIdx.x - local * g.parts;
    const long long row = g.row0 + local;
    const Teacher t = load_teacher<TAIL>(a, row, g.col0[g.n], g.inv_t, lane);
    if constexpr (MARK) mark_listed<DT>(g, t, lds_list[0], mark, words, a.k, part, waves, wave, lane);

    Stats st{kNegInf, 0.0f, 0.0f}, li{kNegInf, 0.0f, 0.0f};
    Ref ref = make_ref(kNegInf, g.c);
    float limit = kNegInf;
    TileWalk w{0, part * waves + wave};
    int ord = wave;
    if (t.live) {                                              // a row without a teacher is not read
        for (w.settle<DT>(g); w.s < g.n; w.j += step, ord += kVocabU * waves, w.settle<DT>(g)) {
            Tile<DT> x;
            load_tile<DT>(x, row_of<DT>(g, w.s, row), w.j, width_of<DT>(g, w.s), lane);
            float tm = kNegInf;
#pragma unroll
            for (int u = 0; u < kVocabU; ++u) {
                if constexpr (TAIL) {
                    if (mark[ord + u * waves] >> lane & 1) {
                        const uint32_t bits =
                            listed_in<DT, false>(lds_list[0], a.k, g.col0[w.s] + elem0<DT>(w.j, u, lane), nullptr);
#pragma unroll
                        for (int i = 0; i < K; ++i) {
                            if (bits >> i & 1) {
                                const float v = x.v[u].v[i];
                                if (v > li.m) shift_stats(li, v, g.c);
                                li.s += exp2_fast(rel(v, make_ref(li.m, g.c), g.c));
                                x.v[u].v[i] = kNegInf;
                            }
                        }
                    }
                }
                tm = __builtin_fmaxf(tm, vec_max<DT>(x.v[u]));
            }
            add_tile<DT, false>(st, ref, limit, x, tm, g.c, g.slack);
        }
    }
    block_stats<false>(st, lds_tail, waves, wave, lane, g.c);
    if constexpr (TAIL) block_stats<false>(li, lds_listed, waves, wave, lane, g.c);
    if (g.parts > 1) {
        if (threadIdx.x == 0) a.part[row * g.parts + part] = make_float4(st.m, st.s, li.m, li.s);
        return;
    }
    const RowSums r = join_sums(st, li, g.c);
    if (wave == 0) {
        const float loss = row_loss<DT, NR, TAIL>(g, t, r, row);
        if (lane == 0) write_row<NR>(a, row, r, loss);
    }
    if constexpr (BOTH) {
        __syncthreads();                                       // the listed logits are read before any is overwritten
        gradient_tiles<DT, NR, TAIL>(g, a, t, lds_list[0], mark, r, row, part, waves, wave, lane);
    }
}

// A row's loss from its parts: one wave, one lane per part.
template <int DT, int NR, bool TAIL>
__global__ __launch_bounds__(64) void distill_join_kernel(const VocabGeom<NR> g, const DistillArgs a) {
    const int lane = threadIdx.x;
    const long long row = g.row0 + blockIdx.x;
    const Teacher t = load_teacher<TAIL>(a, row, g.col0[g.n], g.inv_t, lane);
    Stats st{kNegInf, 0.0f, 0.0f}, li{kNegInf, 0.0f, 0.0f};
    if (lane < g.parts) {
        const float4 p = a.part[row * g.parts + lane];
        st.m = p.x, st.s = p.y, li.m = p.z, li.s = p.w;
    }
    wave_stats<false>(st, g.c);
    wave_stats<false>(li, g.c);
    const RowSums r = join_sums(st, li, g.c);
    const float loss = row_loss<DT, NR, TAIL>(g, t, r, row);
    if (lane == 0) write_row<NR>(a, row, r, loss);
}

template <int DT, int NR, bool TAIL>
__global__ __launch_bounds__(64 * kVocabWaves) void distill_backward_kernel(const VocabGeom<NR> g, const DistillArgs a,
                                                                            const int words) {
    __shared__ Listed lds_list;
    extern __shared__ u64 mark[];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int waves = blockDim.x >> 6;
    const int local = blockIdx.x / g.parts, part = blockIdx.x - local * g.parts;
    const long long row = g.row0 + local;
    const Teacher t = load_teacher<TAIL>(a, row, g.col0[g.n], g.inv_t, lane);
    mark_listed<DT>(g, t, lds_list, mark, words, a.k, part, waves, wave, lane);
    const float *o = a.saved + row * 4;
    const RowSums r{o[0], o[1], o[2]};
    gradient_tiles<DT, NR, TAIL>(g, a, t, lds_list, mark, r, row, part, waves, wave, lane);
}

template <int DT, int NR, bool TAIL>
hipError_t run_distill(const VocabCall &c, const DistillArgs &a, VocabStage stage, hipStream_t s) {
    const int step = c.waves * c.parts;
    const int words = (c.tiles + step - 1) / step * kVocabU * c.waves;
    const size_t lds = (size_t)words * sizeof(unsigned long long);
    switch (stage) {
    case kForward:
        return launch_rows<NR>(c, a, distill_kernel<DT, NR, TAIL, false>, c.parts, c.waves, TAIL ? lds : 0, s, words);
    case kBoth: return launch_rows<NR>(c, a, distill_kernel<DT, NR, TAIL, true>, 1, c.waves, lds, s, words);
    case kBackward: return launch_rows<NR>(c, a, distill_backward_kernel<DT, NR, TAIL>, c.parts, c.waves, lds, s, words);
    default: return launch_rows<NR>(c, a, distill_join_kernel<DT, NR, TAIL>, 1, 1, 0, s);
    }
}

hipError_t launch_distill(const VocabCall &c, const DistillArgs &a, bool tail, VocabStage stage, hipStream_t s) {
    return dispatch_vocab(c, [&](auto dt, auto nr) {
        return tail ? run_distill<dt.value, nr.value, true>(c, a, stage, s)
                    : run_distill<dt.value, nr.value, false>(c, a, stage, s);
    });
}

}  // namespace ar
