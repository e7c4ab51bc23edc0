// logprobs.hip -- log probabilities of given tokens with entropy and top
// alternatives over vocabulary-split rows, and their gradient.
//
// One pass over the logits: every lane keeps the sums of 2^t and t*2^t of its
// vectors relative to a running reference (vocab_device.hpp) and, for the top
// alternatives, its largest logit with the vector it stands in.  That costs
// the stream nothing more, and it is enough: the k largest logits of a row
// lie in the k lanes whose best logits come first in the (value, column)
// order, so after the pass the best-of-lane keys are sorted, and every wave
// reads those of its lanes that are among the k once more (k / (64 W) of the
// row in all); what is not below the k-th of them, seldom much more than k
// logits, is collected and sorted.  The work is bounded whatever the order of
// the logits.
#include "dispatch.hpp"
#include "vocab_device.hpp"
#include "vocab_launch.hpp"

namespace ar {

// The statistics and results of a row once its sums are whole.
struct RowResult {
    float lse;                         // ln of the sum relative to the reference
    float entropy;
    bool empty;                        // no distribution: every logit -inf
};
__device__ __forceinline__ RowResult row_result(const Stats &st) {
    RowResult r;
    r.empty = st.m == kNegInf && st.s == 0.0f;
    r.lse = logf(st.s);
    const float h = r.lse - kLn2 * (st.s1 / st.s);
    r.entropy = r.empty || h < 0.0f ? 0.0f : h;
    return r;
}

template <int NR>
__device__ __forceinline__ void write_row(const VocabGeom<NR> &g, const LogprobsArgs &a, long long row, const Stats &st,
                                          const RowResult &res, float xt, bool token) {
    const Ref ref = make_ref(st.m, g.c);
    if (a.logprobs) a.logprobs[row] = !token ? 0.0f : res.empty ? kNegInf : rel_ln(xt, ref, g.inv_t) - res.lse;
    if (a.entropy) a.entropy[row] = res.entropy;
    if (a.saved) {
        float *o = a.saved + row * 4;
        o[0] = st.m;
        o[1] = st.s;
        o[2] = res.entropy;
        o[3] = 0.0f;
    }
}

template <int NR>
__device__ __forceinline__ void write_top(const VocabGeom<NR> &g, const LogprobsArgs &a, long long row, const Stats &st,
                                          const RowResult &res, u64 key, int i) {
    const Ref ref = make_ref(st.m, g.c);
    const float x = order_value((uint32_t)(key >> 32));
    a.top_ids[row * a.k + i] = key ? (int64_t)key_col(key) : -1;
    a.top_logprobs[row * a.k + i] = !key || res.empty ? kNegInf : rel_ln(x, ref, g.inv_t) - res.lse;
}

// f(keys) with those keys (0: none) that are not below `least` among the
// logits of this wave's lanes in `pending`.  A load takes the vectors of two
// of those lanes in eight tiles (a vector to a lane), four loads at a time are
// in flight, and where the tiles lie is worked out once for all of them.
template <int DT, int NR, typename F>
__device__ __forceinline__ void each_key(const VocabGeom<NR> &g, long long row, u64 lanes, u64 least, int first,
                                         int step, int lane, F f) {
    constexpr int K = Lanes<DT>::value, kAhead = 4;
    const float floor = order_value((uint32_t)(least >> 32));
    const int half = lane >> 5, tile = (lane & 31) / kVocabU, u = lane % kVocabU;
    for (int base = first; base < g.tiles; base += 8 * step) {
        const int t = base + tile * step;
        int s = 0, before = 0, tiles = 0;
        each_later_rank(g, [&](int r) {
            tiles += tiles_of<DT>(g, r - 1);
            s = t >= tiles ? r : s;
            before = t >= tiles ? tiles : before;
        });
        const bool there = t < g.tiles;
        s = there ? s : 0;
        const int w = there ? width_of<DT>(g, s) : 0, col = g.col0[s], j = t - before;
        const char *x = row_of<DT>(g, s, row);
        const int phase = phase_of<DT, kTiny<NR>>(x, w);
        for (u64 pending = lanes; pending;) {
            u32x4 v[kAhead];
            int e0[kAhead];
            const int loads = (__builtin_popcountll(pending) + 1) / 2;
#pragma unroll
            for (int b = 0; b < kAhead; ++b) {
                if (b >= loads) break;
                const int one = pending ? __builtin_ctzll(pending) : -1;
                pending &= pending - 1;
                const int two = pending ? __builtin_ctzll(pending) : -1;
                pending &= pending - 1;
                const int from = half ? two : one;
                e0[b] = ((j * kVocabU + u) * 64 + from) * K - phase;
                if (!there || from < 0 || e0[b] >= w) {
                    e0[b] = w;
                } else if (kTiny<NR> && w < K) {
                    v[b] = u32x4{0, 0, 0, 0};
#pragma unroll
                    for (int i = 0; i < K; ++i) {
                        if (i >= w) continue;
                        if constexpr (DT == F32) v[b][i] = ((const uint32_t *)x)[i];
                        else v[b][i / 2] |= (uint32_t)((const uint16_t *)x)[i] << (i & 1) * 16;
                    }
                } else {
                    v[b] = *(const u32x4e *)(x + (uint32_t)held0<DT, false>(e0[b], w) * elem_bytes<DT>());
                }
            }
            // one copy of what follows, and of f, which may be long
#pragma unroll 1
            for (int b = 0; b < loads && b < kAhead; ++b) {
                u32x4 raw = v[0];
                int from = e0[0];
#pragma unroll
                for (int i = 1; i < kAhead; ++i) {
                    raw = b == i ? v[i] : raw;
                    from = b == i ? e0[i] : from;
                }
                const Pack<DT> z = unpack<DT>(raw);
                const int held = held0<DT, kTiny<NR>>(from, w);
                uint32_t hits = 0;
#pragma unroll
                for (int i = 0; i < K; ++i) hits |= z.v[i] < floor ? 0 : 1u << i;
                hits = from < w ? hits : 0;
                while (__any(hits != 0)) {
                    const int i = __builtin_ctz(hits | 1u << K);
                    float x = z.v[0];
#pragma unroll
                    for (int k = 1; k < K; ++k) x = i == k ? z.v[k] : x;
                    u64 key = top_key(x, col + held + i);
                    if (!hits || held + i < from || held + i >= from + K || held + i >= w || key < least) key = 0;
                    hits &= hits - 1;
                    if (__any(key != 0)) f(key);
                }
            }
        }
    }
}

struct TopScratch {
    u64 keys[kVocabWaves * 64];
    u64 last;                          // the k-th best lane's key
    int count;                         // keys collected
};

// emit(i, key) for the i-th largest key (0: none) of this workgroup's part of
// the row, i < k; best / col: each lane's largest logit and the first column
// of its vector (col < 0: none).
template <int DT, int NR, typename F>
__device__ __forceinline__ void select_top(const VocabGeom<NR> &g, long long row, float best, int col, int k,
                                           TopScratch &lds, int waves, int wave, int first, int lane, F emit) {
    const int step = waves * g.parts, room = waves * 64, thread = wave * 64 + lane;
    // the k-th best lane: every wave's lanes in order, and for each its rank among all
    const u64 key = col >= 0 ? top_key(best, col) : 0;
    const u64 mine = sort_down(key, lane);
    lds.keys[thread] = mine;
    for (int i = thread + room; i < kVocabWaves * 64; i += room) lds.keys[i] = 0;
    if (thread == 0) lds.last = 0, lds.count = 0;
    __syncthreads();
    if (lane < k && mine && count_larger<kVocabWaves>(lds.keys, mine) == k - 1) lds.last = mine;
    __syncthreads();
    const u64 last = lds.last;
    // its logit stands in that vector, so k logits at least have keys from here on
    const u64 least = last ? last - (Lanes<DT>::value - 1) : 1;
    const u64 lanes = __ballot(key != 0 && key >= last);
    each_key<DT>(g, row, lanes, least, first, step, lane, [&](u64 v) {
        if (v) {
            const int at = atomicAdd(&lds.count, 1);
            if (at < room) lds.keys[at] = v;
        }
    });
    __syncthreads();
    const int n = lds.count;
    if (n <= room) {                                                   // rank them by counting
        const u64 v = thread < n ? lds.keys[thread] : 0;
        int rank = 0;
        for (int i = 0; i < n; i += 8) {
#pragma unroll
            for (int b = 0; b < 8; ++b) rank += (lds.keys[i + b] > v) & (i + b < n);    // the array's length is a multiple of 8
        }
        if (thread < n && rank < k) emit(rank, v);
        if (thread >= n && thread < k) emit(thread, 0);
        return;
    }
    // more than fit (long runs of logits in order): every wave keeps the 64 largest of its own
    u64 v = 0;
    each_key<DT>(g, row, lanes, least, first, step, lane,
                 [&](u64 c) { v = merge_lists(v, reversed(sort_down(c, lane), lane), lane); });
    v = block_lists(v, lds.keys, waves, wave, lane);
    if (thread < k) emit(thread, v);
}

// Gradient of a row: with e = 2^t and p = e / S, t relative to m,
//   dx = [v = target] gl/T + e * (a0 + a1 t),
//   a0 = -(gl + gh (H - ln S)) / (T S),  a1 = -gh ln2 / (T S),
// and where term() gives t + d instead: a0 - d a1 for a0, both times 2^-d.
struct RowGradient {
    Ref ref;
    float a0, a1, at_target;
    Place p;                           // of the target
    bool zero;
};
template <int DT, int NR>
__device__ __forceinline__ RowGradient row_gradient(const VocabGeom<NR> &g, const LogprobsArgs &a, long long row,
                                                    const Stats &st, const RowResult &res, int target) {
    const float gl = a.grad_logprobs && target >= 0 ? a.grad_logprobs[row] : 0.0f;
    const float gh = a.grad_entropy ? a.grad_entropy[row] : 0.0f;
    RowGradient r;
    r.ref = make_ref(st.m, g.c);
    r.a0 = -(gl + gh * (res.entropy - res.lse)) * g.inv_t / st.s;
    r.a1 = -gh * kLn2 * g.inv_t / st.s;
    if constexpr (DT != F32) {
        const float d = term_shift<DT>(r.ref), f = exp2_fast(-d);
        r.a0 = __builtin_fmaf(-d, r.a1, r.a0) * f;
        r.a1 *= f;
    }
    r.at_target = gl * g.inv_t;
    r.p = target >= 0 ? place_of<DT>(g, row, target) : Place{0, 0, -1, 0};
    r.zero = res.empty || (gl == 0.0f && gh == 0.0f);
    return r;
}
template <int DT, int NR>
__device__ __forceinline__ void gradient_vec(const VocabGeom<NR> &g, const RowGradient &r, long long row,
                                             const TileWalk &t, int e0, int held, u32x4 raw) {
    constexpr int K = Lanes<DT>::value;
    Pack<DT> x = unpack<DT>(raw);
    if (r.a1 == 0.0f) {
#pragma unroll
        for (int i = 0; i < K; ++i) x.v[i] = term<DT>(x.v[i], r.ref, g).e * r.a0;
    } else {
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const Term y = term<DT>(x.v[i], r.ref, g);
            x.v[i] = y.e * __builtin_fmaf(hold_up(y.t, kTLow), r.a1, r.a0);
        }
    }
    if (t.at == r.p.t) {
        const int d = t.j * kTileElems<DT> + r.p.et - t.phase - held;
#pragma unroll
        for (int i = 0; i < K; ++i) x.v[i] += i == d ? r.at_target : 0.0f;
    }
    store_vec<DT>(grad_row_of<DT>(g, t.s, row), x, t, e0, held);
}
template <int DT, int NR>
__device__ __forceinline__ void gradient_tiles(const VocabGeom<NR> &g, const RowGradient &r, long long row, int first,
                                               int step, int lane) {
    if (r.zero) {
        zero_tiles<DT>(g, row, first, step, lane);
        return;
    }
    VectorStream<DT, true, NR> stream;
    stream.start(g, row, first, lane);
    stream.run(g, row, step, lane, [&](const TileWalk &t, int, int e0, int held, u32x4 raw) {
        gradient_vec<DT>(g, r, row, t, e0, held, raw);
    });
}

__device__ __forceinline__ int token_of(const LogprobsArgs &a, long long row, int vocab) {
    const int64_t t = a.targets[row];
    return t >= 0 && t < vocab ? (int)t : -1;
}

// Statistics of a row (or of one part of it), the results where the row is
// whole, and with BOTH its gradient by the same workgroup.  AGAIN: the logits
// will be read again soon and are left in the caches.
// Bound by HBM where rows are many: 8192 x 131072 bf16 with entropy 331 us, 6.5
// of the 7.1 TB/s that a bare read reaches (about 6.4 instructions a logit
// take 3/4 of the issue slots meanwhile).  With few rows by its dependent
// steps: one row of 32768 takes 4 us, 9 with alternatives.
template <int DT, int NR, bool S1, bool TOP, bool BOTH, bool AGAIN>
__global__ __launch_bounds__(64 * kVocabWaves) void logprobs_kernel(const VocabGeom<NR> g, const LogprobsArgs a) {
    __shared__ Stats lds_stats[kVocabWaves];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int waves = blockDim.x >> 6, step = waves * g.parts;
    const int local = blockIdx.x / g.parts, part = blockIdx.x - local * g.parts;
    const long long row = g.row0 + local;
    const int first = part * waves + wave;
    VectorStream<DT, !AGAIN, NR> stream;
    stream.start(g, row, first, lane);
    const int target = token_of(a, row, g.col0[g.n]);

    Running run;
    float best = kNegInf;
    int best_col = -1;
    stream.run(g, row, step, lane, [&](const TileWalk &t, int u, int e0, int held, u32x4 raw) {
        if (!t.template full<DT>()) mask_vec<DT>(raw, e0, held, t.w);
        const Pack<DT> v = unpack<DT>(raw);
        if constexpr (TOP) {
            float m = kNegInf;                                                     // NaN: ordered as -inf
#pragma unroll
            for (int i = 0; i < Lanes<DT>::value; ++i) m = __builtin_fmaxf(m, v.v[i]);
            if (e0 < t.w && (m > best || best_col < 0)) {
                best = m;
                best_col = t.col + max(e0, 0);
            }
        }
        if (u == 0) end_tile(run);
        add_vec<DT, S1>(run, v, g);
    });
    float xt = 0.0f;
    if (wave == 0 && g.parts == 1 && target >= 0) xt = logit_at<DT>(g, row, target);
    Stats sum = total(run);
    block_stats<S1>(sum, lds_stats, waves, wave, lane, g.c);
    const Stats st = settled(sum, g.c);
    const RowResult res = row_result(st);
    const long long slot = row * g.parts + part;
    if (threadIdx.x == 0) {
        if (g.parts > 1) a.part[slot] = make_float4(sum.m, sum.s, sum.s1, 0.0f);
        else write_row(g, a, row, st, res, xt, target >= 0);
    }
    if constexpr (TOP) {
        __shared__ TopScratch lds_top;
        select_top<DT>(g, row, best, best_col, a.k, lds_top, waves, wave, first, lane, [&](int i, u64 key) {
            if (g.parts > 1) a.part_top[slot * a.k + i] = key;
            else write_top(g, a, row, st, res, key, i);
        });
    }
    if constexpr (BOTH) gradient_tiles<DT>(g, row_gradient<DT>(g, a, row, st, res, target), row, first, step, lane);
}

// A row's results from its parts: one lane per part for the statistics, one
// wave per part (in turn) for the lists.  4.5 us, a launch and two dependent reads.
template <int DT, int NR, bool S1, bool TOP>
__global__ __launch_bounds__(64 * kVocabWaves) void logprobs_join_kernel(const VocabGeom<NR> g, const LogprobsArgs a) {
    __shared__ u64 lds_keys[TOP ? kVocabWaves * 64 : 1];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int waves = blockDim.x >> 6;
    const long long row = g.row0 + blockIdx.x;
    const int target = token_of(a, row, g.col0[g.n]);
    const float xt = target >= 0 ? logit_at<DT>(g, row, target) : 0.0f;
    Stats st{kNegInf, 0.0f, 0.0f};
    if (lane < g.parts) {
        const float4 p = a.part[row * g.parts + lane];
        st = Stats{p.x, p.y, p.z};
    }
    wave_stats<S1>(st, lane, g.c);
    st = settled(st, g.c);
    const RowResult res = row_result(st);
    if (threadIdx.x == 0) write_row(g, a, row, st, res, xt, target >= 0);
    if constexpr (TOP) {
        u64 v = 0;
        for (int p = wave; p < g.parts; p += waves) {
            const int i = 63 - lane;                               // ascending
            const u64 b = i < a.k ? a.part_top[(row * g.parts + p) * a.k + i] : 0;
            v = merge_lists(v, b, lane);
        }
        v = block_lists(v, lds_keys, waves, wave, lane);
        if (wave == 0 && lane < a.k) write_top(g, a, row, st, res, v, lane);
    }
}

// Gradients from saved statistics, one read and one write of the logits'
// bytes: 4096 x 131072 bf16 with an entropy term 374 us, 5.7 TB/s (non-temporal
// stores; plain ones 10 % slower).
template <int DT, int NR>
__global__ __launch_bounds__(64 * kVocabWaves) void logprobs_backward_kernel(const VocabGeom<NR> g, const LogprobsArgs a) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int waves = blockDim.x >> 6;
    const int local = blockIdx.x / g.parts, part = blockIdx.x - local * g.parts;
    const long long row = g.row0 + local;
    const float *o = a.saved + row * 4;
    const Stats st{o[0], o[1], 0.0f};
    RowResult res;
    res.empty = st.m == kNegInf && st.s == 0.0f;
    res.lse = logf(st.s);
    res.entropy = o[2];
    const RowGradient r = row_gradient<DT>(g, a, row, st, res, token_of(a, row, g.col0[g.n]));
    gradient_tiles<DT>(g, r, row, part * waves + wave, waves * g.parts, lane);
}

// Results and gradient of a row held in the workgroup's registers: one read
// and one write.  8192 x 32768 bf16 197 us, 5.5 TB/s (read twice: 220 us).
template <int DT, int NR, bool S1, int T>
__global__ __launch_bounds__(64 * kHeldWaves) void logprobs_held_kernel(const VocabGeom<NR> g, const LogprobsArgs a) {
    __shared__ Stats lds_stats[kHeldWaves];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int waves = blockDim.x >> 6;
    const long long row = g.row0 + blockIdx.x;
    HeldTiles<DT, NR, T> tiles;
    tiles.start(g, row, wave, waves, lane);
    const int target = token_of(a, row, g.col0[g.n]);
    const float xt = wave == 0 && target >= 0 ? logit_at<DT>(g, row, target) : 0.0f;
    Stats st = held_sums<DT, S1>(g, tiles, lane, [](int, int, int, int, u32x4 &) {});
    block_stats<S1>(st, lds_stats, waves, wave, lane, g.c);
    st = settled(st, g.c);
    const RowResult res = row_result(st);
    if (threadIdx.x == 0) write_row(g, a, row, st, res, xt, target >= 0);
    const RowGradient r = row_gradient<DT>(g, a, row, st, res, target);
    if (r.zero) {
        zero_tiles<DT>(g, row, wave, waves, lane);
        return;
    }
    tiles.each(lane, [&](const TileWalk &t, int, int, int e0, int held, u32x4 raw) {
        gradient_vec<DT>(g, r, row, t, e0, held, raw);
    });
}

template <int DT, int NR>
hipError_t run_logprobs(const VocabCall &c, const LogprobsArgs &a, VocabStage stage, hipStream_t s) {
    const bool s1 = a.entropy || a.saved || a.grad_entropy, top = a.k > 0;
    if (stage == kBackward) return launch_rows<NR>(c, a, logprobs_backward_kernel<DT, NR>, c.parts, c.waves, s);
    if (stage == kBoth && c.held == 1)
        return s1 ? launch_rows<NR>(c, a, logprobs_held_kernel<DT, NR, true, 1>, 1, c.waves, s)
                  : launch_rows<NR>(c, a, logprobs_held_kernel<DT, NR, false, 1>, 1, c.waves, s);
    if (stage == kBoth && c.held == 2)
        return s1 ? launch_rows<NR>(c, a, logprobs_held_kernel<DT, NR, true, 2>, 1, c.waves, s)
                  : launch_rows<NR>(c, a, logprobs_held_kernel<DT, NR, false, 2>, 1, c.waves, s);
    if (stage == kBoth && c.held)
        return s1 ? launch_rows<NR>(c, a, logprobs_held_kernel<DT, NR, true, kHeldTiles>, 1, c.waves, s)
                  : launch_rows<NR>(c, a, logprobs_held_kernel<DT, NR, false, kHeldTiles>, 1, c.waves, s);
    if (stage == kBoth) {
        return s1 ? launch_rows<NR>(c, a, logprobs_kernel<DT, NR, true, false, true, true>, 1, c.waves, s)
                  : launch_rows<NR>(c, a, logprobs_kernel<DT, NR, false, false, true, true>, 1, c.waves, s);
    }
    if (stage == kForward) {
        if (top && c.again)
            return launch_rows<NR>(c, a, logprobs_kernel<DT, NR, true, true, false, true>, c.parts, c.waves, s);
        if (top) return s1 ? launch_rows<NR>(c, a, logprobs_kernel<DT, NR, true, true, false, false>, c.parts, c.waves, s)
                           : launch_rows<NR>(c, a, logprobs_kernel<DT, NR, false, true, false, false>, c.parts, c.waves, s);
        if (c.again) return launch_rows<NR>(c, a, logprobs_kernel<DT, NR, true, false, false, true>, c.parts, c.waves, s);
        return s1 ? launch_rows<NR>(c, a, logprobs_kernel<DT, NR, true, false, false, false>, c.parts, c.waves, s)
                  : launch_rows<NR>(c, a, logprobs_kernel<DT, NR, false, false, false, false>, c.parts, c.waves, s);
    }
    int w = 1;
    while (top && w < c.parts && w < kVocabWaves) w *= 2;
    if (top) return s1 ? launch_rows<NR>(c, a, logprobs_join_kernel<DT, NR, true, true>, 1, w, s)
                       : launch_rows<NR>(c, a, logprobs_join_kernel<DT, NR, false, true>, 1, w, s);
    return s1 ? launch_rows<NR>(c, a, logprobs_join_kernel<DT, NR, true, false>, 1, w, s)
              : launch_rows<NR>(c, a, logprobs_join_kernel<DT, NR, false, false>, 1, w, s);
}

hipError_t launch_logprobs(const VocabCall &c, const LogprobsArgs &a, VocabStage stage, hipStream_t s) {
    return dispatch_vocab(c, [&](auto dt, auto nr) { return run_logprobs<dt.value, nr.value>(c, a, stage, s); });
}

}  // namespace ar
