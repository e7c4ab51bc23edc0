// embed.hip -- embedding lookup from a table split by vocabulary entries over
// n rank buffers, and its gradient.
//
//   out[t] = scale table[token_t],   grad[v] = scale sum_{t : token_t = v} g[t]
//
// The lookup reads the ranks' rows where they are: the sum over ranks of rows
// that all but one leave zero needs no adding.  The gradient sorts the tokens,
// so that equal ones stand together and no sum needs atomics: the sorted
// positions are cut into pieces of fixed length, a workgroup adds up the runs
// of equal tokens in one piece, and the few runs that cross a piece's end are
// joined by a second launch.  Entries without a token are written as zeros by
// further workgroups of the same launch.  Sums, zeros and lookups of wide rows are
// bounded by HBM bytes; the launches of the sort, the joining and lookups of few
// tokens or narrow rows by latency (168880 tokens of 99 columns, fp32 to bf16 from
// 16 ranks: 66 us for 45 MB, a wave to a token one step after the other).
#include "dispatch.hpp"
#include "layer_device.hpp"

namespace ar {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

// ---- ranks -------------------------------------------------------------------
// The rank that holds entry v of [0, V), found by halving.  Lanes differ in v only where short rows are zeroed.
template <int NR> __device__ __forceinline__ int rank_of(const EmbedTable<NR> &e, int v) {
    int lo = 0, hi = e.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (e.first[mid] <= v) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}
template <int DT, int NR> __device__ __forceinline__ char *entry_row(const EmbedTable<NR> &e, int v) {
    const int r = rank_of(e, v);
    return e.t[r] + (long long)(v - e.first[r]) * e.pitch[r] * elem_bytes<DT>();
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Columns to a lane: 16 bytes of the type that is written.  (Reading 8 columns of fp32 in two halves costs less than
// writing 8 bytes to a lane: 16384 tokens of 5120 columns, fp32 to bf16, 56 us against 60 with four.)
template <int DT> constexpr int kCols = DT == F32 ? 4 : 8;

// ---- lookup ------------------------------------------------------------------
// A wave writes U runs per lane of one token's row.
constexpr int kLookupCols = 1024;      // of a wave
template <int DT, int OT, bool TINY, int NR>
__global__ __launch_bounds__(kThreads) void embed_kernel(const EmbedTable<NR> e, const int64_t *ids, char *out, long long tokens,
                                                         int width, int slices, int vocab, float scale) {
    constexpr int K = kCols<OT>, U = kLookupCols / 64 / K;
    const int lane = threadIdx.x & 63;
    for (long long item = (long long)blockIdx.x * kWaves + (threadIdx.x >> 6);; item += (long long)gridDim.x * kWaves) {
        const long long token = item / slices;
        if (token >= tokens) return;
        const int run0 = uniform((int)(item - token * slices)) * 64 * U;
        const int64_t id = ids[token];
        const bool known = id >= 0 && id < vocab;
        const char *row = entry_row<DT>(e, uniform(known ? (int)id : 0));
        ColPlace p[U];
        Run<DT, K> o[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            p[u] = col_place<K, TINY>(run0 + u * 64 + lane, width);
            if (known) o[u] = load_at<DT, K, TINY, false>(row, p[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float f[K];
            if (known) {
                widen<DT, K>(o[u], f);
                settle<K, TINY>(f, p[u]);
            }
#pragma unroll
            for (int i = 0; i < K; ++i) f[i] = known ? f[i] * scale : 0.0f;
            store_run<OT, K>(out + (token * width + p[u].col) * elem_bytes<OT>(), narrow<OT, K>(f), p[u].left);
        }
    }
}

// ---- sorting -------------------------------------------------------------------
__device__ __forceinline__ uint32_t key_of(int64_t id, int vocab) {
    return id >= 0 && id < vocab ? (uint32_t)id : (uint32_t)vocab;
}

// Few tokens: a token's place is the number of those before it in the order,
// (key, position) being compared, counted directly.  A workgroup counts for
// eight tokens, its waves dealing out the steps of 64 tokens that these are
// compared with.  The workgroups behind those write which entries have a token,
// kMapEach of them each.
// The whole gradient of 64 columns, 50000 entries, by counting (by passes over
// digits), us: 1024 tokens 16.8 (28.4), 4096 19.9 (30.2), 8192 26.4 (31.5), 12288
// 35.8 (32.1), 16384 47.6 (34.5).
constexpr long long kRankTokens = 10240;
constexpr int kRankEach = 8;
constexpr int kMapEach = 1024;
__global__ __launch_bounds__(kThreads) void embed_rank_kernel(const int64_t *ids, int tokens, int vocab, uint32_t *keys,
                                                              uint32_t *order, uint8_t *map, int ranks) {
    __shared__ uint32_t has[kMapEach / 4];
    __shared__ int parts[kWaves][kRankEach];
    if ((int)blockIdx.x >= ranks) {
        const int v0 = ((int)blockIdx.x - ranks) * kMapEach;
        has[threadIdx.x] = 0;
        __syncthreads();
        constexpr int B = 8;
        for (int i = threadIdx.x; i < tokens; i += B * kThreads) {
            uint32_t k[B];
#pragma unroll
            for (int b = 0; b < B; ++b) {          // past the end: the last token once more
                const int j = i + b * kThreads;
                k[b] = key_of(ids[j < tokens ? j : tokens - 1], vocab) - (uint32_t)v0;
            }
#pragma unroll
            for (int b = 0; b < B; ++b)
                if (k[b] < kMapEach) ((uint8_t *)has)[k[b]] = 1;
        }
        __syncthreads();
        // the map has room for whole workgroups
        ((uint32_t *)(map + v0))[threadIdx.x] = has[threadIdx.x];
        return;
    }
    const int lane = threadIdx.x & 63;
    const int wave = uniform(threadIdx.x >> 6), t0 = blockIdx.x * kRankEach;
    uint32_t mine[kRankEach];
    int before[kRankEach];
#pragma unroll
    for (int k = 0; k < kRankEach; ++k) {
        mine[k] = t0 + k < tokens ? key_of(ids[t0 + k], vocab) : 0u;
        before[k] = 0;
    }
    // Tokens in front of this wave's count where their keys are not above, those behind where they are below.
    const auto count = [&](uint32_t other, uint32_t equal) {
#pragma unroll
        for (int k = 0; k < kRankEach; ++k) before[k] += other < mine[k] + equal ? 1 : 0;
    };
    // Past the end: after everything.  (Read in bounds rather than skipped, so that no load waits for the one before.)
    const auto key_at = [&](int j) {
        const uint32_t key = key_of(ids[j < tokens ? j : tokens - 1], vocab);
        return j < tokens ? key : ~0u;
    };
    constexpr int B = 4, kStep = 64 * kWaves;      // steps whose loads are in flight
    const int own = t0 / 64 * 64;      // the step that holds these tokens
    for (int j0 = wave * 64; j0 < tokens; j0 += kStep * B) {
        uint32_t other[B];
#pragma unroll
        for (int b = 0; b < B; ++b) other[b] = key_at(j0 + b * kStep + lane);
#pragma unroll
        for (int b = 0; b < B; ++b)
            if (j0 + b * kStep != own) count(other[b], j0 + b * kStep < own ? 1 : 0);
    }
    if (wave == 0) {
        const uint32_t other = key_at(own + lane);
#pragma unroll
        for (int k = 0; k < kRankEach; ++k) before[k] += other < mine[k] + (own + lane < t0 + k ? 1 : 0) ? 1 : 0;
    }
#pragma unroll
    for (int k = 0; k < kRankEach; ++k) {
        each_bit([&](auto m) { before[k] += (int)lane_xor<m.value>((uint32_t)before[k], lane); });
        if (lane == 0) parts[wave][k] = before[k];
    }
    __syncthreads();
    const int k = threadIdx.x;
    if (k < kRankEach && t0 + k < tokens) {
        int place = 0;
        for (int w = 0; w < kWaves; ++w) place += parts[w][k];
        keys[place] = key_of(ids[t0 + k], vocab);
        order[place] = (uint32_t)(t0 + k);
    }
}

// Many tokens: stable counting passes over `bits` bits of the key, least
// significant first.  FIRST reads the ids, others keys and positions; it also
// clears (counting) and sets (moving) the map of entries that have a token.
struct CountArgs {
    const int64_t *ids;
    const uint32_t *keys, *order;
    uint32_t *keys_to, *order_to;
    uint32_t *hist;                    // [bins, tiles]
    uint32_t *totals;                  // [bins]
    uint32_t *map;                     // [vocab] bytes, of whole words
    long long tokens, tiles;
    int vocab, shift, bits, tile;
};
template <bool FIRST> __device__ __forceinline__ uint32_t count_key(const CountArgs &a, long long i) {
    return FIRST ? key_of(a.ids[i], a.vocab) : a.keys[i];
}

constexpr int kMostBins = 2048;

template <bool FIRST> __global__ __launch_bounds__(kThreads) void embed_count_kernel(const CountArgs a) {
    __shared__ uint32_t bin[kMostBins];
    const int bins = 1 << a.bits;
    for (int b = threadIdx.x; b < bins; b += kThreads) bin[b] = 0;
    if (FIRST)
        for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < (a.vocab + 3) / 4; i += (long long)gridDim.x * kThreads)
            a.map[i] = 0;
    __syncthreads();
    const long long lo = (long long)blockIdx.x * a.tile, hi = lo + a.tile < a.tokens ? lo + a.tile : a.tokens;
    for (long long i = lo + threadIdx.x; i < hi; i += kThreads) atomicAdd(&bin[(count_key<FIRST>(a, i) >> a.shift) & (bins - 1)], 1u);
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += kThreads) a.hist[b * a.tiles + blockIdx.x] = bin[b];
}

// Inclusive sum over a wave.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t o = __shfl_up(v, d);
        if (lane >= d) v += o;
    }
    return v;
}

// One workgroup to a bin: how many of the bin's tokens stand in earlier tiles, and in all.
__global__ __launch_bounds__(kThreads) void embed_tiles_kernel(uint32_t *hist, uint32_t *totals, long long tiles) {
    __shared__ uint32_t sums[kWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t *h = hist + (long long)blockIdx.x * tiles;
    uint32_t base = 0;
    for (long long t0 = 0; t0 < tiles; t0 += kThreads) {
        const long long t = t0 + threadIdx.x;
        const uint32_t v = t < tiles ? h[t] : 0u, in = wave_scan(v, lane);
        if (lane == 63) sums[wave] = in;
        __syncthreads();
        uint32_t before = base;
        for (int w = 0; w < kWaves; ++w) {
            before += w < wave ? sums[w] : 0u;
            base += sums[w];
        }
        if (t < tiles) h[t] = before + in - v;
        __syncthreads();
    }
    if (threadIdx.x == 0) totals[blockIdx.x] = base;
}

// Moves a tile's tokens to their places, equal digits in the order they stand in:
// every wave owns consecutive tokens and counts its own digits first.  65536 tokens:
// 6 us, as the counting 5 and the sums over tiles 3 to 5: latency, not bytes.
template <bool FIRST> __global__ __launch_bounds__(kThreads) void embed_move_kernel(const CountArgs a) {
    __shared__ uint32_t place[kWaves][kMostBins];      // next place of a digit's token in each wave
    __shared__ uint32_t sums[kWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, bins = 1 << a.bits;
    for (int b = threadIdx.x; b < bins * kWaves; b += kThreads) place[b / bins][b % bins] = 0;
    __syncthreads();
    const int each = a.tile / kWaves;                  // a multiple of 64
    const long long lo = (long long)blockIdx.x * a.tile + (long long)wave * each;
    const long long hi = lo + each < a.tokens ? lo + each : a.tokens;
    for (long long i = lo + lane; i < hi; i += 64) atomicAdd(&place[wave][(count_key<FIRST>(a, i) >> a.shift) & (bins - 1)], 1u);
    __syncthreads();
    // starts: all lower digits' tokens, this digit's in earlier tiles, in earlier waves
    uint32_t base = 0;
    for (int b0 = 0; b0 < bins; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        const uint32_t v = b < bins ? a.totals[b] : 0u, in = wave_scan(v, lane);
        if (lane == 63) sums[wave] = in;
        __syncthreads();
        uint32_t start = base + in - v;
        for (int w = 0; w < kWaves; ++w) {
            start += w < wave ? sums[w] : 0u;
            base += sums[w];
        }
        if (b < bins) {
            start += a.hist[b * a.tiles + blockIdx.x];
            for (int w = 0; w < kWaves; ++w) {
                const uint32_t c = place[w][b];
                place[w][b] = start;
                start += c;
            }
        }
        __syncthreads();
    }
    for (long long i0 = lo; i0 < hi; i0 += 64) {
        const long long i = i0 + lane;
        const bool on = i < hi;
        const uint32_t key = on ? count_key<FIRST>(a, i) : 0u;
        const uint32_t digit = (key >> a.shift) & (bins - 1);
        unsigned long long same = __ballot(on);
        for (int k = 0; k < a.bits; ++k) {
            const unsigned long long set = __ballot((digit >> k) & 1u);
            same &= (digit >> k) & 1u ? set : ~set;
        }
        const int before = __popcll(same & ((1ull << lane) - 1));
        uint32_t to = 0;
        if (on) to = place[wave][digit] + before;
        __builtin_amdgcn_wave_barrier();
        if (on && before == 0) place[wave][digit] += __popcll(same);
        __builtin_amdgcn_wave_barrier();
        if (on) {
            if (FIRST && key < (uint32_t)a.vocab) ((uint8_t *)a.map)[key] = 1;     // every writer writes the same
            a.keys_to[to] = key;
            a.order_to[to] = FIRST ? (uint32_t)i : a.order[i];
        }
    }
}

// ---- sums ----------------------------------------------------------------------
struct SumArgs {
    const uint32_t *keys, *order;
    const char *g;                     // gradient of the looked-up rows
    float *part;                       // [pieces, 2, part_width]: of the run that came in, of the run that goes on
    long long tokens, pieces;
    int piece, width, part_width, vocab;
    int slices;                        // of 64 runs of a row
    int groups;                        // workgroups along a row, a wave to a slice
    long long sums;                    // workgroups that add; those behind them write zeros
    const uint8_t *map;                // which entries have a token; NULL: none has
    int zero_rows, zero_lanes;
    float scale;
    bool accumulate;
};

template <int DT, int K> __device__ __forceinline__ void write_entry(char *row, const ColPlace &p, const float *v, const SumArgs &a) {
    float f[K];
#pragma unroll
    for (int i = 0; i < K; ++i) f[i] = v[i] * a.scale;
    char *to = row + (long long)p.col * elem_bytes<DT>();
    if (a.accumulate) {
        float old[K];
        if (p.left >= K) widen<DT, K>(load_run<DT, K, false>(to), old);
        else widen<DT, K>(load_short<DT, K>(to, p.left), old);
#pragma unroll
        for (int i = 0; i < K; ++i) f[i] += old[i];
    }
    store_run<DT, K>(to, narrow<DT, K>(f), p.left);
}

// A slice's partial sums: four columns of every lane after the other.
template <int K> __device__ __forceinline__ float *part_of(const SumArgs &a, long long piece, int which, int slice, int lane) {
    return a.part + (2 * piece + which) * a.part_width + slice * 64 * K + lane * 4;
}
template <int K> __device__ __forceinline__ void write_part(float *to, const float *v) {
#pragma unroll
    for (int j = 0; j < K / 4; ++j) store_run<F32, 4, false>((char *)(to + j * 256), narrow<F32, 4>(v + 4 * j), 4);
}

// Zeros in the rows of entries without a token, a.zero_rows of them to a
// workgroup, a.zero_lanes lanes (a power of two) to a row.
template <int DT, int NR> __device__ __forceinline__ void zero_rows(const EmbedTable<NR> &e, const SumArgs &a, long long group) {
    const int sets = kThreads / a.zero_lanes, lane = threadIdx.x & (a.zero_lanes - 1);
    const int bytes = a.width * elem_bytes<DT>();
    const long long v0 = group * a.zero_rows, v1 = v0 + a.zero_rows < a.vocab ? v0 + a.zero_rows : a.vocab;
    for (long long v = v0 + threadIdx.x / a.zero_lanes; v < v1; v += sets) {
        if (a.map && a.map[v]) continue;
        char *row = entry_row<DT>(e, a.zero_lanes >= 64 ? uniform((int)v) : (int)v);
        for (int at = lane * 16; at < bytes; at += a.zero_lanes * 16) {
            if (bytes - at >= 16) {
                __builtin_nontemporal_store(u32x4e{0, 0, 0, 0}, (u32x4e *)(row + at));
            } else {
                for (int i = at; i < bytes; i += 2) *(uint16_t *)(row + i) = 0;
            }
        }
    }
}

// 65536 tokens x 4096 bf16 into 131072 entries, zeros included: 300 us, 5.4 TB/s.
template <int DT, int OT, bool TINY, int NR>
__global__ __launch_bounds__(kThreads) void embed_sum_kernel(const EmbedTable<NR> e, const SumArgs a) {
    constexpr int K = kCols<DT>;
    if (blockIdx.x >= a.sums) {
        zero_rows<DT>(e, a, blockIdx.x - a.sums);
        return;
    }
    const int lane = threadIdx.x & 63;
    const long long piece = blockIdx.x / a.groups;
    const int slice = uniform((int)(blockIdx.x - piece * a.groups) * kWaves + (threadIdx.x >> 6));
    if (slice >= a.slices) return;
    const ColPlace p = col_place<K, TINY>(slice * 64 + lane, a.width);
    const long long s0 = piece * a.piece, s1 = s0 + a.piece < a.tokens ? s0 + a.piece : a.tokens;
    const int none = a.vocab;
    const int came = s0 > 0 ? uniform(a.keys[s0 - 1]) : none, goes = s1 < a.tokens ? uniform(a.keys[s1]) : none;
    float sum[K];
#pragma unroll
    for (int i = 0; i < K; ++i) sum[i] = 0.0f;
    bool inside = false;               // the run began in this piece
    int run = came;
    for (long long s = s0; s < s1; s += 64) {
        // 64 tokens' keys and positions, a lane to each; the rows of eight (four of 32 bytes to a lane) are in flight at a time
        const int n = s1 - s < 64 ? (int)(s1 - s) : 64;
        const long long at = s + (lane < n ? lane : n - 1);
        const int keys = (int)a.keys[at], order = (int)a.order[at];
        constexpr int B = Run<OT, K>::W == 8 ? 4 : 8;
        for (int b0 = 0; b0 < n; b0 += B) {
            Run<OT, K> o[B];
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const long long row = (uint32_t)__builtin_amdgcn_readlane(order, b0 + b);
                o[b] = load_at<OT, K, TINY>(a.g + row * a.width * elem_bytes<OT>(), p);
            }
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const int key = b0 + b < n ? __builtin_amdgcn_readlane(keys, b0 + b) : none;
                if (key != run) {
                    if (run != none) {
                        if (inside) write_entry<DT, K>(entry_row<DT>(e, run), p, sum, a);
                        else if (s + b0 + b > s0) write_part<K>(part_of<K>(a, piece, 0, slice, lane), sum);
                    }
                    run = key;
                    inside = true;
#pragma unroll
                    for (int i = 0; i < K; ++i) sum[i] = 0.0f;
                }
                float v[K];
                widen<OT, K>(o[b], v);
                settle<K, TINY>(v, p);
#pragma unroll
                for (int i = 0; i < K; ++i) sum[i] += v[i];
            }
            if (run == none) return;   // no tokens from here on
        }
    }
    if (inside && goes != run) write_entry<DT, K>(entry_row<DT>(e, run), p, sum, a);
    else write_part<K>(part_of<K>(a, piece, inside ? 1 : 0, slice, lane), sum);
}

// The runs that go on past the end of the piece they began in: the waves of a
// workgroup add up every fourth piece of the run, for a slice of the row.
template <int DT, int NR>
__global__ __launch_bounds__(kThreads) void embed_join_kernel(const EmbedTable<NR> e, const SumArgs a) {
    constexpr int K = kCols<DT>;
    __shared__ float lds[kWaves][64 * K];
    const long long piece = blockIdx.x / a.slices;
    const int slice = (int)(blockIdx.x - piece * a.slices);
    const long long s0 = piece * a.piece, s1 = s0 + a.piece;
    if (s1 >= a.tokens) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int before = s0 > 0 ? (int)a.keys[s0 - 1] : a.vocab, last = (int)a.keys[s1 - 1], after = (int)a.keys[s1];
    const int run = uniform(last);
    if (run == a.vocab || uniform(after) != run || uniform(before) == run) return;      // none, ends here, began earlier
    // the last piece that the run reaches: pieces that begin with it, 64 looked at a time
    long long end = piece + 1;
    for (;;) {
        const long long q = end + lane;
        const unsigned long long same = __ballot(q < a.pieces && (int)a.keys[q < a.pieces ? q * a.piece : 0] == run);
        end += same == ~0ull ? 64 : __builtin_ctzll(~same);
        if (same != ~0ull) break;
    }
    float sum[K];
#pragma unroll
    for (int i = 0; i < K; ++i) sum[i] = 0.0f;
    constexpr int B = 4;
    for (long long q = piece + wave; q < end; q += B * kWaves) {
        Run<F32, 4> o[B][K / 4];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const long long at = q + b * kWaves;
            if (at < end)
#pragma unroll
                for (int j = 0; j < K / 4; ++j)
                    o[b][j] = load_run<F32, 4, false>((const char *)(part_of<K>(a, at, at == piece ? 1 : 0, slice, lane) + j * 256));
        }
#pragma unroll
        for (int b = 0; b < B; ++b)
            if (q + b * kWaves < end)
#pragma unroll
                for (int i = 0; i < K; ++i) sum[i] += bits_f32(o[b][i / 4].w[i % 4]);
    }
#pragma unroll
    for (int i = 0; i < K; ++i) lds[wave][i * 64 + lane] = sum[i];
    __syncthreads();
    if (wave != 0) return;
    ColPlace p;
    p.col = p.at = (slice * 64 + lane) * K;
    p.left = a.width - p.col;
#pragma unroll
    for (int w = 1; w < kWaves; ++w)
#pragma unroll
        for (int i = 0; i < K; ++i) sum[i] += lds[w][i * 64 + lane];
    if (p.left > 0) write_entry<DT, K>(entry_row<DT>(e, run), p, sum, a);
}

// ---- host ----------------------------------------------------------------------
template <int NR> EmbedTable<NR> table_of(const EmbedCall &c) {
    EmbedTable<NR> e;
    int first = 0;
    for (int r = 0; r < NR; ++r) {
        e.t[r] = r < c.n ? (char *)c.t[r] : nullptr;
        e.pitch[r] = r < c.n ? (uint32_t)c.pitches[r] : 0;
        e.first[r] = first;
        if (r < c.n) first += (int)c.entries[r];
    }
    e.first[NR] = first;
    e.n = c.n;
    return e;
}

template <typename F> hipError_t by_type(int dtype, F &&f) {
    switch (dtype) {
    case F32: return f(std::integral_constant<int, F32>{});
    case BF16: return f(std::integral_constant<int, BF16>{});
    case F16: return f(std::integral_constant<int, F16>{});
    default: return hipErrorInvalidValue;
    }
}
// f(table's type, rows' type, ranks of the pointer table, whether rows are shorter than eight columns)
template <typename F> hipError_t dispatch_embed(const EmbedCall &c, F &&f) {
    return by_type(c.dtype, [&](auto dt) {
        return by_type(c.out_dtype, [&](auto ot) {
            constexpr std::integral_constant<int, kLayerFew> few{};
            constexpr std::integral_constant<int, kLayerMany> many{};
            if (c.width < 8) return f(dt, ot, many, std::true_type{});
            return c.n <= kLayerFew ? f(dt, ot, few, std::false_type{}) : f(dt, ot, many, std::false_type{});
        });
    });
}

// LDS that a workgroup of the sums reserves at every width, measured at 4096 columns, so that five share a compute unit: 65536 tokens x 4096 bf16 into 131072
// entries 313 us with none, 312, 322, 300, 300, 393 with 16, 24, 32, 40, 60 KB; 1021 tokens into 32000 fp32 101, 102, 97, 95, 93, 91.
constexpr size_t kSumLds = 32 * 1024;
constexpr long long kMostGroups = 1 << 22;             // a grid's threads stay below 2^32
// Slices of 64 runs of a row.
int slices_of(const EmbedCall &c) {
    const int cols = 64 * (c.dtype == F32 ? 4 : 8);
    return (c.width + cols - 1) / cols;
}

}  // namespace

hipError_t launch_embedding(const EmbedCall &c, void *out, hipStream_t s) {
    const int slices = (c.width + kLookupCols - 1) / kLookupCols;
    const long long all = (c.tokens * slices + kWaves - 1) / kWaves, groups = all < kMostGroups ? all : kMostGroups;
    return dispatch_embed(c, [&](auto dt, auto ot, auto nr, auto tiny) {
        return launch(embed_kernel<dt.value, ot.value, tiny.value, nr.value>, dim3((unsigned)groups), dim3(kThreads), 0, s,
                      table_of<nr.value>(c), c.ids, (char *)out, c.tokens, c.width, slices, c.vocab, c.scale);
    });
}

// Places of a partial sum: whole slices, of the longer kind.
static int part_width(int width) { return (width + 511) / 512 * 512; }

EmbedSpace embed_space(long long tokens, int width, int vocab) {
    EmbedSpace w{};
    if (tokens == 0) return w;
    const auto add = [&](size_t bytes) {
        const size_t at = w.bytes;
        w.bytes += (bytes + 255) / 256 * 256;
        return at;
    };
    w.piece = 16;
    while (w.piece < 4096 && w.piece * 1024LL < tokens) w.piece *= 2;
    w.pieces = (tokens + w.piece - 1) / w.piece;
    w.keys = add(tokens * 4);
    w.order = add(tokens * 4);
    w.map = add((size_t)(vocab + kMapEach - 1) / kMapEach * kMapEach);
    if (tokens > kRankTokens) {
        int bits = 1;
        while ((1 << bits) <= vocab) ++bits;            // the key `vocab` among them
        w.passes = bits <= 11 ? 1 : 2;
        w.digit = (bits + w.passes - 1) / w.passes;
        w.tile = 256;
        while (w.tile * 1024LL < tokens) w.tile *= 2;
        w.tiles = (tokens + w.tile - 1) / w.tile;
        w.keys2 = add(tokens * 4);
        w.order2 = add(tokens * 4);
        w.hist = add(((size_t)w.tiles << w.digit) * 4);
        w.totals = add((size_t)4 << w.digit);
    }
    w.part = add((size_t)w.pieces * 2 * part_width(width) * 4);
    return w;
}

hipError_t launch_embed_sort(const EmbedCall &c, const EmbedSpace &w, char *space, hipStream_t s) {
    uint32_t *keys = (uint32_t *)(space + w.keys), *order = (uint32_t *)(space + w.order);
    if (w.passes == 0) {
        const int ranks = (int)((c.tokens + kRankEach - 1) / kRankEach);
        const int maps = c.accumulate ? 0 : (c.vocab + kMapEach - 1) / kMapEach;
        return launch(embed_rank_kernel, dim3((unsigned)(ranks + maps)), dim3(kThreads), 0, s, c.ids, (int)c.tokens, c.vocab, keys, order,
                      (uint8_t *)(space + w.map), ranks);
    }
    uint32_t *keys2 = (uint32_t *)(space + w.keys2), *order2 = (uint32_t *)(space + w.order2);
    hipError_t e = hipSuccess;
    for (int pass = 0; pass < w.passes && e == hipSuccess; ++pass) {
        const bool last = pass == w.passes - 1;
        CountArgs a{c.ids, keys2, order2, last ? keys : keys2, last ? order : order2, (uint32_t *)(space + w.hist),
                    (uint32_t *)(space + w.totals), (uint32_t *)(space + w.map), c.tokens, w.tiles, c.vocab, pass * w.digit, w.digit, w.tile};
        const dim3 grid((unsigned)w.tiles), block(kThreads);
        e = launch(pass ? embed_count_kernel<false> : embed_count_kernel<true>, grid, block, 0, s, a);
        if (e == hipSuccess) e = launch(embed_tiles_kernel, dim3(1u << w.digit), block, 0, s, a.hist, a.totals, w.tiles);
        if (e == hipSuccess) e = launch(pass ? embed_move_kernel<false> : embed_move_kernel<true>, grid, block, 0, s, a);
    }
    return e;
}

hipError_t launch_embed_sum(const EmbedCall &c, const EmbedSpace &w, char *space, const void *grad_out, hipStream_t s) {
    SumArgs a{};
    a.keys = (const uint32_t *)(space + w.keys);
    a.order = (const uint32_t *)(space + w.order);
    a.g = (const char *)grad_out;
    a.part = (float *)(space + w.part);
    a.tokens = c.tokens;
    a.pieces = w.pieces;
    a.piece = w.piece;
    a.width = c.width;
    a.vocab = c.vocab;
    a.part_width = part_width(c.width);
    a.slices = slices_of(c);
    a.groups = (a.slices + kWaves - 1) / kWaves;
    a.sums = w.pieces * a.groups;
    a.scale = c.scale;
    a.accumulate = c.accumulate;
    // About 16 KB to a workgroup, neighbouring rows to neighbouring ones: a fill of 1 GB wrote 6.1 TB/s with 8 KB to a
    // workgroup, 5.5 with 32 KB and 5.2 with 512 KB.
    const int bytes = c.width * (c.dtype == F32 ? 4 : 2);
    a.map = c.tokens ? (const uint8_t *)(space + w.map) : nullptr;
    a.zero_lanes = 8;
    while (a.zero_lanes < kThreads && a.zero_lanes * 16 < bytes) a.zero_lanes *= 2;
    a.zero_rows = kThreads / a.zero_lanes;
    while (a.zero_rows < 1024 && a.zero_rows * bytes < 16384) a.zero_rows *= 2;
    const long long zeros = c.accumulate ? 0 : (c.vocab + a.zero_rows - 1) / a.zero_rows;
    return dispatch_embed(c, [&](auto dt, auto ot, auto nr, auto tiny) {
        const EmbedTable<nr.value> e = table_of<nr.value>(c);
        hipError_t st = hipSuccess;
        if (a.sums + zeros)
            st = launch(embed_sum_kernel<dt.value, ot.value, tiny.value, nr.value>, dim3((unsigned)(a.sums + zeros)),
                        dim3(kThreads), kSumLds, s, e, a);
        if (st == hipSuccess && w.pieces > 1)
            st = launch(embed_join_kernel<dt.value, nr.value>, dim3((unsigned)((w.pieces - 1) * a.slices)), dim3(kThreads), 0, s,
                        e, a);
        return st;
    });
}

}  // namespace ar
