// vocab_api.cpp -- the C ABI of the vocabulary-split reductions: argument
// validation, the split of rows over workgroups, workspace layout, launches.
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "../../include/ar_vocab.h"
#include "ar_host.hpp"
#include "vocab_kernels.hpp"

using namespace ar;

namespace {

static_assert(kTopMax == AR_TOP_MAX && kTeacherMax == AR_TEACHER_MAX && kVocabMany == AR_MAX_RANKS, "limits");

// What every call derives from its shape.
struct Shape {
    VocabCall c{};
    int vocab = 0;
};

ar_status_t check_shape(const ar_vocab_t *v, Shape &s) {
    if (!v || v->n < 1 || v->n > AR_MAX_RANKS || v->rows < 0 || !v->widths) return AR_ERR_INVALID_ARG;
    if (v->dtype < AR_FLOAT32 || v->dtype > AR_INT32) return AR_ERR_INVALID_ARG;
    if (v->dtype == AR_INT32) return AR_ERR_UNSUPPORTED;
    if (!(v->temperature > 0.0f) || !std::isfinite(v->temperature)) return AR_ERR_INVALID_ARG;
    // log2(e) / T and 8 / c have to be normal fp32 numbers
    if (v->temperature < 1e-30f || v->temperature > 1e30f) return AR_ERR_UNSUPPORTED;
    if (v->rows > 0x7fffffffLL) return AR_ERR_UNSUPPORTED;
    const long long *pitches = v->pitches ? v->pitches : v->widths;
    const long long *gpitches = v->grad_pitches ? v->grad_pitches : pitches;
    long long vocab = 0;
    const int tile = 64 * kVocabU * (v->dtype == AR_FLOAT32 ? 4 : 8);
    int tiles = 0;
    for (int r = 0; r < v->n; ++r) {
        const long long w = v->widths[r];
        if (w < 0 || w > AR_VOCAB_MAX) return w < 0 ? AR_ERR_INVALID_ARG : AR_ERR_UNSUPPORTED;
        if (pitches[r] < w || gpitches[r] < w) return AR_ERR_INVALID_ARG;
        if (pitches[r] > 0x7fffffffLL || gpitches[r] > 0x7fffffffLL) return AR_ERR_UNSUPPORTED;
        // byte offsets stay far inside 63 bits
        if (v->rows * std::max(pitches[r], gpitches[r]) > (1LL << 56)) return AR_ERR_UNSUPPORTED;
        s.c.tiny |= w > 0 && w < (v->dtype == AR_FLOAT32 ? 4 : 8);
        vocab += w;
        tiles += (int)((w + tile - 1) / tile);
    }
    if (vocab < 1) return AR_ERR_INVALID_ARG;
    if (vocab > AR_VOCAB_MAX) return AR_ERR_UNSUPPORTED;
    s.vocab = (int)vocab;
    s.c.dtype = v->dtype;
    s.c.rows = v->rows;
    s.c.n = v->n;
    s.c.tiles = tiles;
    s.c.widths = v->widths;
    s.c.pitches = pitches;
    s.c.gpitches = gpitches;
    s.c.temperature = v->temperature;

    // Waves per row, at most one to a tile.  A wave pays about 2 us of set-up
    // and merging per row, so waves are only added while rows * waves leaves
    // compute units short of work; measured on 8192 x 131072 bf16 (us) with 1,
    // 2, 4, 8 waves: 329, 326, 325, 338; on 777 x 50021: 38, 27, 29, 27.
    int waves = 1;
    while (waves < kVocabWaves && waves * 2 <= tiles && v->rows * waves < 16384) waves *= 2;
    // Workgroups per row, while the rows alone leave compute units idle and
    // every wave keeps two tiles; joining them is a second launch (about 4 us),
    // so not below five tiles a wave: 64 x 131072 bf16 with 20 alternatives
    // (us) in 1, 2, 4, 8 workgroups: 19.9, 20.1, 18.5, 21.6; one row of 32768 in 1,
    // 2, 4: 10.5, 13.4, 13.7; a distillation step on 16 x 32768 fp32: 13.2, 19.2, 17.4.
    int parts = 1;
    while (tiles > 4 * waves && parts < kVocabParts && parts * 4 * waves <= tiles && v->rows * parts * 2 <= 256)
        parts *= 2;
    s.c.waves = waves;
    s.c.parts = parts;
    return AR_OK;
}

// The same shape for kernels that come back to a row they have read (its
// gradient in the same call, its top entries): as many waves as there may be,
// so that few rows are in flight and the second look finds them in the caches.
// Measured on 8192 x 131072 bf16 (distillation step, us) with 1, 2, 4, 8
// waves: 1239, 1167, 931, 931; on 512 x 131072 (top 64): 552, 100, 55, 47.
VocabCall short_rows(const Shape &s) {
    VocabCall c = s.c;
    while (c.waves < kVocabWaves && c.waves * 2 <= c.tiles && c.parts == 1) c.waves *= 2;
    return c;
}

// Results and gradient in one launch: the row stays in registers where it
// fits into 16 waves of four tiles (131072 columns of 16-bit logits, half that
// in fp32), elsewhere it is read twice.  A compute unit holds 16 such waves,
// four to each of its SIMDs, so with many rows it depends on the number of
// waves W of a row what that gives.  Time in registers over time reading
// twice, rows of 1/2 GB at 16-byte boundaries / of an odd length in four ranks:
//            bf16                          fp32
//   W        cross     entropy   tail      cross     list      tail
//   2        .84/.70   .93/.84   .88/.71   .86/.73   .86/.71  1.19/.86
//   4        .88/.81   .95/.93   .83/.81   .90/.84   .86/.81  1.12/1.06
//   5        .90/1.09 1.14/1.36 1.27/1.53  .87/.85   .98/1.07 1.49/1.55
//   7        .80/.85   .97/1.06 1.00/1.07  .81/.83   .86/.90  1.22/1.26
//   8        .79/.82   .92/.96   .85/.89   .79/.83   .83/.87  1.11/1.12
//   9        .94/1.09 1.15/1.34 1.31/1.52  .85/.92   .98/1.10 1.33/1.44
//   10       .92/1.00 1.13/1.24 1.30/1.41  .83/.89   .99/1.05 1.33/1.37
//   12       .85/.90  1.03/1.11 1.12/1.21  .82/.87   .91/.97  1.24/1.28
//   13       .85/1.05 1.04/1.28 1.17/1.37  .82/.88   .90/1.03 1.21/1.29
//   16       .83/.91  1.00/1.12 1.03/1.14  .83/.89   .87/.93  1.20/1.23
// (a list without a tail in bf16 about as entropy; fp16 as bf16, but for a
// tail, where its kernel runs out of registers as fp32's does: 1.12-1.86.)
enum class Hold {
    never,
    pairs,                             // where two rows or more fill 7/8 of a compute unit
    even,                              // not where one SIMD has a wave more than all others, nor where six waves idle
    always
};
Hold hold_rule(int dtype, bool weighted, bool list, bool tail) {
    if (tail) return dtype == AR_BFLOAT16 ? Hold::pairs : Hold::never;
    if (dtype == AR_FLOAT32) return list ? Hold::even : Hold::always;
    return list || weighted ? Hold::pairs : Hold::even;
}

// Few rows, a compute unit to each, take as few tiles a wave as they can, to be
// done sooner: 256 x 65280 bf16 (two tiles) cross-entropy 15.3 us (reading twice
// 17.9), with a tail 20.9 (23.1), 200 x 32512 fp32 17.2 (20.9), 16 x 32512 bf16 9.3
// (9.1); with 10 to 14 waves up to 1.2 times slower: 128 x 40704 with a tail 16.3
// (14.1).  Four tiles and a tail, as above: 200 x 52992 fp32 29.5 (24.7).
VocabCall both_rows(const Shape &s, Hold hold) {
    VocabCall c = s.c;
    const bool few = c.rows <= 256;
    c.held = !few || c.tiles > 2 * kHeldWaves ? kHeldTiles : c.tiles > kHeldWaves ? 2 : 1;
    c.waves = (c.tiles + c.held - 1) / c.held;
    const int w = c.waves;
    const bool pays = few ? c.held < kHeldTiles || hold != Hold::never
                          : hold == Hold::always || (hold == Hold::even && (w == 1 || (w % 4 != 1 && w != 10))) ||
                                (hold == Hold::pairs && (w <= 4 || w == 7 || w == 8));
    return pays && w <= kHeldWaves ? c : short_rows(s);
}

// Whether a forward call that saves statistics for a backward one should leave
// the logits in the 256 MB Infinity Cache: where they fit.  Both calls together
// with (without), us, after the logits were written: 2000 x 32000 fp32 135 (152),
// with 20 alternatives 157 (173); bf16 4000 x 32000 144 (163), 500 x 131072 73
// (78), with 5 alternatives 84 (90), 64 x 131072 20 (24).  Where the cache is
// full of other data that has yet to be written back, they lose it: 4000 x 32000 177
// (165).  Past 256 MB non-temporal loads read 7.0 TB/s, plain ones 6.0-6.5.
bool read_again(const Shape &s, const float *saved) {
    const double bytes = (double)s.c.rows * s.vocab * (s.c.dtype == AR_FLOAT32 ? 4 : 2);
    return saved && bytes <= 256.0 * (1 << 20);
}

// Workspace: partial statistics, partial lists, statistics for a gradient
// that follows in a second launch.  Nothing where a row is one workgroup's.
struct Space {
    size_t part = 0, top = 0, saved = 0, bytes = 0;
};
Space space_of(const Shape &s, int top_k) {
    Space w;
    if (s.c.parts == 1) return w;
    const size_t slots = (size_t)s.c.rows * s.c.parts;
    w.top = slots * sizeof(float4);
    w.saved = w.top + (slots * top_k * sizeof(unsigned long long) + 15) / 16 * 16;
    w.bytes = w.saved + (size_t)s.c.rows * 4 * sizeof(float);
    return w;
}

ar_status_t check_space(const Space &w, const void *workspace, size_t bytes) {
    if (w.bytes == 0) return AR_OK;
    if (!workspace || bytes < w.bytes) return AR_ERR_INVALID_ARG;
    return (uintptr_t)workspace % 16 ? AR_ERR_ALIGNMENT : AR_OK;
}

// The row's tiles lie on 16-byte boundaries of memory, so rows off them may
// reach into one tile more.
void set_logits(Shape &s, const void *const *x) {
    const int e = s.c.dtype == AR_FLOAT32 ? 4 : 2, lanes = 16 / e, tile = 64 * kVocabU * lanes;
    s.c.x = x;
    for (int r = 0; r < s.c.n; ++r)
        if (s.c.widths[r] && ((uintptr_t)x[r] % 16 || (s.c.rows > 1 && s.c.pitches[r] * e % 16))) s.c.skew = lanes - 1;
    s.c.tiles = 0;
    for (int r = 0; r < s.c.n; ++r)
        if (s.c.widths[r]) s.c.tiles += (int)((s.c.widths[r] + s.c.skew + tile - 1) / tile);
}

// One rank's buffer: present where it has columns, aligned to its elements.
ar_status_t check_buffers(const Shape &s, const void *const *bufs) {
    if (!bufs) return AR_ERR_INVALID_ARG;
    const uintptr_t e = s.c.dtype == AR_FLOAT32 ? 4 : 2;
    for (int r = 0; r < s.c.n; ++r) {
        if (s.c.widths[r] == 0) continue;
        if (!bufs[r]) return AR_ERR_INVALID_ARG;
        if ((uintptr_t)bufs[r] % e) return AR_ERR_ALIGNMENT;
    }
    return AR_OK;
}

struct Range {
    uintptr_t lo, hi;                  // first byte of the first row, past the last byte of the last
    uintptr_t row, pitch;              // bytes of a row, between rows
    bool grad;
};

// Rows at one pitch that never meet: columns of one wider buffer.
bool interleaved(const Range &a, const Range &b) {
    if (a.pitch != b.pitch || a.pitch == 0) return false;
    const uintptr_t d = (b.lo > a.lo ? b.lo - a.lo : a.pitch - (a.lo - b.lo) % a.pitch) % a.pitch;
    return d >= a.row && d + b.row <= a.pitch;
}

// Every gradient buffer is apart from every other buffer, or is its own
// rank's logits, element for element.
ar_status_t check_grads(const Shape &s, const void *const *x, void *const *g) {
    const long long e = s.c.dtype == AR_FLOAT32 ? 4 : 2;
    Range rs[2 * AR_MAX_RANKS];
    int k = 0;
    for (int r = 0; r < s.c.n; ++r) {
        const long long w = s.c.widths[r];
        if (w == 0) continue;
        const auto add = [&](const void *p, long long pitch, bool grad) {
            const uintptr_t lo = (uintptr_t)p;
            rs[k++] = {lo, lo + (uintptr_t)(((s.c.rows - 1) * pitch + w) * e), (uintptr_t)(w * e),
                       (uintptr_t)(pitch * e), grad};
        };
        const bool same = x[r] == g[r] && (s.c.pitches[r] == s.c.gpitches[r] || s.c.rows == 1);
        if (!same) add(x[r], s.c.pitches[r], false);
        add(g[r], s.c.gpitches[r], true);
    }
    std::sort(rs, rs + k, [](const Range &a, const Range &b) { return a.lo < b.lo; });
    uintptr_t end_any = 0, end_grad = 0;
    bool apart = true;
    for (int i = 0; i < k; ++i) {
        if (rs[i].lo < (rs[i].grad ? end_any : end_grad)) apart = false;
        end_any = std::max(end_any, rs[i].hi);
        if (rs[i].grad) end_grad = std::max(end_grad, rs[i].hi);
    }
    for (int i = 0; i < k && !apart; ++i)
        for (int j = i + 1; j < k && rs[j].lo < rs[i].hi; ++j)
            if ((rs[i].grad || rs[j].grad) && !interleaved(rs[i], rs[j])) return AR_ERR_INVALID_ARG;
    return AR_OK;
}

bool misaligned(const void *p, uintptr_t a) { return (uintptr_t)p % a != 0; }

ar_status_t hip_status(hipError_t e) { return e == hipSuccess ? AR_OK : AR_ERR_HIP; }

ar_status_t check_teacher(const int64_t *ids, const float *values, int k, ar_teacher_t mode) {
    if (!ids || !values || k < 1) return AR_ERR_INVALID_ARG;
    if (mode != AR_TEACHER_RENORM && mode != AR_TEACHER_TAIL) return AR_ERR_INVALID_ARG;
    if (k > AR_TEACHER_MAX) return AR_ERR_UNSUPPORTED;
    return misaligned(ids, 8) || misaligned(values, 4) ? AR_ERR_ALIGNMENT : AR_OK;
}

}  // namespace

extern "C" {

ar_status_t ar_vocab_workspace(const ar_vocab_t *shape, int top_k, size_t *bytes) {
    if (!bytes || top_k < 0) return AR_ERR_INVALID_ARG;
    if (top_k > AR_TOP_MAX) return AR_ERR_UNSUPPORTED;
    Shape s;
    const ar_status_t st = check_shape(shape, s);
    if (st != AR_OK) return st;
    *bytes = space_of(s, top_k).bytes;
    return AR_OK;
}

ar_status_t ar_logprobs(const void *const *logits, const ar_vocab_t *shape, const int64_t *targets, float *logprobs,
                        float *entropy, int top_k, float *top_logprobs, int64_t *top_ids, float *saved,
                        void *workspace, size_t workspace_bytes, hipStream_t stream) {
    Shape s;
    ar_status_t st = check_shape(shape, s);
    if (st != AR_OK) return st;
    if (top_k < 0 || (top_k > 0) != (top_logprobs != nullptr) || (top_k > 0) != (top_ids != nullptr))
        return AR_ERR_INVALID_ARG;
    if (top_k > AR_TOP_MAX) return AR_ERR_UNSUPPORTED;
    if (s.c.rows == 0) return AR_OK;
    if (!targets || !logprobs) return AR_ERR_INVALID_ARG;
    if ((st = check_buffers(s, logits)) != AR_OK) return st;
    if (misaligned(targets, 8) || misaligned(top_ids, 8) || misaligned(logprobs, 4) || misaligned(entropy, 4) ||
        misaligned(top_logprobs, 4) || misaligned(saved, 4))
        return AR_ERR_ALIGNMENT;
    const Space w = space_of(s, top_k);
    if ((st = check_space(w, workspace, workspace_bytes)) != AR_OK) return st;
    set_logits(s, logits);
    s.c.again = read_again(s, saved);
    LogprobsArgs a{};
    a.targets = targets;
    a.logprobs = logprobs;
    a.entropy = entropy;
    a.saved = saved;
    a.k = top_k;
    a.top_logprobs = top_logprobs;
    a.top_ids = top_ids;
    if (s.c.parts > 1) {
        a.part = (float4 *)((char *)workspace + w.part);
        a.part_top = (unsigned long long *)((char *)workspace + w.top);
    }
    hipError_t e = launch_logprobs(top_k ? short_rows(s) : s.c, a, kForward, stream);
    if (e == hipSuccess && s.c.parts > 1) e = launch_logprobs(s.c, a, kJoin, stream);
    return hip_status(e);
}

ar_status_t ar_logprobs_backward(const void *const *logits, void *const *grads, const ar_vocab_t *shape,
                                 const int64_t *targets, const float *saved, const float *grad_logprobs,
                                 const float *grad_entropy, hipStream_t stream) {
    Shape s;
    ar_status_t st = check_shape(shape, s);
    if (st != AR_OK) return st;
    if (s.c.rows == 0) return AR_OK;
    if (!targets || !saved) return AR_ERR_INVALID_ARG;
    if ((st = check_buffers(s, logits)) != AR_OK || (st = check_buffers(s, (const void *const *)grads)) != AR_OK)
        return st;
    if (misaligned(targets, 8) || misaligned(saved, 4) || misaligned(grad_logprobs, 4) || misaligned(grad_entropy, 4))
        return AR_ERR_ALIGNMENT;
    if ((st = check_grads(s, logits, grads)) != AR_OK) return st;
    set_logits(s, logits);
    s.c.g = grads;
    LogprobsArgs a{};
    a.targets = targets;
    a.saved = const_cast<float *>(saved);
    a.grad_logprobs = grad_logprobs;
    a.grad_entropy = grad_entropy;
    return hip_status(launch_logprobs(s.c, a, kBackward, stream));
}

ar_status_t ar_logprobs_grad(const void *const *logits, void *const *grads, const ar_vocab_t *shape,
                             const int64_t *targets, const float *grad_logprobs, const float *grad_entropy,
                             float *logprobs, float *entropy, float *saved, void *workspace, size_t workspace_bytes,
                             hipStream_t stream) {
    Shape s;
    ar_status_t st = check_shape(shape, s);
    if (st != AR_OK) return st;
    if (s.c.rows == 0) return AR_OK;
    if (!targets) return AR_ERR_INVALID_ARG;
    if ((st = check_buffers(s, logits)) != AR_OK || (st = check_buffers(s, (const void *const *)grads)) != AR_OK)
        return st;
    if (misaligned(targets, 8) || misaligned(saved, 4) || misaligned(grad_logprobs, 4) || misaligned(grad_entropy, 4) ||
        misaligned(logprobs, 4) || misaligned(entropy, 4))
        return AR_ERR_ALIGNMENT;
    if ((st = check_grads(s, logits, grads)) != AR_OK) return st;
    const Space w = space_of(s, 0);
    if ((st = check_space(w, workspace, workspace_bytes)) != AR_OK) return st;
    set_logits(s, logits);
    s.c.g = grads;
    LogprobsArgs a{};
    a.targets = targets;
    a.logprobs = logprobs;
    a.entropy = entropy;
    a.saved = saved;
    a.grad_logprobs = grad_logprobs;
    a.grad_entropy = grad_entropy;
    if (s.c.parts == 1) {
        const Hold hold = hold_rule(s.c.dtype, entropy || saved || grad_entropy, false, false);
        return hip_status(launch_logprobs(both_rows(s, hold), a, kBoth, stream));
    }
    a.part = (float4 *)((char *)workspace + w.part);
    if (!a.saved) a.saved = (float *)((char *)workspace + w.saved);
    s.c.again = read_again(s, a.saved);
    hipError_t e = launch_logprobs(s.c, a, kForward, stream);
    if (e == hipSuccess) e = launch_logprobs(s.c, a, kJoin, stream);
    if (e == hipSuccess) e = launch_logprobs(s.c, a, kBackward, stream);
    return hip_status(e);
}

ar_status_t ar_distill(const void *const *logits, const ar_vocab_t *shape, const int64_t *teacher_ids,
                       const float *teacher_values, int k, ar_teacher_t mode, float *loss, float *saved,
                       void *workspace, size_t workspace_bytes, hipStream_t stream) {
    Shape s;
    ar_status_t st = check_shape(shape, s);
    if (st != AR_OK) return st;
    if (s.c.rows == 0) return AR_OK;
    if ((st = check_teacher(teacher_ids, teacher_values, k, mode)) != AR_OK) return st;
    if (!loss) return AR_ERR_INVALID_ARG;
    if ((st = check_buffers(s, logits)) != AR_OK) return st;
    if (misaligned(loss, 4) || misaligned(saved, 4)) return AR_ERR_ALIGNMENT;
    const Space w = space_of(s, 0);
    if ((st = check_space(w, workspace, workspace_bytes)) != AR_OK) return st;
    set_logits(s, logits);
    DistillArgs a{};
    a.ids = teacher_ids;
    a.values = teacher_values;
    a.k = k;
    a.loss = loss;
    a.saved = saved;
    s.c.again = read_again(s, saved);
    const bool tail = mode == AR_TEACHER_TAIL;
    if (s.c.parts > 1) a.part = (float4 *)((char *)workspace + w.part);
    hipError_t e = launch_distill(s.c, a, tail, kForward, stream);
    if (e == hipSuccess && s.c.parts > 1) e = launch_distill(s.c, a, tail, kJoin, stream);
    return hip_status(e);
}

ar_status_t ar_distill_backward(const void *const *logits, void *const *grads, const ar_vocab_t *shape,
                                const int64_t *teacher_ids, const float *teacher_values, int k, ar_teacher_t mode,
                                const float *saved, const float *grad_loss, hipStream_t stream) {
    Shape s;
    ar_status_t st = check_shape(shape, s);
    if (st != AR_OK) return st;
    if (s.c.rows == 0) return AR_OK;
    if ((st = check_teacher(teacher_ids, teacher_values, k, mode)) != AR_OK) return st;
    if (!saved) return AR_ERR_INVALID_ARG;
    if ((st = check_buffers(s, logits)) != AR_OK || (st = check_buffers(s, (const void *const *)grads)) != AR_OK)
        return st;
    if (misaligned(saved, 4) || misaligned(grad_loss, 4)) return AR_ERR_ALIGNMENT;
    if ((st = check_grads(s, logits, grads)) != AR_OK) return st;
    set_logits(s, logits);
    s.c.g = grads;
    DistillArgs a{};
    a.ids = teacher_ids;
    a.values = teacher_values;
    a.k = k;
    a.saved = const_cast<float *>(saved);
    a.grad_loss = grad_loss;
    return hip_status(launch_distill(s.c, a, mode == AR_TEACHER_TAIL, kBackward, stream));
}

ar_status_t ar_distill_grad(const void *const *logits, void *const *grads, const ar_vocab_t *shape,
                            const int64_t *teacher_ids, const float *teacher_values, int k, ar_teacher_t mode,
                            const float *grad_loss, float *loss, float *saved, void *workspace,
                            size_t workspace_bytes, hipStream_t stream) {
    Shape s;
    ar_status_t st = check_shape(shape, s);
    if (st != AR_OK) return st;
    if (s.c.rows == 0) return AR_OK;
    if ((st = check_teacher(teacher_ids, teacher_values, k, mode)) != AR_OK) return st;
    if ((st = check_buffers(s, logits)) != AR_OK || (st = check_buffers(s, (const void *const *)grads)) != AR_OK)
        return st;
    if (misaligned(loss, 4) || misaligned(saved, 4) || misaligned(grad_loss, 4)) return AR_ERR_ALIGNMENT;
    if ((st = check_grads(s, logits, grads)) != AR_OK) return st;
    const Space w = space_of(s, 0);
    if ((st = check_space(w, workspace, workspace_bytes)) != AR_OK) return st;
    set_logits(s, logits);
    s.c.g = grads;
    DistillArgs a{};
    a.ids = teacher_ids;
    a.values = teacher_values;
    a.k = k;
    a.loss = loss;
    a.saved = saved;
    a.grad_loss = grad_loss;
    const bool tail = mode == AR_TEACHER_TAIL;
    if (s.c.parts == 1)
        return hip_status(launch_distill(both_rows(s, hold_rule(s.c.dtype, false, true, tail)), a, tail, kBoth, stream));
    a.part = (float4 *)((char *)workspace + w.part);
    if (!a.saved) a.saved = (float *)((char *)workspace + w.saved);
    s.c.again = read_again(s, a.saved);
    hipError_t e = launch_distill(s.c, a, tail, kForward, stream);
    if (e == hipSuccess) e = launch_distill(s.c, a, tail, kJoin, stream);
    if (e == hipSuccess) e = launch_distill(s.c, a, tail, kBackward, stream);
    return hip_status(e);
}

}  // extern "C"
