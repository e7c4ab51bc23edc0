// layer_api.cpp -- the C ABI of the operators around a step's collectives:
// argument validation, workspace layout, launches.
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <memory>
#include <new>

#include "../../include/ar_layer.h"
#include "ar_host.hpp"
#include "layer_kernels.hpp"

using namespace ar;

namespace {

static_assert(kLayerMany == AR_MAX_RANKS, "limits");

bool misaligned(const void *p, uintptr_t a) { return (uintptr_t)p % a != 0; }
ar_status_t hip_status(hipError_t e) { return e == hipSuccess ? AR_OK : AR_ERR_HIP; }

long long bytes_of(int dtype) { return dtype == AR_FLOAT32 ? 4 : 2; }

ar_status_t check_type(int dtype) {
    if (dtype < AR_FLOAT32 || dtype > AR_INT32) return AR_ERR_INVALID_ARG;
    return dtype == AR_INT32 ? AR_ERR_UNSUPPORTED : AR_OK;
}

ar_status_t check_pitches(const long long *pitches, int n, long long width) {
    for (int r = 0; pitches && r < n; ++r) {
        if (pitches[r] < width) return AR_ERR_INVALID_ARG;
        if (pitches[r] > 0x7fffffffLL) return AR_ERR_UNSUPPORTED;
    }
    return AR_OK;
}

ar_status_t check_space(size_t need, const void *workspace, size_t bytes) {
    if (need == 0) return AR_OK;
    if (!workspace || bytes < need) return AR_ERR_INVALID_ARG;
    return misaligned(workspace, 16) ? AR_ERR_ALIGNMENT : AR_OK;
}

// Memory that a call touches: rows of `row` bytes, `pitch` bytes apart.
struct Span {
    uintptr_t lo, hi, row, pitch;
    bool written;
};
Span span_of(const void *p, long long rows, long long row, long long pitch, bool written) {
    const uintptr_t lo = (uintptr_t)p;
    return {lo, lo + (uintptr_t)((rows - 1) * pitch + row), (uintptr_t)row, (uintptr_t)pitch, written};
}
Span flat_span(const void *p, long long bytes, bool written) { return span_of(p, 1, bytes, bytes, written); }

// Rows at one pitch that never meet: columns of one wider buffer.
bool interleaved(const Span &a, const Span &b) {
    if (a.pitch != b.pitch || a.pitch == 0) return false;
    const uintptr_t d = (b.lo > a.lo ? b.lo - a.lo : a.pitch - (a.lo - b.lo) % a.pitch) % a.pitch;
    return d >= a.row && d + b.row <= a.pitch;
}

// Whether everything that is written is apart from everything else.
bool apart(Span *s, long long k) {
    const auto below = [](const Span &a, const Span &b) { return a.lo < b.lo; };
    if (!std::is_sorted(s, s + k, below)) std::sort(s, s + k, below);
    uintptr_t end_any = 0, end_written = 0;
    bool fine = true;
    for (long long i = 0; i < k; ++i) {
        if (s[i].lo < (s[i].written ? end_any : end_written)) fine = false;
        end_any = std::max(end_any, s[i].hi);
        if (s[i].written) end_written = std::max(end_written, s[i].hi);
    }
    for (long long i = 0; i < k && !fine; ++i)
        for (long long j = i + 1; j < k && s[j].lo < s[i].hi; ++j)
            if ((s[i].written || s[j].written) && !interleaved(s[i], s[j])) return false;
    return true;
}

// ---- reduction, residual, norm ---------------------------------------------
ar_status_t check_norm(const ar_norm_t *v, NormRow &r) {
    if (!v || v->n < 1 || v->n > AR_MAX_RANKS || v->rows < 0 || v->width < 1) return AR_ERR_INVALID_ARG;
    ar_status_t st = check_type(v->dtype);
    if (st == AR_OK) st = check_type(v->weight_dtype);
    if (st != AR_OK) return st;
    if (v->weight_dtype != v->dtype && v->weight_dtype != AR_FLOAT32) return AR_ERR_UNSUPPORTED;
    if (v->rows > 0x7fffffffLL || v->width > AR_NORM_WIDTH_MAX) return AR_ERR_UNSUPPORTED;
    if (!(v->eps >= 0.0f) || !std::isfinite(v->eps) || !std::isfinite(v->offset)) return AR_ERR_INVALID_ARG;
    if (v->group < 0) return AR_ERR_INVALID_ARG;
    if (v->group && (v->group < 32 || v->group > 512 || (v->group & (v->group - 1)))) return AR_ERR_UNSUPPORTED;
    if ((st = check_pitches(v->pitches, v->n, v->width)) != AR_OK) return st;
    r = NormRow{};
    r.weight32 = v->weight_dtype == AR_FLOAT32;
    r.width = (int)v->width;
    r.eps = v->eps;
    r.offset = v->offset;
    r.rows = v->rows;
    return AR_OK;
}

size_t norm_space(const NormBackPlan &p) { return (size_t)p.groups * p.width * sizeof(float); }

// ---- embedding ---------------------------------------------------------------
ar_status_t check_embed(const ar_embed_t *v, EmbedCall &c) {
    if (!v || v->n < 1 || v->n > AR_MAX_RANKS || v->tokens < 0 || v->width < 1 || !v->entries) return AR_ERR_INVALID_ARG;
    ar_status_t st = check_type(v->dtype);
    if (st == AR_OK) st = check_type(v->out_dtype);
    if (st != AR_OK) return st;
    if (!std::isfinite(v->scale)) return AR_ERR_INVALID_ARG;
    if (v->tokens > AR_EMBED_TOKENS_MAX || v->width > AR_EMBED_WIDTH_MAX) return AR_ERR_UNSUPPORTED;
    if ((st = check_pitches(v->pitches, v->n, v->width)) != AR_OK ||
        (st = check_pitches(v->grad_pitches, v->n, v->width)) != AR_OK)
        return st;
    long long vocab = 0;
    for (int r = 0; r < v->n; ++r) {
        if (v->entries[r] < 0) return AR_ERR_INVALID_ARG;
        if (v->entries[r] > AR_EMBED_ENTRIES_MAX) return AR_ERR_UNSUPPORTED;
        vocab += v->entries[r];
    }
    if (vocab < 1) return AR_ERR_INVALID_ARG;
    if (vocab > AR_EMBED_ENTRIES_MAX) return AR_ERR_UNSUPPORTED;
    c = EmbedCall{};
    c.dtype = v->dtype;
    c.out_dtype = v->out_dtype;
    c.n = v->n;
    c.entries = v->entries;
    c.tokens = v->tokens;
    c.width = (int)v->width;
    c.vocab = (int)vocab;
    c.scale = v->scale;
    return AR_OK;
}

// The ranks' buffers: present where a rank has entries, aligned to their elements; adds their spans.
ar_status_t check_tables(const EmbedCall &c, const void *const *t, bool written, Span *s, int &k) {
    if (!t) return AR_ERR_INVALID_ARG;
    const long long e = bytes_of(c.dtype);
    for (int r = 0; r < c.n; ++r) {
        if (c.entries[r] == 0) continue;
        if (!t[r]) return AR_ERR_INVALID_ARG;
        if (misaligned(t[r], e)) return AR_ERR_ALIGNMENT;
        s[k++] = span_of(t[r], c.entries[r], c.width * e, c.pitches[r] * e, written);
    }
    return AR_OK;
}

struct Widths {                        // pitches that are all the width
    long long w[AR_MAX_RANKS];
    const long long *use(const long long *given, int n, long long width) {
        if (given) return given;
        std::fill(w, w + n, width);
        return w;
    }
};

// ---- gradient norm -----------------------------------------------------------
ar_status_t check_grads(const ar_grads_t *g) {
    if (!g || g->count < 0 || (g->count && (!g->bufs || !g->sizes || !g->dtypes))) return AR_ERR_INVALID_ARG;
    if (g->count > AR_GRADS_MAX) return AR_ERR_UNSUPPORTED;
    long long all = 0;
    for (long long i = 0; i < g->count; ++i) {
        if (g->sizes[i] < 0) return AR_ERR_INVALID_ARG;
        const ar_status_t st = check_type(g->dtypes[i]);
        if (st != AR_OK) return st;
        if (g->sizes[i] > (1LL << 40) || (all += g->sizes[i]) > (1LL << 40)) return AR_ERR_UNSUPPORTED;
    }
    return AR_OK;
}

ar_status_t check_grad_buffers(const ar_grads_t *g, const void *const *bufs) {
    if (g->count && !bufs) return AR_ERR_INVALID_ARG;
    for (long long i = 0; i < g->count; ++i) {
        if (!g->sizes[i]) continue;
        if (!bufs[i]) return AR_ERR_INVALID_ARG;
        if (misaligned(bufs[i], bytes_of(g->dtypes[i]))) return AR_ERR_ALIGNMENT;
    }
    return AR_OK;
}

// Elements of a chunk, and whether the list stays in the 256 MB Infinity Cache.
void grad_rule(const ar_grads_t *g, GradTable &t) {
    long long all = 0, bytes = 0;
    for (long long i = 0; i < g->count; ++i) all += g->sizes[i], bytes += g->sizes[i] * bytes_of(g->dtypes[i]);
    t.chunk = kGradChunk;
    while (t.chunk < kGradLongChunk && all > (long long)kGradGroups * t.chunk) t.chunk *= 2;
    t.again = bytes <= 256LL << 20;
}

// Partial sums of a list at most: buffers that adjoin are taken as one, so there may be fewer.
size_t grad_parts(const ar_grads_t *g) {
    GradTable t;
    grad_rule(g, t);
    long long entries = 0, chunks = 0;
    for (long long i = 0; i < g->count; ++i) {
        entries += (g->sizes[i] + kGradPieceMax - 1) / kGradPieceMax;
        chunks += (g->sizes[i] + t.chunk - 1) / t.chunk;
    }
    const long long launches = (entries + kGradTable - 1) / kGradTable;
    return (size_t)std::min(chunks, launches * kGradGroups);
}
// Workspace: the norm, the partial sums.
size_t grad_space(const ar_grads_t *g) {
    const size_t parts = grad_parts(g);
    return parts ? (1 + parts) * sizeof(double) : 0;
}

// f(piece) for the list's buffers in turn, those that adjoin (in the outputs too) as one.
template <typename F> hipError_t each_piece(const ar_grads_t *g, void *const *outs, F &&f) {
    GradPiece p{};
    for (long long i = 0; i < g->count; ++i) {
        if (!g->sizes[i]) continue;
        const char *in = (const char *)g->bufs[i];
        char *out = outs ? (char *)outs[i] : nullptr;
        const long long bytes = p.size * bytes_of(p.dtype);
        if (p.size && p.dtype == g->dtypes[i] && p.in + bytes == in && (!outs || p.out + bytes == out)) {
            p.size += g->sizes[i];
            continue;
        }
        if (p.size) {
            const hipError_t e = f(p);
            if (e != hipSuccess) return e;
        }
        p = {in, out, g->sizes[i], g->dtypes[i]};
    }
    return p.size ? f(p) : hipSuccess;
}

// Chunks after which a table is launched: those of one more piece keep a grid's threads below 2^32.
constexpr uint32_t kGradMostChunks = 1u << 22;

// f(table, chunks) for full tables of the list's pieces, chunks of t.chunk elements or (0) of kGradScaleBytes.
template <typename F> hipError_t each_table(const ar_grads_t *g, void *const *outs, GradTable &t, F &&f) {
    t.n = 0;
    t.first[0] = 0;
    const auto flush = [&]() {
        if (!t.n) return hipSuccess;
        const uint32_t chunks = t.first[t.n];
        for (int i = t.n; i < kGradTable; ++i) t.in[i] = nullptr, t.out[i] = nullptr, t.size[i] = 0, t.dtype[i] = 0, t.first[i + 1] = chunks;
        const hipError_t e = f(t, chunks);
        t.n = 0;
        return e;
    };
    const hipError_t e = each_piece(g, outs, [&](GradPiece p) {
        while (p.size) {
            const long long size = std::min(p.size, kGradPieceMax), bytes = size * bytes_of(p.dtype);
            const int i = t.n++;
            t.in[i] = p.in;
            t.out[i] = p.out;
            t.size[i] = (uint32_t)size;
            t.dtype[i] = (uint8_t)p.dtype;
            const long long chunk = t.chunk ? t.chunk : kGradScaleBytes / bytes_of(p.dtype);
            t.first[i + 1] = t.first[i] + (uint32_t)((size + chunk - 1) / chunk);
            p.in += bytes;
            if (p.out) p.out += bytes;
            p.size -= size;
            if (t.n == kGradTable || (!t.chunk && t.first[t.n] > kGradMostChunks)) {
                const hipError_t e = flush();
                if (e != hipSuccess) return e;
            }
        }
        return hipSuccess;
    });
    return e == hipSuccess ? flush() : e;
}

int grad_groups(uint32_t chunks) { return (int)std::min<uint32_t>(chunks, kGradGroups); }

// The launches that leave the list's partial sums in the workspace; how many there are goes into t.parts.
hipError_t sum_squares(const ar_grads_t *g, void *const *outs, GradTable &t, double *part, hipStream_t stream) {
    int parts = 0;
    grad_rule(g, t);
    const hipError_t e = each_table(g, outs, t, [&](GradTable &t, uint32_t chunks) {
        t.part = part + parts;
        parts += grad_groups(chunks);
        return launch_grad_sum(t, grad_groups(chunks), stream);
    });
    t.part = part;
    t.parts = parts;
    return e;
}

}  // namespace

extern "C" {

ar_status_t ar_reduce_norm(const void *const *partials, const ar_norm_t *shape, const void *weight,
                           const void *residual, void *summed, void *out, float *rstd, void *out8, float *scales,
                           hipStream_t stream) {
    NormCall c{};
    ar_status_t st = check_norm(shape, c.a.r);
    if (st != AR_OK) return st;
    if ((out8 != nullptr) != (scales != nullptr) || (!summed && !out && !rstd && !out8)) return AR_ERR_INVALID_ARG;
    if (shape->rows == 0) return AR_OK;
    if (!partials || !weight) return AR_ERR_INVALID_ARG;
    Widths widths;
    c.pitches = widths.use(shape->pitches, shape->n, shape->width);
    const long long e = bytes_of(shape->dtype), rows = shape->rows, row = shape->width * e;
    for (int r = 0; r < shape->n; ++r) {
        if (!partials[r]) return AR_ERR_INVALID_ARG;
        if (misaligned(partials[r], e)) return AR_ERR_ALIGNMENT;
    }
    if (misaligned(weight, bytes_of(shape->weight_dtype)) || misaligned(residual, e) || misaligned(summed, e) ||
        misaligned(out, e) || misaligned(rstd, 4) || misaligned(scales, 4))
        return AR_ERR_ALIGNMENT;
    c.a.group = shape->group / (shape->dtype == AR_FLOAT32 ? 4 : 8);
    c.a.groups = shape->group ? (int)((shape->width + shape->group - 1) / shape->group) : 1;

    Span s[AR_MAX_RANKS + 8];
    int k = 0;
    const auto in = [&](const void *p, long long pitch) {
        const bool same = (p == summed || p == out) && (pitch == row || rows == 1);
        if (!same) s[k++] = span_of(p, rows, row, pitch, false);
    };
    for (int r = 0; r < shape->n; ++r) in(partials[r], c.pitches[r] * e);
    if (residual) in(residual, row);
    s[k++] = flat_span(weight, shape->width * bytes_of(shape->weight_dtype), false);
    if (summed) s[k++] = flat_span(summed, rows * row, true);
    if (out) s[k++] = flat_span(out, rows * row, true);
    if (rstd) s[k++] = flat_span(rstd, rows * 4, true);
    if (out8) s[k++] = flat_span(out8, rows * shape->width, true);
    if (scales) s[k++] = flat_span(scales, rows * c.a.groups * 4, true);
    if (!apart(s, k)) return AR_ERR_INVALID_ARG;

    c.dtype = shape->dtype;
    c.n = shape->n;
    c.x = partials;
    c.a.r.weight = weight;
    c.a.residual = (const char *)residual;
    c.a.summed = (char *)summed;
    c.a.out = (char *)out;
    c.a.rstd = rstd;
    c.a.out8 = (uint8_t *)out8;
    c.a.scales = scales;
    return hip_status(launch_reduce_norm(c, stream));
}

ar_status_t ar_norm_workspace(const ar_norm_t *shape, size_t *bytes) {
    NormRow r;
    if (!bytes) return AR_ERR_INVALID_ARG;
    const ar_status_t st = check_norm(shape, r);
    if (st != AR_OK) return st;
    *bytes = norm_space(norm_back_plan(shape->dtype, shape->rows, (int)shape->width));
    return AR_OK;
}

ar_status_t ar_reduce_norm_backward(const void *x, long long x_pitch, const ar_norm_t *shape, const void *weight,
                                    const float *rstd, const void *grad_out, const void *grad_summed, void *grad_x,
                                    float *grad_weight, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    NormBackArgs a{};
    ar_status_t st = check_norm(shape, a.r);
    if (st != AR_OK) return st;
    if (x_pitch == 0) x_pitch = shape->width;
    if ((st = check_pitches(&x_pitch, 1, shape->width)) != AR_OK) return st;
    if (misaligned(grad_weight, 4)) return AR_ERR_ALIGNMENT;
    const long long e = bytes_of(shape->dtype), rows = shape->rows, row = shape->width * e;
    const NormBackPlan plan = norm_back_plan(shape->dtype, rows, (int)shape->width);
    if (rows) {
        if (!x || !weight || !rstd || !grad_out || !grad_x) return AR_ERR_INVALID_ARG;
        if (misaligned(x, e) || misaligned(weight, bytes_of(shape->weight_dtype)) || misaligned(rstd, 4) ||
            misaligned(grad_out, e) || misaligned(grad_summed, e) || misaligned(grad_x, e))
            return AR_ERR_ALIGNMENT;
        const size_t need = grad_weight ? norm_space(plan) : 0;
        if ((st = check_space(need, workspace, workspace_bytes)) != AR_OK) return st;
        Span s[8];
        int k = 0;
        if (x != grad_x || (x_pitch != shape->width && rows > 1)) s[k++] = span_of(x, rows, row, x_pitch * e, false);
        if (grad_out != grad_x) s[k++] = flat_span(grad_out, rows * row, false);
        if (grad_summed && grad_summed != grad_x) s[k++] = flat_span(grad_summed, rows * row, false);
        s[k++] = flat_span(weight, shape->width * bytes_of(shape->weight_dtype), false);
        s[k++] = flat_span(rstd, rows * 4, false);
        s[k++] = flat_span(grad_x, rows * row, true);
        if (grad_weight) {
            s[k++] = flat_span(grad_weight, shape->width * 4, true);
            s[k++] = flat_span(workspace, (long long)need, true);
        }
        if (!apart(s, k)) return AR_ERR_INVALID_ARG;
    }
    a.r.weight = weight;
    a.x = (const char *)x;
    a.x_pitch = x_pitch;
    a.rstd = rstd;
    a.grad_out = (const char *)grad_out;
    a.grad_summed = (const char *)grad_summed;
    a.grad_x = (char *)grad_x;
    a.part = grad_weight ? (float *)workspace : nullptr;
    a.part_width = plan.width;
    return hip_status(launch_norm_back(shape->dtype, a, plan, grad_weight, stream));
}

ar_status_t ar_embedding(const void *const *tables, const ar_embed_t *shape, const int64_t *token_ids, void *out,
                         hipStream_t stream) {
    EmbedCall c;
    ar_status_t st = check_embed(shape, c);
    if (st != AR_OK) return st;
    if (c.tokens == 0) return AR_OK;
    if (!token_ids || !out) return AR_ERR_INVALID_ARG;
    Widths widths;
    c.pitches = widths.use(shape->pitches, c.n, c.width);
    Span s[AR_MAX_RANKS + 2];
    int k = 0;
    if ((st = check_tables(c, tables, false, s, k)) != AR_OK) return st;
    if (misaligned(token_ids, 8) || misaligned(out, bytes_of(c.out_dtype))) return AR_ERR_ALIGNMENT;
    s[k++] = flat_span(token_ids, c.tokens * 8, false);
    s[k++] = flat_span(out, c.tokens * c.width * bytes_of(c.out_dtype), true);
    if (!apart(s, k)) return AR_ERR_INVALID_ARG;
    c.t = (void *const *)tables;
    c.ids = token_ids;
    return hip_status(launch_embedding(c, out, stream));
}

ar_status_t ar_embedding_workspace(const ar_embed_t *shape, size_t *bytes) {
    EmbedCall c;
    if (!bytes) return AR_ERR_INVALID_ARG;
    const ar_status_t st = check_embed(shape, c);
    if (st != AR_OK) return st;
    *bytes = embed_space(c.tokens, c.width, c.vocab).bytes;
    return AR_OK;
}

ar_status_t ar_embedding_backward(const void *grad_out, const ar_embed_t *shape, const int64_t *token_ids,
                                  void *const *grads, int accumulate, void *workspace, size_t workspace_bytes,
                                  hipStream_t stream) {
    EmbedCall c;
    ar_status_t st = check_embed(shape, c);
    if (st != AR_OK) return st;
    if (c.tokens == 0 && accumulate) return AR_OK;
    if (c.tokens && (!token_ids || !grad_out)) return AR_ERR_INVALID_ARG;
    Widths widths;
    c.pitches = widths.use(shape->grad_pitches ? shape->grad_pitches : shape->pitches, c.n, c.width);
    Span s[AR_MAX_RANKS + 3];
    int k = 0;
    if ((st = check_tables(c, (const void *const *)grads, true, s, k)) != AR_OK) return st;
    const EmbedSpace w = embed_space(c.tokens, c.width, c.vocab);
    if (c.tokens) {
        if (misaligned(token_ids, 8) || misaligned(grad_out, bytes_of(c.out_dtype))) return AR_ERR_ALIGNMENT;
        if ((st = check_space(w.bytes, workspace, workspace_bytes)) != AR_OK) return st;
        s[k++] = flat_span(token_ids, c.tokens * 8, false);
        s[k++] = flat_span(grad_out, c.tokens * c.width * bytes_of(c.out_dtype), false);
        s[k++] = flat_span(workspace, (long long)w.bytes, true);
    }
    if (!apart(s, k)) return AR_ERR_INVALID_ARG;
    c.t = grads;
    c.ids = token_ids;
    c.accumulate = accumulate != 0;
    hipError_t e = hipSuccess;
    if (c.tokens) e = launch_embed_sort(c, w, (char *)workspace, stream);
    if (e == hipSuccess) e = launch_embed_sum(c, w, (char *)workspace, grad_out, stream);
    return hip_status(e);
}

ar_status_t ar_grad_workspace(const ar_grads_t *grads, size_t *bytes) {
    if (!bytes) return AR_ERR_INVALID_ARG;
    const ar_status_t st = check_grads(grads);
    if (st != AR_OK) return st;
    *bytes = grad_space(grads);
    return AR_OK;
}

ar_status_t ar_grad_norm(const ar_grads_t *grads, float scale, float *norm, void *workspace, size_t workspace_bytes,
                         hipStream_t stream) {
    ar_status_t st = check_grads(grads);
    if (st != AR_OK) return st;
    if (!(scale > 0.0f) || !std::isfinite(scale) || !norm) return AR_ERR_INVALID_ARG;
    if ((st = check_grad_buffers(grads, grads->bufs)) != AR_OK) return st;
    if (misaligned(norm, 4)) return AR_ERR_ALIGNMENT;
    const size_t need = grad_space(grads);
    if ((st = check_space(need, workspace, workspace_bytes)) != AR_OK) return st;
    const uintptr_t n0 = (uintptr_t)norm, w0 = (uintptr_t)workspace;
    bool meets = need && n0 < w0 + need && w0 < n0 + 4;
    for (long long i = 0; i < grads->count; ++i) {
        const uintptr_t lo = (uintptr_t)grads->bufs[i], hi = lo + (uintptr_t)(grads->sizes[i] * bytes_of(grads->dtypes[i]));
        meets |= lo < hi && ((n0 < hi && lo < n0 + 4) || (w0 < hi && lo < w0 + need));
    }
    if (meets) return AR_ERR_INVALID_ARG;
    GradTable t{};
    t.scale = scale;
    hipError_t e = sum_squares(grads, nullptr, t, (double *)workspace + 1, stream);
    t.norm = norm;
    if (e == hipSuccess) e = launch_grad_finish(t, stream);
    return hip_status(e);
}

ar_status_t ar_clip_grads(const ar_grads_t *grads, void *const *outs, float max_norm, float scale, float eps,
                          float *norm, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    ar_status_t st = check_grads(grads);
    if (st != AR_OK) return st;
    if (!(scale > 0.0f) || !std::isfinite(scale) || !norm || !(max_norm >= 0.0f) || !(eps >= 0.0f) || !std::isfinite(eps))
        return AR_ERR_INVALID_ARG;
    if ((st = check_grad_buffers(grads, grads->bufs)) != AR_OK ||
        (st = check_grad_buffers(grads, (const void *const *)outs)) != AR_OK)
        return st;
    if (misaligned(norm, 4)) return AR_ERR_ALIGNMENT;
    const size_t need = grad_space(grads);
    if ((st = check_space(need, workspace, workspace_bytes)) != AR_OK) return st;
    {
        std::unique_ptr<Span[]> s(new (std::nothrow) Span[2 * grads->count + 2]);
        if (!s) return AR_ERR_UNSUPPORTED;
        long long k = 0;
        (void)each_piece(grads, outs, [&](const GradPiece &p) {
            const long long bytes = p.size * bytes_of(p.dtype);
            if (p.in != p.out) s[k++] = flat_span(p.in, bytes, false);
            s[k++] = flat_span(p.out, bytes, true);
            return hipSuccess;
        });
        s[k++] = flat_span(norm, 4, true);
        if (need) s[k++] = flat_span(workspace, (long long)need, true);
        if (!apart(s.get(), k)) return AR_ERR_INVALID_ARG;
    }
    GradTable t{};
    t.scale = scale;
    t.max_norm = max_norm;
    t.eps = eps;
    hipError_t e = sum_squares(grads, outs, t, (double *)workspace + 1, stream);
    t.norm = norm;
    if (e == hipSuccess && (t.parts == 0 || t.parts > kGradInline)) {
        t.wide = t.parts ? (double *)workspace : nullptr;
        e = launch_grad_finish(t, stream);
        t.parts = 0;
        t.norm = nullptr;
    }
    t.chunk = 0;
    if (e == hipSuccess)
        e = each_table(grads, outs, t, [&](GradTable &t, uint32_t chunks) {
            const hipError_t e = launch_grad_scale(t, chunks, stream);
            t.norm = nullptr;
            return e;
        });
    return hip_status(e);
}

}  // extern "C"
