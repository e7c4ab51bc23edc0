// layer_kernels.hpp -- launch arguments of the operators around a step's
// collectives (host and device side): reduction with residual and RMS norm,
// embedding over a split vocabulary, gradient norm.  Tables of ranks and of
// buffers travel by value, within the 4 KB of a kernel's arguments.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ar {

constexpr int kLayerFew = 16;          // ranks of the small pointer table
constexpr int kLayerMany = 128;        // ranks of the large one
constexpr float kE4m3Max = 448.0f;
constexpr float kLeastScale = 0x1p-100f;

// ---- reduction, residual, norm ---------------------------------------------
struct NormRow {                       // what forward and backward have in common
    const void *weight;
    bool weight32;                     // the weight is fp32 (else of the storage type)
    int width;
    float eps, offset;
    long long rows, row0;              // rows in all; the first one of this launch
};

template <int NR> struct NormArgs {
    const char *x[NR];                 // partials
    uint32_t pitch[NR];                // elements between rows
    int n;
    int group;                         // runs that share a scale; 0: the row
    int groups;                        // scales of a row
    NormRow r;
    const char *residual;
    char *summed, *out;
    float *rstd;
    uint8_t *out8;
    float *scales;
};

struct NormBackArgs {
    NormRow r;
    const char *x;
    long long x_pitch;
    const float *rstd;
    const char *grad_out, *grad_summed;
    char *grad_x;
    float *part;                       // [workgroups, part_width] partial weight gradients; NULL: none wanted
    int part_width;
};

// Host-side description of a forward launch, rank tables of any size.
struct NormCall {
    int dtype, n;
    const void *const *x;
    const long long *pitches;
    NormArgs<1> a;                     // all but the rank table
};

hipError_t launch_reduce_norm(const NormCall &c, hipStream_t s);
// Workgroups of the backward pass, and the places of the partial weight gradient that each leaves.
struct NormBackPlan {
    int groups, width;
};
NormBackPlan norm_back_plan(int dtype, long long rows, int width);
hipError_t launch_norm_back(int dtype, const NormBackArgs &a, const NormBackPlan &plan, float *grad_weight, hipStream_t s);

// ---- embedding ---------------------------------------------------------------
template <int NR> struct EmbedTable {
    char *t[NR];                       // each rank's rows (only read by the lookup)
    uint32_t pitch[NR];
    int first[NR + 1];                 // first entry of each rank; V from first[n] on
    int n;
};

struct EmbedCall {
    int dtype, out_dtype;              // of the table and of the looked-up rows
    int n;
    void *const *t;
    const long long *entries, *pitches;
    long long tokens;
    int width, vocab;
    float scale;
    const int64_t *ids;
    bool accumulate;
};

// Sorted tokens: key s of the order is token keys[s] at position order[s],
// equal tokens by position; what is no token has the key `vocab`, after all others.
struct EmbedSorted {
    uint32_t *keys, *order;
};

// Pieces of the backward pass's workspace.
struct EmbedSpace {
    size_t keys, order, map, keys2, order2, hist, totals, part, bytes;
    int piece;                         // sorted positions to a workgroup
    long long pieces;
    int digit, passes;                 // bits of a counting pass, and how many (0: ranked in one launch)
    int tile;                          // tokens of a workgroup of a counting pass
    long long tiles;
};
EmbedSpace embed_space(long long tokens, int width, int vocab);

hipError_t launch_embedding(const EmbedCall &c, void *out, hipStream_t s);
hipError_t launch_embed_sort(const EmbedCall &c, const EmbedSpace &w, char *space, hipStream_t s);
hipError_t launch_embed_sum(const EmbedCall &c, const EmbedSpace &w, char *space, const void *grad_out, hipStream_t s);

// ---- gradient norm -----------------------------------------------------------
constexpr int kGradTable = 120;        // buffers of a launch
constexpr int kGradChunk = 4096;       // elements that a workgroup takes at a time, doubled while there are more chunks than
constexpr int kGradLongChunk = 65536;  // workgroups, up to this
constexpr int kGradGroups = 4096;      // most workgroups, one partial sum each, of a launch

constexpr int kGradScaleBytes = 8192;  // that a workgroup scales
constexpr int kGradInline = 256;       // most partial sums that every workgroup of the scaling launch adds up by itself

struct GradPiece {                     // buffers that adjoin, as one
    const char *in;
    char *out;
    long long size;
    int dtype;
};

struct GradTable {
    const char *in[kGradTable];
    char *out[kGradTable];
    uint32_t size[kGradTable];         // elements
    uint32_t first[kGradTable + 1];    // first chunk; all chunks from first[n] on
    uint8_t dtype[kGradTable];
    int n;
    int chunk;                         // elements, kGradChunk to kGradLongChunk
    bool again;                        // what is read for the norm stays in the cache for the scaling
    double *part;                      // of this launch (sums) or of all launches (scaling)
    int parts;                         // partial sums of all launches; 0 (scaling): `wide` holds the norm
    float scale, max_norm, eps;
    float *norm;                       // where the norm is written, by one launch
    double *wide;                      // the norm in 64 bits
};

// Most elements of a table entry, whole chunks (larger buffers are cut).
constexpr long long kGradPieceMax = (1LL << 32) - kGradLongChunk;

hipError_t launch_grad_sum(const GradTable &t, int groups, hipStream_t s);
hipError_t launch_grad_finish(const GradTable &t, hipStream_t s);
hipError_t launch_grad_scale(const GradTable &t, uint32_t groups, hipStream_t s);

}  // namespace ar
