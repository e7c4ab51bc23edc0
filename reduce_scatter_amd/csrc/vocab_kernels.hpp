// vocab_kernels.hpp -- launch arguments of the vocabulary-split reductions
// (host and device side): softmax statistics, top alternatives, distillation
// and their gradients over rows whose columns lie in n rank buffers.
//
// A row is cut into tiles of 64 lanes x kVocabU 16-byte vectors, each within
// one rank (a rank's last tile may be short), numbered rank by rank.  `parts`
// workgroups of W waves share a row; wave w of part p takes tiles p*W + w,
// p*W + w + parts*W, ...  Pointer tables travel by value (about 0.6 KB for up
// to 16 ranks, 3.7 KB for up to 128).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ar {

constexpr int kVocabU = 4;             // 16-byte vectors per lane and tile
constexpr int kVocabWaves = 8;         // most waves per workgroup
constexpr int kHeldWaves = 16;         // the same for rows held in registers
constexpr int kHeldTiles = 4;          // most tiles per wave of such a row (64 registers)
constexpr int kVocabParts = 32;        // most workgroups per row
constexpr int kVocabFew = 16;          // ranks of the small pointer table
constexpr int kVocabMany = 128;        // ranks of the large one
constexpr int kTopMax = 64;            // one list entry per lane
constexpr int kTeacherMax = 256;

template <int NR> struct VocabGeom {
    const char *x[NR];                 // logits of each rank
    char *g[NR];                       // gradients (unused by forward kernels)
    uint32_t pitch[NR], gpitch[NR];    // elements between rows
    int col0[NR + 1];                  // first column of each rank; V from col0[n] on
    int n, parts;
    int tiles;                         // of the row, over all ranks
    int skew;                          // 0, or where some row is off a 16-byte boundary a vector's elements less one
    float c, c_low;                    // log2(e) / T, and what rounding it to c leaves
    float inv_t;                       // 1 / T
    long long row0;                    // first row of this launch
};

struct LogprobsArgs {
    const int64_t *targets;
    float *logprobs, *entropy, *saved;
    const float *grad_logprobs, *grad_entropy;
    float *top_logprobs;
    int64_t *top_ids;
    int k;
    float4 *part;                      // [rows * parts] partial statistics
    unsigned long long *part_top;      // [rows * parts * k] partial lists
};

struct DistillArgs {
    const int64_t *ids;
    const float *values;
    int k;
    float *loss, *saved;
    const float *grad_loss;
    float4 *part;
};

// Host-side description of a launch, rank tables of any size.
struct VocabCall {
    int dtype;                         // ar::Dtype
    long long rows;
    int n, tiles, parts, waves;
    int held;                          // kBoth: tiles per wave where a row fits in registers, 1, 2 or kHeldTiles; 0: it does not
    int skew;                          // as VocabGeom's
    bool again;                        // kForward: a backward call on the same logits follows, and they fit the cache
    bool tiny;                         // a rank has columns, but not enough for one vector
    const void *const *x;
    void *const *g;                    // nullptr for forward calls
    const long long *widths, *pitches, *gpitches;
    float temperature;
};

enum VocabStage : int {
    kForward = 0,                      // statistics, and the row's results when parts == 1
    kJoin = 1,                         // results from the parts' partials
    kBackward = 2,                     // gradients from saved statistics
    kBoth = 3                          // statistics and gradients of a row in one workgroup (parts == 1)
};

hipError_t launch_logprobs(const VocabCall &c, const LogprobsArgs &a, VocabStage stage, hipStream_t s);
hipError_t launch_distill(const VocabCall &c, const DistillArgs &a, bool tail, VocabStage stage, hipStream_t s);

}  // namespace ar
