// vocab_launch.hpp -- host side of the vocabulary-split launches: geometry
// from the call, one workgroup per row and part.
#pragma once

#include <cmath>

#include "dispatch.hpp"
#include "vocab_kernels.hpp"

namespace ar {

// Rows per launch: the grid's threads must stay below 2^32.
constexpr long long kVocabGridThreads = 1LL << 31;

template <int NR> void fill_geom(const VocabCall &c, VocabGeom<NR> &g) {
    int col = 0;
    for (int r = 0; r < c.n; ++r) {
        g.x[r] = (const char *)c.x[r];
        g.g[r] = c.g ? (char *)c.g[r] : nullptr;
        g.pitch[r] = (uint32_t)c.pitches[r];
        g.gpitch[r] = (uint32_t)c.gpitches[r];
        g.col0[r] = col;
        col += (int)c.widths[r];
    }
    for (int r = c.n; r <= NR; ++r) g.col0[r] = col;           // no column is past them
    for (int r = c.n; r < NR; ++r) g.x[r] = nullptr, g.g[r] = nullptr, g.pitch[r] = g.gpitch[r] = 0;
    g.n = c.n;
    g.parts = c.parts;
    g.tiles = c.tiles;
    g.skew = c.skew;
    const double scale = 1.4426950408889634 / (double)c.temperature;
    g.c = (float)scale;
    g.c_low = (float)(scale - (double)g.c);
    g.inv_t = (float)(1.0 / (double)c.temperature);
}

// One workgroup of ``waves`` waves for each of ``per_row`` parts of every row,
// with ``lds`` bytes beside what the kernel declares.
template <int NR, typename A>
hipError_t launch_rows(const VocabCall &c, const A &a, void (*k)(const VocabGeom<NR>, const A), int per_row, int waves,
                       hipStream_t s, size_t lds = 0) {
    VocabGeom<NR> g;
    fill_geom(c, g);
    const long long most = kVocabGridThreads / (64LL * waves * per_row);
    for (long long row = 0; row < c.rows; row += most) {
        g.row0 = row;
        const long long n = c.rows - row < most ? c.rows - row : most;
        const hipError_t e = launch(k, dim3((unsigned)(n * per_row)), dim3(64u * (unsigned)waves), lds, s, g, a);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <typename F> hipError_t dispatch_vocab(const VocabCall &c, F &&f) {
    auto by_n = [&](auto dt) {
        return c.n <= kVocabFew && !c.tiny ? f(dt, std::integral_constant<int, kVocabFew>{})
                                : f(dt, std::integral_constant<int, kVocabMany>{});
    };
    switch (c.dtype) {
    case F32: return by_n(std::integral_constant<int, F32>{});
    case BF16: return by_n(std::integral_constant<int, BF16>{});
    case F16: return by_n(std::integral_constant<int, F16>{});
    default: return hipErrorInvalidValue;
    }
}

}  // namespace ar
