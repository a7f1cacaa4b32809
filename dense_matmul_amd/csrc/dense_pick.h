// dense_pick.h -- which tile shape a product of the tile engine takes, from
// its sizes alone.  Plain C++.
//
// Each shape's time is modelled as rounds of workgroups over the compute
// units, a round costing a start-and-end part plus a part per K tile (128
// bytes of K).  The constants are microseconds fitted to kernel times measured
// on one MI355X over twelve problems of 129 to 8192 rows (all three layout
// pairs; the model is within 15 % of most and picks the fastest shape or one
// within 10 % of it).  What the choice is worth, measured, rows x K -> columns:
//   1003 x 1024 -> 1024:  64 x 64   5.6 us, 128 x 128 10.0,  256 x 256 20.8
//   600 x 1792 -> 4096:   128 x 128 (4 stages) 14.9 us, 64 x 64 18.5, 256 x 256 36.2
//   4096 x 1024 -> 2048:  128 x 128 (2 stages) 21.9 us, 256 x 256 26.0, 64 x 64 29.6
//   8192 x 1024 -> 2048:  256 x 256 31.0 us, 128 x 128 36.4, 64 x 64 59.6
#pragma once
#include <stdint.h>

namespace dmm {
namespace dense {

enum Tile {
    kTile256,   // 256 x 256, two stages: one workgroup per compute unit
    kTile128,   // 128 x 128, two stages: two per unit, for grids of more than one round
    kTile128D,  // 128 x 128, four stages: one per unit, for grids of one round
    kTile64     // 64 rows x 64 columns (or x 64 columns of each of two matrices), four stages
};

// Compute units of the part this library is built for.  A constant and not the
// device's property: a workspace query makes no HIP call, and the choices, with
// them the workspace and the order of a call's sums, depend on the problem
// alone.  On a device of fewer units a wrong choice costs time only.
constexpr int kUnits = 256;

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t larger(int64_t a, int64_t b) { return a > b ? a : b; }

// Time of t 64 x 64 tiles beside others in the same launch, and alone.
inline double cost64_more(int64_t t, int64_t kt) {
    return (double)t / (double)kUnits * (0.8 + 0.19 * (double)kt);
}
inline double cost64(int64_t t, int64_t kt) {
    return 2.7 + cost64_more(t < kUnits ? kUnits : t, kt);
}

// rows x cols output (count matrices of them in one launch), kt K tiles.
// gated: a tile's columns are half of each of two matrices.
// cost: where to put the modelled microseconds.
inline Tile pick_tile(int64_t rows, int64_t cols, int64_t kt, bool gated, int count = 1, double* cost = nullptr) {
    constexpr int64_t cus = kUnits;
    const int64_t t256 = count * ceil_div(rows, 256) * ceil_div(cols, gated ? 128 : 256);
    const int64_t t128 = count * ceil_div(rows, 128) * ceil_div(cols, gated ? 64 : 128);
    const int64_t t64 = count * ceil_div(rows, 64) * ceil_div(cols, 64);
    const double k = (double)kt;
    const double c256 = (double)ceil_div(t256, cus) * (6.0 + (2 * t256 <= cus ? 1.1 : 1.5) * k);
    const double c128 = t128 <= cus ? 2.5 + 0.64 * k : (double)ceil_div(t128, 2 * cus) * (6.0 + 0.83 * k);
    const double c128d = (double)ceil_div(t128, cus) * (4.8 + (t128 <= cus ? 0.36 : 0.42) * k);
    const double c64 = gated ? (double)ceil_div(t64, cus) * (2.7 + 0.27 * k)
                             : cost64(t64, kt);
    Tile best = kTile256;
    double c = c256;
    if (c128 < c) best = kTile128, c = c128;
    if (c128d < c) best = kTile128D, c = c128d;
    if (c64 < c) best = kTile64, c = c64;
    if (cost) *cost = c;
    return best;
}

}  // namespace dense
}  // namespace dmm
