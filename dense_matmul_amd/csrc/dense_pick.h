// dense_pick.h -- which kernels a product of the feed-forward block or of the
// adapters takes, from its sizes alone.  Plain C++.
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
    kTile64,    // 64 rows x 64 columns (or x 64 columns of each of two matrices), four stages
    kSplit,     // kTile64 with K shared out over workgroups (split.h)
    kThin       // the kernels for few tokens (thin.h)
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

namespace split {
using namespace dense;

constexpr int kMost = 16;  // shares of one output value

// How K is shared: `per` K tiles to a share, `shares` shares in all; with two
// segments (a b + a2 b2) the first half of the shares takes the first product.
struct Plan {
    int shares, per, segs;
};

// The plan for rows x cols outputs over kt K tiles (of each segment), or shares
// = 1 where no split pays.  Model as in pick_tile: the tiles' round, the shares'
// way to memory and back, and a second launch.  Worth it where the tiles alone
// would leave most compute units idle: at 64 x 7168 -> 2 x 2048 columns there
// are 32 tiles of 112 K tiles each for 256 units.
inline Plan plan(int64_t rows, int64_t cols, int64_t kt, int segs, bool gated, double unsplit) {
    const int64_t cus = kUnits, tiles = ceil_div(rows, 64) * ceil_div(cols, 64);
    Plan best{1, (int)kt, segs};
    double c = unsplit;
    for (int64_t s = 2 / segs; s * segs <= kMost; ++s) {
        if (s * segs < 2) continue;
        const int64_t per = ceil_div(kt, s), n = ceil_div(kt, per) * segs;
        if (per < 4 || n < 2) break;
        const double round = (double)ceil_div(tiles * n, cus) * (2.7 + (gated ? 0.27 : 0.23) * (double)per);
        const double t = round + 4.0 + (double)(n * rows * cols * (gated ? 2 : 1)) * 8e-6 / 4.0;
        if (t < c) best = Plan{(int)n, (int)per, segs}, c = t;
    }
    return best;
}

inline int64_t bytes(const Plan& p, int64_t m, int64_t n, bool gated) {
    return p.shares < 2 ? 0 : (int64_t)p.shares * m * n * (gated ? 8 : 4);
}
}  // namespace split

namespace thin {
// Waves for a row of kb bytes: two 128-byte units or more each.
constexpr int waves_for(int kb) { return kb >= 4096 ? 16 : kb >= 2048 ? 8 : 4; }
}  // namespace thin

namespace ffn {
using namespace dense;

constexpr int kThinMost = 16;  // tokens that take the thin kernels

struct Choice {
    Tile tile;
    split::Plan plan;  // shares > 1 with kSplit only
};

// The gate and up projections together; eb: bytes of an operand's value.
inline Choice up_choice(int64_t m, int64_t d, int64_t f, int eb) {
    if (m <= kThinMost) return {kThin, {1, 0, 1}};
    double unsplit;
    const int64_t kt = ceil_div(d * eb, 128);
    const Tile t = pick_tile(m, f, kt, true, 1, &unsplit);
    const split::Plan p = split::plan(m, f, kt, 1, true, unsplit);
    return {p.shares > 1 ? kSplit : t, p};
}

// A bf16 product of m x n values over k, with seg the sum of two such.
inline Choice product_choice(int64_t m, int64_t n, int64_t k, bool seg) {
    double unsplit;
    const int64_t kt = ceil_div(k, 64), segs = seg ? 2 : 1;
    const Tile t = pick_tile(m, n, segs * kt, false, 1, &unsplit);
    const split::Plan p = split::plan(m, n, kt, (int)segs, false, unsplit);
    return {p.shares > 1 ? kSplit : t, p};
}

// The three weight gradients, in one launch.
inline Tile grads_choice(int64_t m, int64_t d, int64_t f) { return pick_tile(d, f, ceil_div(m, 64), false, 3); }

// Whether dx and the weight gradients are one launch of 64 x 64 tiles.
inline bool grads_with_dx(int64_t m, int64_t d, int64_t f) {
    double apart_x, apart_w;
    pick_tile(m, d, 2 * ceil_div(f, 64), false, 1, &apart_x);
    pick_tile(d, f, ceil_div(m, 64), false, 3, &apart_w);
    const double launch = 1.5;  // of a second kernel
    return product_choice(m, d, f, true).tile != kSplit &&
           cost64(ceil_div(m, 64) * ceil_div(d, 64), 2 * ceil_div(f, 64)) +
                   cost64_more(3 * ceil_div(d, 64) * ceil_div(f, 64), ceil_div(m, 64)) <
               apart_x + apart_w + launch;
}
}  // namespace ffn

namespace lora {
using namespace dense;

// Tokens whose adapters' part is summed value by value, at most.  256 tokens x
// 4096 -> 4096, 32 adapters of rank 16 in any order, take 40 us so, 512 the other
// way 76; the sums' reads of B grow with tokens x columns x rank, and at 256 x
// 7168 -> 7168, rank 128, they are 61 of 137 us where 257 tokens take 86.
constexpr int kJoinMost = 256;

// Shares of the few-token first product: 2 KiB of a row each, kMost at most.
inline int shrink_per(int k) {
    const int64_t per = larger(2048, ceil_div(ceil_div(2 * (int64_t)k, split::kMost), 128) * 128);
    return (int)per;
}
inline int shrink_shares(int k) { return (int)ceil_div(2 * (int64_t)k, shrink_per(k)); }

// Its workgroups: 16 tokens, one of their ids, 16 mb ranks and a share each.
inline int shrink_mb(int r) { return r <= 16 ? 1 : r <= 32 ? 2 : 4; }
inline int shrink_blocks(int m, int k, int r, int adapters) {
    const int nids = adapters < 16 ? adapters : 16;
    return (int)(ceil_div(m, 16) * nids * ceil_div(r, 16 * shrink_mb(r)) * shrink_shares(k));
}

// Whether it and the shared product's shares are one launch: where its
// workgroups take one place on each unit at most; more of them are held up by
// the stages they do not use (256 tokens x 4096, 32 adapters of rank 16: 52 us
// against 42).
inline bool shrink_with_base(int blocks) { return blocks <= kUnits; }

// How the shared product of few tokens is shared out.
inline split::Plan base_plan(int m, int n, int k) {
    const int64_t kt = ceil_div(k, 64);
    const double one = (double)ceil_div(ceil_div(m, 64) * ceil_div(n, 64), kUnits) * (2.7 + 0.23 * (double)kt);
    return split::plan(m, n, kt, 1, false, one);
}

// How the first product of many tokens is shared out: two workgroups a unit,
// four K tiles at least to a share.
inline split::Plan shrink_plan(int m, int k, int r) {
    const int64_t kt = ceil_div(k, 64), tiles = ceil_div(m, 64) * ceil_div(r, 64);
    int64_t s = 2 * kUnits / tiles;
    s = s > kt / 4 ? kt / 4 : s;
    s = s < 1 ? 1 : s > split::kMost ? split::kMost : s;
    const int64_t per = ceil_div(kt, s);
    return split::Plan{(int)ceil_div(kt, per), (int)per, 1};
}

// The second product of many tokens with the shared one; beside a given c there
// is little to do per tile, so 64 x 64 tiles of two stages, many at once.
inline Tile second_choice(int64_t m, int64_t n, int64_t k) { return pick_tile(m, n, ceil_div(k, 64), false); }
}  // namespace lora
}  // namespace dmm
