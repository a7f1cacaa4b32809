// dense_layout.h -- where the tile engine's operands lie in LDS and when its
// steps issue what.  Plain constexpr C++ shared by the kernels and their proofs
// on the host.
//
// A stage holds one K tile, 128 bytes of K, of ROWS rows.
//   KC (K contiguous): row r at 128 r, its 16-byte chunk c at position
//     c ^ ((r >> 1) & 7).  A fragment (16 rows) is one 16-byte read per lane and
//     k half: lane (i, g) = (l % 16, l / 16) reads row i, chunk 4 h + g; the 16
//     lanes of a read phase touch 16 distinct 16-byte bank groups.
//   KR (one line of all rows per K value, 16-bit): K value k at 2 ROWS k, its
//     32-byte chunk c (16 rows) at position c ^ kr_xor(k, ROWS).  A fragment is
//     two transposing 8-byte reads per lane and k half: lane i of a 16-lane
//     group names the 8 bytes of K value (i / 4), rows 4 (i % 4) .. + 3, and
//     receives row i's four K values.  32 lanes cover eight K values, whose
//     32-byte chunks fall on distinct banks.
// Both give lane (i, g) the K values 32 h + 8 g .. + 7 of row i, so layouts mix.
//
// The DMA that fills a stage writes 16 bytes per lane at consecutive addresses,
// so the permutation is applied on the global side: that lane fetches the
// chunk that belongs there.
#pragma once

namespace dmm {
namespace dense {

// 16-byte chunk position in a KC row (an involution in c)
constexpr int kc_pos(int r, int c) { return c ^ ((r >> 1) & 7); }

// XOR of the 32-byte chunk index of a KR line.  A line of 64 rows has four
// chunks, and two lines lie side by side in the 256 bytes of bank space.
constexpr int kr_xor(int k, int rows) {
    return rows > 64 ? (k & 3) | (((k >> 3) & 1) << 2) : ((k >> 1) & 1) | (((k >> 3) & 1) << 1);
}

// What the lane that writes byte `byte` of a stage fetches.
constexpr int kc_row(int byte) { return byte / 128; }
constexpr int kc_chunk(int byte) { return kc_pos(byte / 128, byte % 128 / 16); }
constexpr int kr_k(int byte, int rows) { return byte / (2 * rows); }
constexpr int kr_col(int byte, int rows) {  // the first of eight rows
    const int p16 = byte % (2 * rows) / 16;
    return 16 * ((p16 >> 1) ^ kr_xor(kr_k(byte, rows), rows)) + 8 * (p16 & 1);
}

// Fragment reads of lane (i, g), 16-row block q of a wave whose rows start at
// row0 (a multiple of 16): KC, the 16 bytes of half h; KR, the 8 bytes of the
// first four K values of half 0 (half h: + 64 rows h; the other four: + 8 rows).
constexpr int kc_read(int row0, int q, int i, int g, int h) {
    return (row0 + 16 * q + i) * 128 + kc_pos(i, 4 * h + g) * 16;
}
constexpr int kr_read(int row0, int q, int i, int g, int rows) {
    const int k = 8 * g + (i >> 2);
    return k * (2 * rows) + (((row0 >> 4) + q) ^ kr_xor(k, rows)) * 32 + (i & 3) * 8;
}

// Where in a step's T matrix ops its other work goes.  One memory instruction
// at most follows a matrix op wherever there is room: the op keeps the matrix
// unit busy for 16 cycles (32 in fp8), the issue of up to three other
// instructions fits in there, and a run of them leaves the unit idle.  The
// DMAs are spread widest: the path from the L1 into LDS moves 64 bytes a
// cycle, so a K tile of the 256 x 256 shape takes half a step.  Against
// a spread over five eighths of a step, timed in turn, the forward and backward
// passes of the feed-forward block at 16384 x 7168 x 2048 take 1.6 and 2.0 % more
// with one over half, 4.4 and 5.2 % over three eighths; eleven sixteenths, or the
// barrier an eighth of a step later, are within 1 %.
template <int T, int FIRST, int SECOND, int DMAS>
struct Plan {
    static constexpr int kMid = T * 9 / 32;  // the wait and the barrier come before matrix op kMid
    // How many of a kind have been issued once matrix op t has been: the u-th
    // of n goes after op at + u * span / n.
    static constexpr int due(int t, int at, int span, int n) {
        const int v = t < at ? 0 : ((t - at + 1) * n + span - 1) / span;
        return v < n ? v : n;
    }
    // reads of this stage: over by the barrier, with time to return
    static constexpr int first(int t) { return due(t, 0, T * 3 / 16, FIRST); }
    static constexpr int dma(int t) { return due(t, kMid, T * 5 / 8, DMAS); }
    // reads of the next stage, from matrix op FROM on
    template <int FROM>
    static constexpr int second(int t) {
        return due(t, FROM, T * 7 / 8 - FROM, SECOND);
    }
};

}  // namespace dense
}  // namespace dmm
