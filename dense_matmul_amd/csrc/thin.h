// thin.h -- products of few rows, gfx950: 16 streamed rows (a weight's, or for
// the adapters the tokens) against 16 MB rows of the other operand x per
// workgroup, K split over its waves.
//
// Such a product is bound by reading the streamed rows once, so they go
// straight from memory to the matrix op's registers (no LDS: no wave uses
// another's) and every wave keeps all of its K share's loads in
// flight: lane (i, g) = (l % 16, l / 16) reads 16 bytes of streamed row i, four
// lanes a 64-byte run, two such steps a 128-byte unit.  x comes from the L2 in
// the same shape.  The waves' partial products meet in LDS and are summed in
// wave order, so the result does not depend on timing.
#pragma once
#include "common.h"
#include "dense_pick.h"

namespace dmm {
namespace thin {

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ v4f matrix_op(bool fp8, v4i w, v4i x, v4f c) {
#if defined(__HIP_DEVICE_COMPILE__)
    if (fp8) {
        const long w0 = ((long)(uint32_t)w[1] << 32) | (uint32_t)w[0], w1 = ((long)(uint32_t)w[3] << 32) | (uint32_t)w[2];
        const long x0 = ((long)(uint32_t)x[1] << 32) | (uint32_t)x[0], x1 = ((long)(uint32_t)x[3] << 32) | (uint32_t)x[2];
        c = __builtin_amdgcn_mfma_f32_16x16x32_fp8_fp8(w0, x0, c, 0, 0, 0);
        return __builtin_amdgcn_mfma_f32_16x16x32_fp8_fp8(w1, x1, c, 0, 0, 0);
    }
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, w), __builtin_bit_cast(bf8, x), c, 0, 0, 0);
#else
    (void)fp8, (void)w, (void)x;
    return c;
#endif
}

// acc[b]: this wave's share of x rows 16 b .. times the streamed rows; lane
// (i, g) ends with x row 16 b + i, streamed rows 4 g .. + 3.  wrow and xrow are
// the lane's rows (any valid row where there is none: such outputs are not
// used), kb the bytes of a row, a multiple of 16.
template <bool FP8, int MB, int WAVES>
__device__ __forceinline__ void product(const char* wrow, const char* const (&xrow)[MB], int kb, v4f (&acc)[MB]) {
    constexpr int UN = MB == 1 ? 4 : 2;  // 128-byte units in flight
    const int lane = lane_id(), w = wave_id(), at = 16 * (lane >> 4);
    const int units = (kb + 127) / 128, per = (units + WAVES - 1) / WAVES;
    const int lo = w * per, end = lo + per < units ? lo + per : units, whole = kb / 128;
    const int full = end < whole ? end : whole;
#pragma unroll
    for (int b = 0; b < MB; ++b) acc[b] = (v4f){0.f, 0.f, 0.f, 0.f};
    int u = lo;
    for (; u + UN <= full; u += UN) {
        v4i wv[2 * UN], xv[MB][2 * UN];
#pragma unroll
        for (int s = 0; s < 2 * UN; ++s) wv[s] = __builtin_nontemporal_load((const v4i*)(wrow + u * 128 + 64 * s + at));
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
            for (int s = 0; s < 2 * UN; ++s) xv[b][s] = *(const v4i*)(xrow[b] + u * 128 + 64 * s + at);
#pragma unroll
        for (int s = 0; s < 2 * UN; ++s)
#pragma unroll
            for (int b = 0; b < MB; ++b) acc[b] = matrix_op(FP8, wv[s], xv[b][s], acc[b]);
    }
    // what is left of the share, the row's last partial unit included: both
    // operands are zero past the row's end
    for (; u < end; ++u)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int off = u * 128 + 64 * s + at;
            const bool in = off < kb;
            const int from = in ? off : 0;
            v4i wv = *(const v4i*)(wrow + from);
            if (!in) wv = (v4i){0, 0, 0, 0};
#pragma unroll
            for (int b = 0; b < MB; ++b) {
                v4i xv = *(const v4i*)(xrow[b] + from);
                if (!in) xv = (v4i){0, 0, 0, 0};
                acc[b] = matrix_op(FP8, wv, xv, acc[b]);
            }
        }
}

// The waves' shares in LDS, and the sum over them of x row r, streamed row n.
template <int MB, int WAVES>
struct Join {
    v4f part[WAVES][MB][64];
    __device__ __forceinline__ void put(const v4f (&acc)[MB]) {
#pragma unroll
        for (int b = 0; b < MB; ++b) part[wave_id()][b][lane_id()] = acc[b];
        __syncthreads();
    }
    __device__ __forceinline__ float sum(int r, int n) const {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) s += part[w][r >> 4][(r & 15) + 16 * (n >> 2)][n & 3];
        return s;
    }
};

__device__ __forceinline__ uint16_t to_bf16(float v) { return (uint16_t)(pack_bf16(v, 0.f) & 0xffff); }

}  // namespace thin
}  // namespace dmm

// F<WAVES> for rows of kb bytes
#define THIN_BY_SIZE(F, kb, ...)                     \
    (thin::waves_for(kb) == 16  ? F<16>(__VA_ARGS__) \
     : thin::waves_for(kb) == 8 ? F<8>(__VA_ARGS__)  \
                                : F<4>(__VA_ARGS__))
