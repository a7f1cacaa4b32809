// split.h -- products with few output tiles and a long K, gfx950: K is split
// over workgroups as well, each writes its share of the sums as fp32, and a
// second kernel adds the shares in order and finishes the values.  The shares
// are joined in a fixed order, so results do not depend on timing.  How K is
// shared: dense_pick.h.
#pragma once
#include "dense_core.h"
#include "dense_pick.h"

namespace dmm {
namespace split {
using namespace dense;

struct Args {
    const void* a[2];  // one per segment
    const void* b[2];  // one per segment, or the two stacked matrices of a gated tile
    float* part;       // [shares][m][n] (gated: [shares][m][2][n])
    int m, n, kext;    // kext: K bytes of a row of a
    Plan plan;
    int tiles_m, tiles_n;
};

template <class C>
__device__ __forceinline__ void partial_body(const Ring& ring, const Args& p, int block) {
    Ctx<C> x = make_ctx<C>(ring);
    const int tiles = p.tiles_m * p.tiles_n, per_seg = p.plan.shares / p.plan.segs;
    const int share = block / tiles, seg = share / per_seg;
    int tm, tn;
    order::coords(block - share * tiles, p.tiles_m, p.tiles_n, tm, tn);
    constexpr int COLS = C::GATED ? C::HALF : C::BN;
    const int m0 = tm * C::BM, n0 = tn * COLS, wm = x.w >> 1, wn = x.w & 1;
    const int first = (share - seg * per_seg) * p.plan.per;
    x.la.init(Mat{p.a[seg], p.kext, p.m}, m0, p.kext, x.w, x.lane);
    if constexpr (C::GATED)
        x.lb.init(Mat{p.b[wm], p.kext, p.n}, n0, p.kext, x.w, x.lane, C::HALF, wn);
    else if constexpr (C::LB == KC)
        x.lb.init(Mat{p.b[seg], p.kext, p.n}, n0, p.kext, x.w, x.lane);
    else
        x.lb.init(Mat{p.b[seg], (int64_t)p.n * 2, p.n}, n0, p.kext / 2, x.w, x.lane);
    x.KT = (p.kext + 127) / 128 - first;
    x.KT = x.KT < 0 ? 0 : x.KT > p.plan.per ? p.plan.per : x.KT;
    x.la.range(first, x.KT);
    x.lb.range(first, x.KT);
    x.ra.init(wm * (C::BM / 2), x.lane);
    x.rb.init(wn * (COLS / 2), x.lane);
    run(x);

    const int width = C::GATED ? 2 * p.n : p.n;
    const FloatRows out(p.part + (int64_t)share * p.m * width, m0, C::BM, p.m, width);
#pragma unroll
    for (int mb = 0; mb < C::MB; ++mb) {
        claim(x.acc[mb]);
        const int row = wm * (C::BM / 2) + 16 * mb + (x.lane & 15);
#pragma unroll
        for (int nb = 0; nb < C::NB; nb += 2) {
            const bool up = C::GATED && nb >= C::NB / 2;
            const int col = n0 + wn * (COLS / 2) + 16 * (nb - (up ? C::NB / 2 : 0)) + pair_column(x.lane);
            float v[8];
            pair_columns(x.acc[mb][nb], x.acc[mb][nb + 1], v);
            out.store(row, col < p.n ? col + (up ? p.n : 0) : -1, v);
        }
    }
}

template <class C>
__global__ void __launch_bounds__(kThreads) partial_kernel(Args p) {
    DENSE_LDS(C, ring);
    partial_body<C>(ring, p, (int)blockIdx.x);
}

// Sets the tile counts; the workgroups that partial_body takes.
template <class C>
inline int partial_blocks(Args& p) {
    p.tiles_m = (int)ceil_div(p.m, C::BM);
    p.tiles_n = (int)ceil_div(p.n, C::GATED ? C::HALF : C::BN);
    return p.tiles_m * p.tiles_n * p.plan.shares;
}

template <class C>
hipError_t launch_partial(Args p, hipStream_t st) {
    const int blocks = partial_blocks<C>(p);
    hipLaunchKernelGGL((partial_kernel<C>), dim3(blocks), dim3(kThreads), 0, st, p);
    return hipGetLastError();
}

// Eight consecutive values of row r, columns c .. c + 7, summed over the shares.
__device__ __forceinline__ void sum8(const float* part, int shares, int64_t stride, int64_t at, float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
#pragma unroll 4
    for (int s = 0; s < shares; ++s) {
        const v4f* q = (const v4f*)(part + s * stride + at);
        const v4f lo = q[0], hi = q[1];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] += lo[e];
            v[4 + e] += hi[e];
        }
    }
}

}  // namespace split
}  // namespace dmm
