// ffn.hip -- the gated feed-forward block for gfx950, forward and backward:
//   g = x Wg^T, u = x Wu^T, h = act(g) u, y = h Wd^T
//   dh = dy Wd, dg = dh u act'(g), du = dh act(g), dWd = dy^T h,
//   dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x
// x, y [m, d]; Wg, Wu [f, d]; Wd [d, f]; all bf16, sums in fp32.  h, dg and du
// are rounded to bf16 once, as operands of the products that follow: the
// matrix op of the full rate takes 16-bit operands.  Relative error in the mean
// square against 64 bits 0.0022-0.0024, where one rounding of the result alone
// gives 0.0017.
//
// Many tokens are bound by the matrix cores: 6 m d f operations forward, 12 m d
// f backward, which the tile engine takes in two launches and three (dh with
// its gradients through the activation in the epilogue; dx over both pairs in
// one sum; the three weight gradients together, none through a transposed
// copy).  Measured at 16384 x 7168 x 2048: forward with gate and up kept
// 1040-1058 us (1.36-1.39 PFLOP/s), backward 2193-2207 (1.31), the matrix unit
// 63-72 % busy at the 1.6-1.9 GHz that the part's power allows.  Up to 16 tokens
// are bound by reading the weights once: one token of 7168 x 2048 takes 14 + 7 us
// in two launches (4.3 TB/s); 64 tokens, K shared out, 14 + 4 + 8.
#include "dense_core.h"
#include "dense_pick.h"
#include "split.h"
#include "thin.h"

namespace dmm {
namespace ffn {
using namespace dense;

enum Act { SILU = 0, GELU = 1 };

// Results that this call does not read again bypass the caches (nt sc1): timed in
// turn, the forward pass of 16384 x 7168 x 2048 with gate and up kept takes 2.1 %
// more without, the backward pass the same.  What the next product reads (h,
// dgate, dup) does not: 1.5 % slower backward.
constexpr int kStream = 2 | 16;

__device__ __forceinline__ float sigmoid(float z) {
    // exp2 overflows to infinity below z = -88 and its reciprocal is then 0
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.442695040888963f * z));
}

// act(z): silu z s(z); gelu 0.5 z (1 + tanh v) = z s(2 v), v = c (z + 0.044715 z^3)
template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    return z * sigmoid(ACT == SILU ? z : 1.5957691216057308f * (z + 0.044715f * z * z * z));
}
// act and its derivative: s + z s (1 - s) q'
template <int ACT>
__device__ __forceinline__ void act_both(float z, float& val, float& slope) {
    if constexpr (ACT == SILU) {
        const float s = sigmoid(z);
        val = z * s;
        slope = s + val * (1.f - s);
    } else {
        const float zz = z * z, s = sigmoid(1.5957691216057308f * (z + 0.044715f * zz * z));
        val = z * s;
        // past |z| = 2^20 the second term is 0 (s is 0 or 1), and q' would overflow
        const float dq = 1.5957691216057308f * (1.f + 0.134145f * zz);
        slope = __builtin_fabsf(z) > 1048576.f ? s : s + val * (1.f - s) * dq;
    }
}
// f(constant act): the choice is made once, outside a tile's loop over its values
template <class F>
__device__ __forceinline__ void with_act(int act, const F& f) {
    if (act == SILU)
        f(std::integral_constant<int, SILU>{});
    else
        f(std::integral_constant<int, GELU>{});
}

// fp8 operands' scales: one per token, one per weight row.  A sum takes one
// after the other: their product may be outside fp32's range where the value
// is not.
struct Scales {
    const float *x, *gate, *up;
};

// h tile of BM rows and BN / 2 columns; gate and up may be null.  The B stage
// holds half its rows from each weight, so g and u of a value are two
// accumulators of one lane and act(g) u needs no exchange.
template <class C>
__global__ void __launch_bounds__(kThreads) gated_up_kernel(const void* xp, const void* wg, const void* wu, Scales sc,
                                                            uint16_t* gate, uint16_t* up, uint16_t* h, int m, int d,
                                                            int f, int act, int tiles_m, int tiles_n) {
    constexpr int E = C::FP8 ? 1 : 2;  // bytes per value
    DENSE_LDS(C, ring);
    Ctx<C> x = make_ctx<C>(ring);
    int tm, tn;
    order::coords(order::xcd_list(blockIdx.x, gridDim.x, tiles_m * tiles_n).first, tiles_m, tiles_n, tm, tn);
    const int m0 = tm * C::BM, n0 = tn * C::HALF;
    const int wm = x.w >> 1, wn = x.w & 1;
    x.KT = (d * E + 127) / 128;
    x.la.init(Mat{xp, (int64_t)d * E, m}, m0, d * E, x.w, x.lane);
    // waves 0 and 1 load the gate half of a B stage, 2 and 3 the up half
    x.lb.init(Mat{wm ? wu : wg, (int64_t)d * E, f}, n0, d * E, x.w, x.lane, C::HALF, wn);
    x.ra.init(wm * (C::BM / 2), x.lane);
    x.rb.init(wn * (C::HALF / 2), x.lane);
    run(x);
    const Rows oh(h, m0, C::BM, m, f), og(gate, m0, C::BM, m, f), ou(up, m0, C::BM, m, f);
    with_act(act, [&](auto a) __attribute__((always_inline)) {
#pragma unroll
        for (int mb = 0; mb < C::MB; ++mb) {
            claim(x.acc[mb]);
            const int row = wm * (C::BM / 2) + 16 * mb + (x.lane & 15);
#pragma unroll
            for (int nb = 0; nb < C::NB / 2; nb += 2) {
                const int col = n0 + wn * (C::HALF / 2) + 16 * nb + pair_column(x.lane);
                float g[8], u[8], v[8];
                pair_columns(x.acc[mb][nb], x.acc[mb][nb + 1], g);
                pair_columns(x.acc[mb][C::NB / 2 + nb], x.acc[mb][C::NB / 2 + nb + 1], u);
                if constexpr (C::FP8) {
                    const float sx = m0 + row < m ? sc.x[m0 + row] : 0.f;
#pragma unroll
                    for (int t = 0; t < 8; ++t) {
                        g[t] = g[t] * sx * (col < f ? sc.gate[col + t] : 0.f);
                        u[t] = u[t] * sx * (col < f ? sc.up[col + t] : 0.f);
                    }
                }
#pragma unroll
                for (int t = 0; t < 8; ++t) v[t] = act_value<a>(g[t]) * u[t];
                oh.store(row, col, pack8(v));
                if (gate) {
                    og.template store<kStream>(row, col, pack8(g));
                    ou.template store<kStream>(row, col, pack8(u));
                }
            }
        }
    });
}

// What follows the products of a plain tile.
enum Out { STORE, GATE_GRAD };

struct GateGrad {
    const uint16_t *gate, *up;
    uint16_t *dgate, *dup, *h;
    int act;
};

template <class C, Out O>
__device__ __forceinline__ void finish(Ctx<C>& x, uint16_t* c, const GateGrad& gg, int m0, int m, int n0, int n) {
    const int wm = x.w >> 1, wn = x.w & 1;
    const int row0 = wm * (C::BM / 2) + (x.lane & 15), col0 = n0 + wn * (C::BN / 2) + pair_column(x.lane);
    const Rows oc(O == STORE ? c : gg.dgate, m0, C::BM, m, n);
    if constexpr (O == STORE) {
#pragma unroll
        for (int mb = 0; mb < C::MB; ++mb) {
            claim(x.acc[mb]);
#pragma unroll
            for (int nb = 0; nb < C::NB; nb += 2) {
                float v[8];
                pair_columns(x.acc[mb][nb], x.acc[mb][nb + 1], v);
                oc.template store<kStream>(row0 + 16 * mb, col0 + 16 * nb, pack8(v));
            }
        }
    } else {
        const Rows ou(gg.dup, m0, C::BM, m, n), oh(gg.h, m0, C::BM, m, n);
        const Rows ig(gg.gate, m0, C::BM, m, n), iu(gg.up, m0, C::BM, m, n);
        // the next row block's gate and up are loaded before this one's are used
        v4i gq[2][C::NB / 2], uq[2][C::NB / 2];
        const auto load = [&](int mb) __attribute__((always_inline)) {
#pragma unroll
            for (int q = 0; q < C::NB / 2; ++q) {
                gq[mb & 1][q] = ig.load(row0 + 16 * mb, col0 + 32 * q);
                uq[mb & 1][q] = iu.load(row0 + 16 * mb, col0 + 32 * q);
            }
        };
        load(0);
        with_act(gg.act, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
            for (int mb = 0; mb < C::MB; ++mb) {
                if (mb + 1 < C::MB) load(mb + 1);
                claim(x.acc[mb]);
#pragma unroll
                for (int q = 0; q < C::NB / 2; ++q) {
                    float v[8], g[8], u[8], a[8];
                    pair_columns(x.acc[mb][2 * q], x.acc[mb][2 * q + 1], v);
                    unpack8(gq[mb & 1][q], g);
                    unpack8(uq[mb & 1][q], u);
#pragma unroll
                    for (int t = 0; t < 8; ++t) {
                        float val, slope;
                        act_both<act>(g[t], val, slope);
                        a[t] = val * u[t];           // h
                        g[t] = v[t] * u[t] * slope;  // dg
                        u[t] = v[t] * val;           // du
                    }
                    oc.store(row0 + 16 * mb, col0 + 32 * q, pack8(g));
                    ou.store(row0 + 16 * mb, col0 + 32 * q, pack8(u));
                    oh.store(row0 + 16 * mb, col0 + 32 * q, pack8(a));
                }
            }
        });
    }
}

// c = a b over K values: a [m, k] KC, b [n, k] KC or [k, n] KR, and with SEG
// c = a b + a2 b2 of the same shapes.
struct Product {
    const uint16_t *a, *a2, *b, *b2;
    uint16_t* c;
    int m, n, k, tiles_m, tiles_n;
};

// tile: the tile's place in the order.
template <class C, Out O>
__device__ __forceinline__ void product_body(const Ring& ring, const Product& p, const GateGrad& gg, int tile) {
    Ctx<C> x = make_ctx<C>(ring);
    int tm, tn;
    order::coords(tile, p.tiles_m, p.tiles_n, tm, tn);
    const int m0 = tm * C::BM, n0 = tn * C::BN;
    x.KT = (C::SEG ? 2 : 1) * ((p.k + 63) / 64);
    x.la.init(Mat{p.a, (int64_t)p.k * 2, p.m}, m0, p.k * 2, x.w, x.lane, C::BM, -1, p.a2);
    if constexpr (C::LB == KC)
        x.lb.init(Mat{p.b, (int64_t)p.k * 2, p.n}, n0, p.k * 2, x.w, x.lane, C::BN, -1, p.b2);
    else
        x.lb.init(Mat{p.b, (int64_t)p.n * 2, p.n}, n0, p.k, x.w, x.lane, C::BN, -1, p.b2);
    x.ra.init((x.w >> 1) * (C::BM / 2), x.lane);
    x.rb.init((x.w & 1) * (C::BN / 2), x.lane);
    run(x);
    finish<C, O>(x, p.c, gg, m0, p.m, n0, p.n);
}

template <class C, Out O>
__global__ void __launch_bounds__(kThreads) product_kernel(Product p, GateGrad gg) {
    DENSE_LDS(C, ring);
    product_body<C, O>(ring, p, gg, order::xcd_list(blockIdx.x, gridDim.x, p.tiles_m * p.tiles_n).first);
}

// The three weight gradients, sums over the m tokens: dWg = dg^T x and
// dWu = du^T x [f, d], dWd = dy^T h [d, f], one launch.
struct Grads {
    const uint16_t *dgate, *dup, *x, *dy, *h;
    uint16_t *dwg, *dwu, *dwd;
};

template <class C>
__device__ __forceinline__ void weight_grad_body(const Ring& ring, const Grads& p, int m, int d, int f, int td, int tf,
                                                 int t) {
    Ctx<C> x = make_ctx<C>(ring);
    const int per = td * tf, which = t / per;
    t -= which * per;
    const bool down = which == 2;
    const int rows = down ? d : f, cols = down ? f : d;
    int tm, tn;
    order::coords(t, down ? td : tf, down ? tf : td, tm, tn);
    const int m0 = tm * C::BM, n0 = tn * C::BN;
    x.KT = (m + 63) / 64;
    x.la.init(Mat{down ? p.dy : which ? p.dup : p.dgate, (int64_t)rows * 2, rows}, m0, m, x.w, x.lane);
    x.lb.init(Mat{down ? p.h : p.x, (int64_t)cols * 2, cols}, n0, m, x.w, x.lane);
    x.ra.init((x.w >> 1) * (C::BM / 2), x.lane);
    x.rb.init((x.w & 1) * (C::BN / 2), x.lane);
    run(x);
    finish<C, STORE>(x, down ? p.dwd : which ? p.dwu : p.dwg, GateGrad{}, m0, rows, n0, cols);
}

template <class C>
__global__ void __launch_bounds__(kThreads) weight_grad_kernel(Grads p, int m, int d, int f, int td, int tf) {
    DENSE_LDS(C, ring);
    weight_grad_body<C>(ring, p, m, d, f, td, tf, order::xcd_list(blockIdx.x, gridDim.x, 3 * td * tf).first);
}

// dx and the weights' gradients in one launch of 64 x 64 tiles, where that is
// no slower than each in its own shape: neither needs the other, and each
// alone leaves units idle at its end.
template <class CX, class CW>
__global__ void __launch_bounds__(kThreads) input_and_weight_grad_kernel(Product px, Grads p, int m, int d, int f, int td,
                                                                         int tf) {
    static_assert(CX::SA == CW::SA && CX::SB == CW::SB && CX::NS == CW::NS, "one set of stages for both");
    DENSE_LDS(CX, ring);
    const int first = px.tiles_m * px.tiles_n;
    if ((int)blockIdx.x < first)
        product_body<CX, STORE>(ring, px, GateGrad{}, order::xcd_list(blockIdx.x, first, first).first);
    else
        weight_grad_body<CW>(ring, p, m, d, f, td, tf, order::xcd_list(blockIdx.x - first, 3 * td * tf, 3 * td * tf).first);
}

// At most 16 tokens: eight columns of h per workgroup, whose 16 weight rows are
// the eight gate rows and the eight up rows.
template <bool FP8, int WAVES>
__global__ void __launch_bounds__(64 * WAVES) thin_up_kernel(const char* xp, const char* wg, const char* wu, Scales sc,
                                                             uint16_t* gate, uint16_t* up, uint16_t* h, int m, int d,
                                                             int f, int act) {
    __shared__ thin::Join<1, WAVES> join;
    const int i = lane_id() & 15, n0 = blockIdx.x * 8, kb = FP8 ? d : 2 * d;
    const char* xrow[1] = {xp + (int64_t)(i < m ? i : m - 1) * kb};
    v4f acc[1];
    thin::product<FP8, 1, WAVES>((i < 8 ? wg : wu) + (int64_t)(n0 + (i & 7)) * kb, xrow, kb, acc);
    join.put(acc);
    for (int e = threadIdx.x; e < 8 * m; e += 64 * WAVES) {
        const int r = e >> 3, c = e & 7;
        float g = join.sum(r, c), u = join.sum(r, 8 + c);
        if constexpr (FP8) {
            g = g * sc.x[r] * sc.gate[n0 + c];
            u = u * sc.x[r] * sc.up[n0 + c];
        }
        const int64_t at = (int64_t)r * f + n0 + c;
        h[at] = thin::to_bf16((act == SILU ? act_value<SILU>(g) : act_value<GELU>(g)) * u);
        if (gate) {
            gate[at] = thin::to_bf16(g);
            up[at] = thin::to_bf16(u);
        }
    }
}

// y [m, n] = a [m, k] b [n, k]^T for at most 16 rows of a: 16 columns per
// workgroup.
template <int WAVES>
__global__ void __launch_bounds__(64 * WAVES) thin_product_kernel(const uint16_t* a, const uint16_t* b, uint16_t* y,
                                                                  int m, int n, int k) {
    __shared__ thin::Join<1, WAVES> join;
    const int i = lane_id() & 15, n0 = blockIdx.x * 16;
    const char* xrow[1] = {(const char*)(a + (int64_t)(i < m ? i : m - 1) * k)};
    v4f acc[1];
    thin::product<false, 1, WAVES>((const char*)(b + (int64_t)(n0 + i < n ? n0 + i : n - 1) * k), xrow, k * 2, acc);
    join.put(acc);
    for (int e = threadIdx.x; e < 16 * m; e += 64 * WAVES) {
        const int r = e >> 4, c = e & 15;
        if (n0 + c < n) y[(int64_t)r * n + n0 + c] = thin::to_bf16(join.sum(r, c));
    }
}

// h (and gate, up) from the shares of the two projections: eight columns a thread.
template <bool FP8>
__global__ void __launch_bounds__(256) join_up_kernel(const float* part, int shares, Scales sc, uint16_t* gate,
                                                      uint16_t* up, uint16_t* h, int m, int f, int act) {
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
    if (at >= (int64_t)m * f) return;
    const int64_t row = at / f, col = at - row * f, from = row * 2 * f + col, stride = (int64_t)m * 2 * f;
    float g[8], u[8], v[8];
    split::sum8(part, shares, stride, from, g);
    split::sum8(part, shares, stride, from + f, u);
    if constexpr (FP8) {
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            g[t] = g[t] * sc.x[row] * sc.gate[col + t];
            u[t] = u[t] * sc.x[row] * sc.up[col + t];
        }
    }
    with_act(act, [&](auto a) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < 8; ++t) v[t] = act_value<a>(g[t]) * u[t];
    });
    *(v4i*)(h + at) = pack8(v);
    if (gate) {
        *(v4i*)(gate + at) = pack8(g);
        *(v4i*)(up + at) = pack8(u);
    }
}

// y from the shares of a product.
__global__ void __launch_bounds__(256) join_kernel(const float* part, int shares, uint16_t* y, int64_t values) {
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
    if (at >= values) return;
    float v[8];
    split::sum8(part, shares, values, at, v);
    *(v4i*)(y + at) = pack8(v);
}

// dgate, dup and h from the shares of dh.
__global__ void __launch_bounds__(256) join_gate_grad_kernel(const float* part, int shares, GateGrad gg, int64_t values) {
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
    if (at >= values) return;
    float v[8], g[8], u[8], a[8];
    unpack8(*(const v4i*)(gg.gate + at), g);
    unpack8(*(const v4i*)(gg.up + at), u);
    split::sum8(part, shares, values, at, v);
    with_act(gg.act, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            float val, slope;
            act_both<act>(g[t], val, slope);
            a[t] = val * u[t];
            g[t] = v[t] * u[t] * slope;
            u[t] = v[t] * val;
        }
    });
    *(v4i*)(gg.dgate + at) = pack8(g);
    *(v4i*)(gg.dup + at) = pack8(u);
    *(v4i*)(gg.h + at) = pack8(a);
}

static unsigned join_blocks(int64_t values) { return (unsigned)ceil_div(values, 2048); }

template <bool FP8, int WAVES>
static hipError_t launch_thin_up_any(const void* x, const void* wg, const void* wu, const Scales& sc, uint16_t* gate,
                                     uint16_t* up, uint16_t* h, int m, int d, int f, int act, hipStream_t st) {
    hipLaunchKernelGGL((thin_up_kernel<FP8, WAVES>), dim3(f / 8), dim3(64 * WAVES), 0, st, (const char*)x,
                       (const char*)wg, (const char*)wu, sc, gate, up, h, m, d, f, act);
    return hipGetLastError();
}
template <int WAVES, class... A>
static hipError_t launch_thin_up(A... a) {
    return launch_thin_up_any<false, WAVES>(a...);
}
template <int WAVES, class... A>
static hipError_t launch_thin_up_fp8(A... a) {
    return launch_thin_up_any<true, WAVES>(a...);
}
template <class C>
static hipError_t launch_up_as(const void* x, const void* wg, const void* wu, const Scales& sc, uint16_t* gate,
                               uint16_t* up, uint16_t* h, int m, int d, int f, int act, hipStream_t st) {
    const int tm = (int)ceil_div(m, C::BM), tn = (int)ceil_div(f, C::HALF);
    hipLaunchKernelGGL((gated_up_kernel<C>), dim3(tm * tn), dim3(kThreads), 0, st, x, wg, wu, sc, gate, up, h, m, d, f,
                       act, tm, tn);
    return hipGetLastError();
}

template <bool FP8>
static hipError_t launch_up(const void* x, const void* wg, const void* wu, const Scales& sc, uint16_t* gate,
                            uint16_t* up, uint16_t* h, float* part, int m, int d, int f, int act, hipStream_t st) {
    constexpr int E = FP8 ? 1 : 2;
    constexpr int S = FP8 ? 2 : 4;  // the fp8 steps alternate two fragment sets, so two stages
    using C64 = Cfg<64, 128, S, KC, KC, true, false, FP8>;
    const Choice c = up_choice(m, d, f, E);
    switch (c.tile) {
        case kThin:
            if constexpr (FP8)
                return THIN_BY_SIZE(launch_thin_up_fp8, d * E, x, wg, wu, sc, gate, up, h, m, d, f, act, st);
            else
                return THIN_BY_SIZE(launch_thin_up, d * E, x, wg, wu, sc, gate, up, h, m, d, f, act, st);
        case kSplit: {
            const hipError_t e = split::launch_partial<C64>({{x, x}, {wg, wu}, part, m, f, d * E, c.plan, 0, 0}, st);
            if (e != hipSuccess) return e;
            hipLaunchKernelGGL((join_up_kernel<FP8>), dim3(join_blocks((int64_t)m * f)), dim3(256), 0, st, part,
                               c.plan.shares, sc, gate, up, h, m, f, act);
            return hipGetLastError();
        }
        case kTile256:
            return launch_up_as<Cfg<256, 256, 2, KC, KC, true, false, FP8>>(x, wg, wu, sc, gate, up, h, m, d, f, act, st);
        case kTile128:
            return launch_up_as<Cfg<128, 128, 2, KC, KC, true, false, FP8>>(x, wg, wu, sc, gate, up, h, m, d, f, act, st);
        case kTile128D:
            return launch_up_as<Cfg<128, 128, S, KC, KC, true, false, FP8>>(x, wg, wu, sc, gate, up, h, m, d, f, act, st);
        default: return launch_up_as<C64>(x, wg, wu, sc, gate, up, h, m, d, f, act, st);
    }
}

template <class C>
static Product product_of(const uint16_t* a, const uint16_t* a2, const uint16_t* b, const uint16_t* b2, uint16_t* c,
                          int m, int n, int k) {
    return Product{a, a2, b, b2, c, m, n, k, (int)ceil_div(m, C::BM), (int)ceil_div(n, C::BN)};
}

template <class C, Out O>
static hipError_t launch_product_as(const uint16_t* a, const uint16_t* a2, const uint16_t* b, const uint16_t* b2,
                                    uint16_t* c, const GateGrad& gg, int m, int n, int k, hipStream_t st) {
    const Product p = product_of<C>(a, a2, b, b2, c, m, n, k);
    hipLaunchKernelGGL((product_kernel<C, O>), dim3(p.tiles_m * p.tiles_n), dim3(kThreads), 0, st, p, gg);
    return hipGetLastError();
}

template <Lay LB, bool SEG, Out O>
static hipError_t launch_product(const uint16_t* a, const uint16_t* a2, const uint16_t* b, const uint16_t* b2,
                                 uint16_t* c, const GateGrad& gg, float* part, int m, int n, int k, hipStream_t st) {
    const Choice ch = product_choice(m, n, k, SEG);
    switch (ch.tile) {
        case kSplit: {
            const hipError_t e =
                split::launch_partial<Cfg<64, 64, 4, KC, LB>>({{a, a2}, {b, b2}, part, m, n, 2 * k, ch.plan, 0, 0}, st);
            if (e != hipSuccess) return e;
            const int64_t values = (int64_t)m * n;
            if constexpr (O == STORE)
                hipLaunchKernelGGL(join_kernel, dim3(join_blocks(values)), dim3(256), 0, st, part, ch.plan.shares, c, values);
            else
                hipLaunchKernelGGL(join_gate_grad_kernel, dim3(join_blocks(values)), dim3(256), 0, st, part,
                                   ch.plan.shares, gg, values);
            return hipGetLastError();
        }
        case kTile256: return launch_product_as<Cfg<256, 256, 2, KC, LB, false, SEG>, O>(a, a2, b, b2, c, gg, m, n, k, st);
        case kTile128: return launch_product_as<Cfg<128, 128, 2, KC, LB, false, SEG>, O>(a, a2, b, b2, c, gg, m, n, k, st);
        case kTile128D: return launch_product_as<Cfg<128, 128, 4, KC, LB, false, SEG>, O>(a, a2, b, b2, c, gg, m, n, k, st);
        default: return launch_product_as<Cfg<64, 64, 4, KC, LB, false, SEG>, O>(a, a2, b, b2, c, gg, m, n, k, st);
    }
}

template <class C>
static hipError_t launch_grads_as(const Grads& p, int m, int d, int f, hipStream_t st) {
    const int td = (int)ceil_div(d, C::BM), tf = (int)ceil_div(f, C::BM);
    hipLaunchKernelGGL((weight_grad_kernel<C>), dim3(3 * td * tf), dim3(kThreads), 0, st, p, m, d, f, td, tf);
    return hipGetLastError();
}

static hipError_t launch_grads(const Grads& p, int m, int d, int f, hipStream_t st) {
    switch (grads_choice(m, d, f)) {
        case kTile256: return launch_grads_as<Cfg<256, 256, 2, KR, KR>>(p, m, d, f, st);
        case kTile128: return launch_grads_as<Cfg<128, 128, 2, KR, KR>>(p, m, d, f, st);
        case kTile128D: return launch_grads_as<Cfg<128, 128, 4, KR, KR>>(p, m, d, f, st);
        default: return launch_grads_as<Cfg<64, 64, 4, KR, KR>>(p, m, d, f, st);
    }
}

// dx = dgate w_gate + dup w_up and the weights' gradients.
static hipError_t launch_input_and_grads(const Grads& p, const uint16_t* wg, const uint16_t* wu, uint16_t* dx,
                                         float* part, int m, int d, int f, hipStream_t st) {
    if (grads_with_dx(m, d, f)) {
        using CX = Cfg<64, 64, 4, KC, KR, false, true>;
        using CW = Cfg<64, 64, 4, KR, KR>;
        const Product px = product_of<CX>(p.dgate, p.dup, wg, wu, dx, m, d, f);
        const int td = (int)ceil_div(d, CW::BM), tf = (int)ceil_div(f, CW::BM);
        hipLaunchKernelGGL((input_and_weight_grad_kernel<CX, CW>), dim3(px.tiles_m * px.tiles_n + 3 * td * tf),
                           dim3(kThreads), 0, st, px, p, m, d, f, td, tf);
        return hipGetLastError();
    }
    const hipError_t e =
        launch_product<KR, true, STORE>(p.dgate, p.dup, wg, wu, dx, GateGrad{}, part, m, d, f, st);
    return e != hipSuccess ? e : launch_grads(p, m, d, f, st);
}

template <int WAVES>
static hipError_t launch_thin_product(const uint16_t* a, const uint16_t* b, uint16_t* y, int m, int n, int k,
                                      hipStream_t st) {
    hipLaunchKernelGGL((thin_product_kernel<WAVES>), dim3((n + 15) / 16), dim3(64 * WAVES), 0, st, a, b, y, m, n,
                       k);
    return hipGetLastError();
}
}  // namespace ffn

using namespace ffn;

// Workspaces: the bf16 intermediates in front, then the shares of whichever
// split product is largest (its products run one after the other).
static int64_t front_bytes(int64_t arrays, int64_t m, int64_t f) { return (arrays * m * f * 2 + 255) / 256 * 256; }

int64_t gated_up_a8w8_shares_bytes(int m, int d, int f) { return split::bytes(up_choice(m, d, f, 1).plan, m, f, true); }

int64_t gated_ffn_workspace_bytes(int m, int d, int f) {
    const int64_t down = m <= kThinMost ? 0 : split::bytes(product_choice(m, d, f, false).plan, m, d, false);
    return front_bytes(1, m, f) + larger(split::bytes(up_choice(m, d, f, 2).plan, m, f, true), down);
}

int64_t gated_ffn_backward_workspace_bytes(int m, int d, int f) {
    return front_bytes(3, m, f) + larger(split::bytes(product_choice(m, f, d, false).plan, m, f, false),
                                         split::bytes(product_choice(m, d, f, true).plan, m, d, false));
}

hipError_t launch_gated_ffn(const uint16_t* x, const uint16_t* wg, const uint16_t* wu, const uint16_t* wd,
                            uint16_t* gate, uint16_t* up, void* ws, uint16_t* y, int m, int d, int f, int act,
                            hipStream_t st) {
    uint16_t* h = (uint16_t*)ws;
    float* part = (float*)((char*)ws + front_bytes(1, m, f));
    const hipError_t e = launch_up<false>(x, wg, wu, Scales{}, gate, up, h, part, m, d, f, act, st);
    if (e != hipSuccess) return e;
    if (m <= kThinMost) return THIN_BY_SIZE(launch_thin_product, f * 2, h, wd, y, m, d, f, st);
    return launch_product<KC, false, STORE>(h, nullptr, wd, nullptr, y, GateGrad{}, part, m, d, f, st);
}

hipError_t launch_gated_up_a8w8(const uint8_t* x, const uint8_t* wg, const uint8_t* wu, const float* sx, const float* sg,
                                const float* su, uint16_t* h, void* ws, int m, int d, int f, int act, hipStream_t st) {
    return launch_up<true>(x, wg, wu, Scales{sx, sg, su}, nullptr, nullptr, h, (float*)ws, m, d, f, act, st);
}

hipError_t launch_gated_ffn_backward(const uint16_t* dy, const uint16_t* x, const uint16_t* wg, const uint16_t* wu,
                                     const uint16_t* wd, const uint16_t* gate, const uint16_t* up, void* ws,
                                     uint16_t* dx, uint16_t* dwg, uint16_t* dwu, uint16_t* dwd, int m, int d, int f,
                                     int act, hipStream_t st) {
    const int64_t one = (int64_t)m * f;
    uint16_t *dgate = (uint16_t*)ws, *dup = dgate + one, *h = dup + one;
    float* part = (float*)((char*)ws + front_bytes(3, m, f));
    const Grads p{dgate, dup, x, dy, h, dwg, dwu, dwd};
    if (m == 0) return launch_grads(p, m, d, f, st);
    const GateGrad gg{gate, up, dgate, dup, h, act};
    const hipError_t e = launch_product<KR, false, GATE_GRAD>(dy, nullptr, wd, nullptr, nullptr, gg, part, m, f, d, st);
    return e != hipSuccess ? e : launch_input_and_grads(p, wg, wu, dx, part, m, d, f, st);
}

}  // namespace dmm
