// dense_core.h -- the tile engine of the feed-forward and adapter kernels
// (gfx950): a BM x BN output tile per 256-thread workgroup, 2 x 2 waves, both
// operands streamed global -> LDS by direct-to-LDS loads, fp32 accumulators.
//
// Operand layouts.  The A operand gives the output's rows, the B operand its
// columns; each is stored either with K contiguous (KC: [rows, K]) or with
// one line of all rows per K value (KR: [K, rows]), so the three products of
// a projection and its gradients (x W^T, dy W, dy^T x) run without a
// transposed copy of anything.
//
// K tiles are 128 bytes of K wide (64 bf16, 128 fp8 codes); dense_layout.h has
// where a K tile's values lie in LDS and why.
//
// Pipeline (NS stages, D(j) the DMAs of K tile j, R(j, h) the fragment reads
// of its k half h):
//   prologue: D(0) .. D(NS-1); wait for D(0); barrier; R(0, 0)
//   step kt : R(kt, 1) under the first quarter of its matrix ops;
//             wait: D(kt+1) landed, own reads of stage kt % NS retired; barrier;
//             D(kt + NS) into stage kt % NS under the ops that follow;
//             R(kt+1, 0) once half 0's ops are done.
// A K tile is loaded about NS - 1/4 steps ahead of its first matrix op and
// there is one barrier per step.  K tiles past the end go through empty descriptors:
// they read as zero and still count, so every wait is a constant.
//
// Bounds.  Every descriptor starts at the tile's own first row (KC) or at the
// K tile's first line (KR), in 64-bit arithmetic, and ends where the tile's
// rows or the operand end; rows, columns and K values past the operand read
// as zero.  So operands may exceed 2^31 bytes; one line times 256 may not.
#pragma once
#include "common.h"
#include "dense_layout.h"
#include "kpipe.h"
#include "tile_order.h"

#include <utility>

namespace dmm {
namespace dense {

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf4 __attribute__((ext_vector_type(4)));

enum Lay { KC, KR };

constexpr int kThreads = 256;
constexpr int kOob = (int)0x80000000;  // a byte offset past every descriptor

__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ const char* uni_ptr(const char* p) {
    const uint64_t v = (uint64_t)p;
    return (const char*)(((uint64_t)(uint32_t)uni((int)(v >> 32)) << 32) | (uint32_t)uni((int)v));
}

// A matrix as an operand: `rows` is its extent along the output, kbytes the
// K extent in bytes (KC) or kcount lines (KR), ld the bytes of one line.
struct Mat {
    const void* p;
    int64_t ld;
    int rows;
};

// The share of one wave in the DMAs of one operand's stages.  SEG: K runs over
// two matrices of one shape, one after the other.
template <Lay L, int ROWS, bool SEG, bool GATHER = false>
struct Loader {
    static constexpr int NL = ROWS / 32;        // 1 KiB DMAs per wave per stage
    static constexpr int STEP = L == KC ? 128 : 64;  // K tile: bytes (KC), lines (KR)
    int64_t ld;         // bytes of a line
    const char* cur;    // next K tile; KC: at the tile's first row, KR: K line at the tile's first column
    const char* other;  // SEG: the second matrix's first K tile, null once it is current
    int left, kext;     // what is left of, and all of, a matrix's K: bytes (KC), lines (KR)
    int nrec;           // KC: bytes of the tile's rows; KR: bytes of a line from the tile's column on
    // Byte offsets of this lane's 16 bytes from cur.  KC: of DMAs 0 and 1, DMA j
    // being j & 1's plus (j / 2) rows16 (the swizzle repeats every 16 rows; rows
    // past the operand's last fall past nrec by themselves).
    // GATHER: each DMA's rows come from anywhere, so each has its own.
    static_assert(!GATHER || L == KC, "only rows with K contiguous are gathered");
    static constexpr int NO = L == KC && !GATHER ? 2 : NL;
    int voff[NO];
    int rows16;  // KC: bytes of 16 rows
    int ch[2];   // KC: byte position in the K tile of the chunks of even / odd DMAs

    // Rows [row0, ...) of m, whose K extent is kextent bytes (KC) or lines (KR).
    // wslot: the wave's place among those that load from m, where a stage is
    // stacked from two matrices of rows_here rows.
    __device__ __forceinline__ void init(const Mat& m, int row0, int kextent, int w, int lane, int rows_here = ROWS,
                                         int wslot = -1, const void* second = nullptr) {
        ld = m.ld;
        left = kext = kextent;
        const int ws = wslot < 0 ? w : wslot;
        int rows = m.rows - row0;
        rows = rows < 0 ? 0 : rows > rows_here ? rows_here : rows;
        const int64_t skip = L == KC ? (int64_t)row0 * ld : 2 * (int64_t)row0;
        cur = uni_ptr((const char*)m.p + skip);
        other = SEG ? uni_ptr((const char*)second + skip) : nullptr;
        if constexpr (L == KC) {
            nrec = uni((int)(rows * ld));
            static_assert(NL % 2 == 0, "DMAs in pairs of 16 rows");
            rows16 = uni((int)(16 * ld));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int byte = (NL * w + j) * 1024 + 16 * lane;  // where the DMA writes
                const int r = kc_row(byte) - 8 * NL * (w - ws);    // the matrix row it holds
                ch[j] = kc_chunk(byte) * 16;
                voff[j] = (int)(r * ld) + ch[j];
            }
        } else {
            nrec = uni(2 * rows);
#pragma unroll
            for (int j = 0; j < NL; ++j) {
                const int byte = (NL * w + j) * 1024 + 16 * lane;
                const int col = kr_col(byte, ROWS);
                voff[j] = col < rows ? (int)(kr_k(byte, ROWS) * ld) + 2 * col : kOob;
            }
            rows16 = ch[0] = ch[1] = 0;
        }
    }

    // After init of a KC operand whose rows are all of a span: line q of the
    // tile takes row row(q) of it.  A row past the span's end reads as zero.
    template <class F>
    __device__ __forceinline__ void gather(int w, F row) {
        static_assert(GATHER, "rows are consecutive");
#pragma unroll
        for (int j = 0; j < NL; ++j)
            voff[j] = row(kc_row((NL * w + j) * 1024 + 16 * lane_id())) * (int)ld + ch[j & 1];
    }

    // Only K tiles [first, first + count) of the matrix.
    __device__ __forceinline__ void range(int first, int count) {
        cur += (int64_t)first * STEP * (L == KC ? 1 : ld);
        left -= first * STEP;
        left = left > count * STEP ? count * STEP : left;
    }

    // The next K tile's descriptor and offsets.  Past the last K value nothing
    // is left and every offset is out of range; no branch in here.
    struct Tile {
        __amdgpu_buffer_rsrc_t r;
        int at[2];
    };
    __device__ __forceinline__ void turn() {
        if constexpr (SEG) {
            const bool go = left <= 0 && other != nullptr;
            cur = go ? other : cur;
            left = go ? kext : left;
            other = go ? nullptr : other;
        }
    }
    __device__ __forceinline__ Tile next() {
        Tile t;
        if constexpr (L == KC) {
            t.r = make_rsrc(cur, (uint32_t)nrec);
#pragma unroll
            for (int e = 0; e < 2; ++e) t.at[e] = ch[e] < left ? GATHER ? 0 : voff[e] : kOob;
            cur += STEP;
        } else {
            const int lines = left < STEP ? left : STEP;
            const int bytes = (lines - 1) * (int)ld + nrec;
            t.r = make_rsrc(cur, lines > 0 && nrec > 0 ? (uint32_t)bytes : 0u);
            t.at[0] = t.at[1] = 0;
            cur += STEP * ld;
        }
        left -= STEP;
        return t;
    }
    __device__ __forceinline__ void issue_one(const Tile& t, lds_char* lds, int j, int w) const {
        // kOob plus a tile's rows stays past every descriptor, and below 2^32
        const int off = GATHER    ? t.at[j & 1] + voff[GATHER ? j : 0]
                        : L == KC ? t.at[j & 1] + (j >> 1) * rows16
                                  : voff[L == KC ? 0 : j];
        lds_dma16(t.r, lds + (NL * w + j) * 1024, off);
    }
};

// Reads of one operand's fragments: NB blocks of 16 rows of this wave.
template <Lay L, int ROWS, int NB>
struct Reader {
    static constexpr int NV = L == KC ? 2 : NB;
    int rd[NV];

    // row0: the wave's first row in the stage, a multiple of 16.  Block q is
    // rows row0 + 16 q, or for the two-matrix tile (HALF > 0) rows
    // row0 + 16 q of the first half and HALF + ... of the second.
    __device__ __forceinline__ void init(int row0, int lane) {
        const int i = lane & 15, g = lane >> 4;
        if constexpr (L == KC) {
#pragma unroll
            for (int h = 0; h < 2; ++h) rd[h] = kc_read(row0, 0, i, g, h);
        } else {
#pragma unroll
            for (int q = 0; q < NB; ++q) rd[q] = kr_read(row0, q, i, g, ROWS);
        }
    }

    template <int H, int HALF>
    __device__ __forceinline__ bf8 read(lds_char* st, int q) const {
        if constexpr (L == KC) {
            typedef __attribute__((address_space(3))) const bf8 lds_bf8;
            const int row = HALF == 0 ? 16 * q : q < NB / 2 ? 16 * q : HALF + 16 * (q - NB / 2);
            return *(lds_bf8*)(st + row * 128 + rd[H]);
        } else {
            static_assert(HALF == 0, "two-matrix tiles have K contiguous");
            typedef __attribute__((address_space(3))) bf4 lds_bf4;
#if defined(__HIP_DEVICE_COMPILE__)
            const bf4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf4*)(st + rd[q] + (32 * H) * (2 * ROWS)));
            const bf4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf4*)(st + rd[q] + (32 * H + 4) * (2 * ROWS)));
#else
            const bf4 lo{}, hi{};
#endif
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }
};

// Everything that shapes a tile: BM x BN, stages, layouts, HALF (> 0: the B
// stage is two stacked matrices of HALF rows each, and a wave owns the same
// columns of both).
template <int BM_, int BN_, int NS_, Lay LA_, Lay LB_, bool GATED_ = false, bool SEG_ = false, bool FP8_ = false,
          bool GATHER_ = false>
struct Cfg {
    static constexpr int BM = BM_, BN = BN_, NS = NS_;
    static constexpr Lay LA = LA_, LB = LB_;
    static constexpr bool GATED = GATED_, SEG = SEG_, FP8 = FP8_, GATHER = GATHER_;
    static_assert(!FP8 || (LA == KC && LB == KC), "fp8 operands have K contiguous");
    static constexpr int HALF = GATED ? BN / 2 : 0;
    static constexpr int SA = BM * 128, SB = BN * 128;  // bytes per stage
    static constexpr int MB = BM / 32, NB = BN / 32;    // 16 x 16 blocks per wave
    static constexpr int NL = (SA + SB) / 4096;         // DMAs per wave per K tile
};

struct Ring {
    lds_char* a[4];
    lds_char* b[4];
};

template <class C>
struct Ctx {
    Ring lds;
    Loader<C::LA, C::BM, C::SEG, C::GATHER> la;
    Loader<C::LB, C::BN, C::SEG> lb;
    Reader<C::LA, C::BM, C::MB> ra;
    Reader<C::LB, C::BN, C::NB> rb;
    int KT, w, lane;  // K tiles
    v4f acc[C::MB][C::NB];
};

template <class C>
struct Frags {
    bf8 a[C::MB], b[C::NB];
};

// Fragment u of stage S, k half H: the B blocks, then the A blocks.
template <class C, int S, int H>
__device__ __forceinline__ void read_one(const Ctx<C>& x, Frags<C>& f, int u) {
    if (u < C::NB)
        f.b[u] = x.rb.template read<H, C::HALF>(x.lds.b[S], u);
    else
        f.a[u - C::NB] = x.ra.template read<H, 0>(x.lds.a[S], u - C::NB);
}

// One matrix op.  The accumulator is pinned to the AGPRs and updated in place:
// left to itself the compiler copies accumulators between the two register
// files and spills.  It does not see the op's latency either: what reads an
// accumulator afterwards goes through settle().
__device__ __forceinline__ void mfma(v4f& acc, const bf8& b, const bf8& a) {
#if defined(__HIP_DEVICE_COMPILE__)
    asm("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(b), "v"(a));
#endif
}

// Barrier that no memory operation crosses in the compiler's eyes either.
__device__ __forceinline__ void barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// f(constant 0), ..., f(constant N - 1), each an instance of its own: a step is
// too long for the compiler to unroll as a loop.
template <int N, class F>
__device__ __forceinline__ void each(const F& f) {
    [&]<int... I>(std::integer_sequence<int, I...>) __attribute__((always_inline)) {
        (f(std::integral_constant<int, I>{}), ...);
    }(std::make_integer_sequence<int, N>{});
}

// The next K tile's DMAs into stage DS, one at a time.  Its descriptors are
// worked out in two parts ahead of the first of them.
template <class C, int DS>
struct Feeder {
    static constexpr int NLA = C::BM / 32, N = NLA + C::BN / 32;
    typename Loader<C::LA, C::BM, C::SEG, C::GATHER>::Tile ta;
    typename Loader<C::LB, C::BN, C::SEG>::Tile tb;
    template <int PART>
    __device__ __forceinline__ void prepare(Ctx<C>& x) {
        if constexpr (PART == 0) {
            x.la.turn();
            ta = x.la.next();
        } else {
            x.lb.turn();
            tb = x.lb.next();
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    __device__ __forceinline__ void one(const Ctx<C>& x, int j) const {
        if (j < NLA)
            x.la.issue_one(ta, x.lds.a[DS], j, x.w);
        else
            x.lb.issue_one(tb, x.lds.b[DS], j - NLA, x.w);
    }
};

template <class C>
__device__ __forceinline__ void mid_wait() {
    __builtin_amdgcn_sched_barrier(0);
    wait_vm_lgkm0<sched::bf16_mid_wait(C::NS, C::NL)>();
    barrier();
    __builtin_amdgcn_sched_barrier(0);
}

// The next step (stage S): h0 holds its first k half's fragments on entry, the next
// step's on exit.
template <class C, int S>
__device__ __forceinline__ void step(Ctx<C>& x, Frags<C>& h0) {
    constexpr int MF = C::MB * C::NB, U = C::MB + C::NB, T = 2 * MF;
    using P = Plan<2 * MF, U, U, C::NL>;
    constexpr int R = (S + 1) % C::NS;
    Frags<C> h1;
    Feeder<C, S> feed;
    each<2 * MF>([&](auto op) __attribute__((always_inline)) {
        constexpr int t = op, nb = t % C::NB, mb = (t / C::NB) % C::MB;
        if constexpr (t == P::kMid - T / 16) feed.template prepare<0>(x);
        if constexpr (t == P::kMid - T / 32) feed.template prepare<1>(x);
        if constexpr (t == P::kMid) mid_wait<C>();
        if constexpr (t < MF)
            mfma(x.acc[mb][nb], h0.b[nb], h0.a[mb]);
        else
            mfma(x.acc[mb][nb], h1.b[nb], h1.a[mb]);
#pragma unroll
        for (int u = P::first(t - 1); u < P::first(t); ++u) read_one<C, S, 1>(x, h1, u);
#pragma unroll
        for (int d = P::dma(t - 1); d < P::dma(t); ++d) feed.one(x, d);
        // into the registers of the first half's fragments, which are done with
#pragma unroll
        for (int u = P::template second<MF>(t - 1); u < P::template second<MF>(t); ++u) read_one<C, R, 0>(x, h0, u);
        if constexpr (P::first(t) > P::first(t - 1) || P::dma(t) > P::dma(t - 1) ||
                      P::template second<MF>(t) > P::template second<MF>(t - 1))
            __builtin_amdgcn_sched_barrier(0);
    });
    __builtin_amdgcn_sched_barrier(0);
}

// fp8: one matrix op takes both k halves of a block (128 K values), so a step
// splits by row blocks instead: the upper row blocks while the lower ones'
// fragments are read, then the lower ones; the next K tile's column and upper
// row fragments go to a second set.
struct Wide {
    bf8 h[2];  // chunks g and 4 + g of the row: the same 128 K values, in one order for both operands
};
template <class C>
struct Frags8 {
    Wide a[C::MB / 2], b[C::NB];
};

__device__ __forceinline__ void mfma8(v4f& acc, const Wide& b, const Wide& a) {
#if defined(__HIP_DEVICE_COMPILE__)
    const v8i bb = __builtin_bit_cast(v8i, b), aa = __builtin_bit_cast(v8i, a);
    asm("v_mfma_f32_16x16x128_f8f6f4 %0, %1, %2, %0" : "+a"(acc) : "v"(bb), "v"(aa));
#else
    (void)acc, (void)b, (void)a;
#endif
}

// 16-byte read u of stage S: both halves of the column blocks, then of row
// blocks FIRST, FIRST + 1, ...
template <class C, int S>
__device__ __forceinline__ void read_col8(const Ctx<C>& x, Wide (&b)[C::NB], int u) {
    b[u / 2].h[u % 2] = u % 2 ? x.rb.template read<1, C::HALF>(x.lds.b[S], u / 2)
                              : x.rb.template read<0, C::HALF>(x.lds.b[S], u / 2);
}
template <class C, int S, int FIRST>
__device__ __forceinline__ void read_row8(const Ctx<C>& x, Wide (&a)[C::MB / 2], int u) {
    a[u / 2].h[u % 2] = u % 2 ? x.ra.template read<1, 0>(x.lds.a[S], FIRST + u / 2)
                              : x.ra.template read<0, 0>(x.lds.a[S], FIRST + u / 2);
}

// `now` holds the step's column and upper row fragments, `next` gets the
// following step's.
template <class C, int S>
__device__ __forceinline__ void step8(Ctx<C>& x, Frags8<C>& now, Frags8<C>& next) {
    constexpr int HM = C::MB / 2, MF = HM * C::NB, T = 2 * MF, UA = 2 * HM, UB = 2 * C::NB;
    using P = Plan<2 * MF, UA, UA + UB, C::NL>;
    constexpr int R = (S + 1) % C::NS;
    Wide low[HM];
    Feeder<C, S> feed;
    each<2 * MF>([&](auto op) __attribute__((always_inline)) {
        constexpr int t = op, nb = t % C::NB, mb = (t / C::NB) % HM;
        if constexpr (t == P::kMid - T / 16) feed.template prepare<0>(x);
        if constexpr (t == P::kMid - T / 32) feed.template prepare<1>(x);
        if constexpr (t == P::kMid) mid_wait<C>();
        if constexpr (t < MF)
            mfma8(x.acc[mb][nb], now.b[nb], now.a[mb]);
        else
            mfma8(x.acc[HM + mb][nb], now.b[nb], low[mb]);
#pragma unroll
        for (int u = P::first(t - 1); u < P::first(t); ++u) read_row8<C, S, HM>(x, low, u);
#pragma unroll
        for (int d = P::dma(t - 1); d < P::dma(t); ++d) feed.one(x, d);
#pragma unroll
        for (int u = P::template second<P::kMid>(t - 1); u < P::template second<P::kMid>(t); ++u) {
            if (u < UB)
                read_col8<C, R>(x, next.b, u);
            else
                read_row8<C, R, 0>(x, next.a, u - UB);
        }
        if constexpr (P::first(t) > P::first(t - 1) || P::dma(t) > P::dma(t - 1) ||
                      P::template second<P::kMid>(t) > P::template second<P::kMid>(t - 1))
            __builtin_amdgcn_sched_barrier(0);
    });
    __builtin_amdgcn_sched_barrier(0);
}

// The next K tile into stage S, all at once.
template <class C, int S>
__device__ __forceinline__ void issue(Ctx<C>& x) {
    Feeder<C, S> feed;
    feed.template prepare<0>(x);
    feed.template prepare<1>(x);
#pragma unroll
    for (int j = 0; j < Feeder<C, S>::N; ++j) feed.one(x, j);
}

// A matrix op's result may be read by another instruction 7 wait states after
// the op (11 in fp8), and the op may read an accumulator 2 after another instruction
// wrote it; this ties every accumulator to a point past either.
template <class C>
__device__ __forceinline__ void settle(Ctx<C>& x) {
    asm volatile("s_nop 7\n\ts_nop 7" ::: "memory");
#pragma unroll
    for (int mb = 0; mb < C::MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < C::NB; ++nb) asm volatile("" : "+a"(x.acc[mb][nb]));
}

// The product of the loaders' K tiles.
template <class C>
__device__ __forceinline__ void run(Ctx<C>& x) {
    constexpr int NS = C::NS;
#pragma unroll
    for (int mb = 0; mb < C::MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < C::NB; ++nb) x.acc[mb][nb] = (v4f){0.f, 0.f, 0.f, 0.f};
    settle(x);
    issue<C, 0>(x);
    issue<C, 1>(x);
    if constexpr (NS > 2) issue<C, 2>(x);
    if constexpr (NS > 3) issue<C, 3>(x);
    wait_vm_lgkm0<sched::bf16_prologue_wait(NS, C::NL)>();
    barrier();
    if constexpr (C::FP8) {
        static_assert(NS == 2, "two stages, two fragment sets");
        Frags8<C> f[2];
#pragma unroll
        for (int u = 0; u < 2 * C::NB; ++u) read_col8<C, 0>(x, f[0].b, u);
#pragma unroll
        for (int u = 0; u < C::MB; ++u) read_row8<C, 0, 0>(x, f[0].a, u);
        for (int kt = 0; kt < x.KT; kt += NS) {
            step8<C, 0>(x, f[0], f[1]);
            step8<C, 1>(x, f[1], f[0]);
        }
        settle(x);
        return;
    }
    Frags<C> h0;
#pragma unroll
    for (int u = 0; u < C::MB + C::NB; ++u) read_one<C, 0, 0>(x, h0, u);
    // Whole rounds of the ring: K tiles past the end are zero.  (A step that
    // could be skipped would join its path to the loop's head, and the
    // compiler would wait there, in every round, for the youngest DMAs.)
    for (int kt = 0; kt < x.KT; kt += NS) {
        step<C, 0>(x, h0);
        step<C, 1>(x, h0);
        if constexpr (NS > 2) step<C, 2>(x, h0);
        if constexpr (NS > 3) step<C, 3>(x, h0);
    }
    settle(x);
}

// A kernel's stages: one LDS object per stage and operand, so that the
// compiler's tracking of DMAs into LDS tells the stages apart.
#define DENSE_LDS(C, ring)                                                                                  \
    __shared__ __attribute__((aligned(1024))) char lds_a0[C::SA], lds_a1[C::SA], lds_a2[C::NS > 2 ? C::SA : 16], \
        lds_a3[C::NS > 3 ? C::SA : 16], lds_b0[C::SB], lds_b1[C::SB], lds_b2[C::NS > 2 ? C::SB : 16],       \
        lds_b3[C::NS > 3 ? C::SB : 16];                                                                     \
    const Ring ring{{(lds_char*)lds_a0, (lds_char*)lds_a1, (lds_char*)lds_a2, (lds_char*)lds_a3},           \
                    {(lds_char*)lds_b0, (lds_char*)lds_b1, (lds_char*)lds_b2, (lds_char*)lds_b3}}

template <class C>
__device__ __forceinline__ Ctx<C> make_ctx(const Ring& ring) {
    Ctx<C> x;
    x.lds = ring;
    x.w = wave_id();
    x.lane = lane_id();
    return x;
}

// Keeps a row block's accumulators in their AGPRs up to this point, so that
// an epilogue reads them block by block instead of all at once (which spills).
template <int NB>
__device__ __forceinline__ void claim(v4f (&acc)[NB]) {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) asm volatile("" : "+a"(acc[nb]));
}

// Exchanges the accumulators of two neighbouring column blocks between lane
// groups, so that a lane ends with eight consecutive columns of its row: lane
// (i, g) holds columns 16 (g & 1) + 8 (g >> 1) .. + 7 of the 32-column pair.
__device__ __forceinline__ void pair_columns(const v4f& even, const v4f& odd, float (&out)[8]) {
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        // copied out first: a bit cast of a vector's element lvalue takes element 0
        const float e = even[t], o = odd[t];
        const auto s = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, e),
                                                        __builtin_bit_cast(unsigned, o), false, false);
        out[t] = __builtin_bit_cast(float, (unsigned)s[0]);
        out[4 + t] = __builtin_bit_cast(float, (unsigned)s[1]);
    }
#else
    (void)even, (void)odd, (void)out;
#endif
}
__device__ __forceinline__ int pair_column(int lane) { return 16 * ((lane >> 4) & 1) + 8 * (lane >> 5); }

__device__ __forceinline__ v4i pack8(const float (&v)[8]) {
    return (v4i){pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
}
__device__ __forceinline__ void unpack8(const v4i& p, float (&v)[8]) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        v[2 * t] = __builtin_bit_cast(float, (uint32_t)p[t] << 16);
        v[2 * t + 1] = __builtin_bit_cast(float, (uint32_t)p[t] & 0xffff0000u);
    }
}

// The rows [m0, m0 + 256) of a bf16 [m, n] matrix, for 16-byte accesses of
// eight columns: past the last row or column they read zero or are dropped.
struct Rows {
    __amdgpu_buffer_rsrc_t r;
    int n;
    __device__ __forceinline__ Rows(const void* p, int m0, int rows, int m, int n_) : n(n_) {
        int left = m - m0;
        left = left < 0 ? 0 : left > rows ? rows : left;
        const char* b = p ? (const char*)p + (int64_t)m0 * n_ * 2 : nullptr;
        r = make_rsrc(uni_ptr(b), p ? (uint32_t)(left * n_ * 2) : 0u);
    }
    __device__ __forceinline__ int at(int row, int col) const { return col < n ? (row * n + col) * 2 : kOob; }
    // POLICY: the store's cache policy bits (1 sc0, 2 nt, 16 sc1)
    template <int POLICY = 0>
    __device__ __forceinline__ void store(int row, int col, v4i v) const {
        __builtin_amdgcn_raw_buffer_store_b128(v, r, at(row, col), 0, POLICY);
    }
    __device__ __forceinline__ v4i load(int row, int col) const {
        return __builtin_amdgcn_raw_buffer_load_b128(r, at(row, col), 0, 0);
    }
};

// The same for fp32, stores only; column -1: none.
struct FloatRows {
    __amdgpu_buffer_rsrc_t r;
    int n;
    __device__ __forceinline__ FloatRows(float* p, int m0, int rows, int m, int n_) : n(n_) {
        int left = m - m0;
        left = left < 0 ? 0 : left > rows ? rows : left;
        r = make_rsrc(uni_ptr((const char*)(p + (int64_t)m0 * n_)), (uint32_t)(left * n_ * 4));
    }
    __device__ __forceinline__ void store(int row, int col, const float (&v)[8]) const {
        const int at = col < 0 ? kOob : (row * n + col) * 4;
        const v4i lo = __builtin_bit_cast(v4i, (v4f){v[0], v[1], v[2], v[3]});
        const v4i hi = __builtin_bit_cast(v4i, (v4f){v[4], v[5], v[6], v[7]});
        __builtin_amdgcn_raw_buffer_store_b128(lo, r, at, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(hi, r, at + 16, 0, 0);
    }
};

}  // namespace dense
}  // namespace dmm
