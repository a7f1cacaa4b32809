// lora.hip -- low-rank adapters of many requests beside a shared projection,
// gfx950, bf16 with fp32 sums:
//   y_t = x_t W^T + s_i (x_t A_i^T) B_i^T,  i = ids[t]
// (a token whose id names no adapter gets the shared part alone), or the same
// with x_t W^T replaced by a given c_t.
//
// Many tokens: v_t = s_i x_t A_i^T [m, r] is computed first and rounded to bf16
// once, as the operand of the second product; that is the shared product
// with the adapters' part as further K tiles over the rank, so y is rounded
// once and x W^T never goes through memory.  Few tokens (up to 256): v and the
// shared product, K shared out, go through memory in fp32, and a last kernel
// adds the r products of v and B to each value.
//
// Tokens come in any order.  A group of rows takes the distinct ids among its
// rows in ascending order, one pass each, and keeps a pass's result in the
// rows of that id only: an adapter's infinities and NaN reach its own tokens
// and no others, and what v holds for a token without an adapter is never
// used.
//
// Rounding v costs little: relative error in the mean square against 64 bits
// 0.0019-0.0020, where the result's own rounding gives 0.0017 (few tokens: that).
//
// Bound by the shared product's operations for many tokens: 8192 x 7168 -> 2048,
// 8 adapters of rank 64 in runs, 37 us for v's shares, 5 for their join and
// 180-201 for the product (1.21-1.35 PFLOP/s).  Few tokens read every weight
// once: 48 x 4096 -> 4096, 32 adapters of rank 16, 10 + 4 us.  Beside a given c,
// 2041 x 1792 -> 1168, 5 adapters of rank 40: 7.5 + 4 + 6.6 us, three launches'
// latency.  Between the two, and with many ids to a tile, it is passes over ids
// that cost: 512 x 4096 -> 4096, 32 adapters of rank 16, 24 + 5 + 50 us.
#include "dense_core.h"
#include "dense_pick.h"
#include "split.h"
#include "thin.h"

namespace dmm {
namespace lora {
using namespace dense;

constexpr int kNone = 0x7fffffff;

// The id itself, or kNone where it names no adapter.
__device__ __forceinline__ int valid_id(int id, int adapters) { return id >= 0 && id < adapters ? id : kNone; }

// The nth smallest of the ids of a workgroup's TOK tokens (one per lane,
// repeated across the wave), kNone where there are fewer.  Every lane counts
// the distinct ids below its own.  Kept a loop: unrolled, its code is longer
// than the rest of the kernel, and fetching it cost 5 us of a 7 us call.
template <int TOK>
__device__ __forceinline__ int nth_id(int mine, int nth) {
    int below = 0;
#pragma unroll 1
    for (int j = 0; j < TOK; ++j) {
        const int id = __builtin_amdgcn_readlane(mine, j);
        const uint64_t same = __ballot(mine == id);
        const bool first = (same & ((1ull << j) - 1)) == 0;
        below += (first ? id : kNone) < mine ? 1 : 0;
    }
    const uint64_t hit = __ballot(mine != kNone && below == nth);
    return hit == 0 ? kNone : __builtin_amdgcn_readlane(mine, (int)__builtin_ctzll(hit));
}

// Few tokens: x A^T for 16 tokens, one of their ids, 16 MB ranks and one share
// of K (`per` bytes of a row, so that the reads of an adapter's rows are spread
// over the compute units: one unit takes in some 40 GB/s of such reads); part
// [shares][m][r] fp32.  The tokens are the streamed operand.
struct Shrink {
    const uint16_t *x, *a;
    const int* ids;
    float* part;
    int m, k, r, adapters;
    int per, shares;      // bytes of K to a share
    int groups, rblocks;  // 16 tokens; 16 MB ranks
};
constexpr int kWaves = kThreads / 64;

template <int MB>
__device__ __forceinline__ void shrink_body(thin::Join<MB, kWaves>& join, const Shrink& p, int block) {
    const int share = block % p.shares, rest = block / p.shares, group = rest % p.groups, more = rest / p.groups;
    const int r0 = more % p.rblocks * 16 * MB, nth = more / p.rblocks;
    const int i = lane_id() & 15, t0 = group * 16;
    const int mine = valid_id(p.ids[t0 + i < p.m ? t0 + i : p.m - 1], p.adapters);
    const int cur = nth_id<16>(mine, nth);
    if (cur == kNone) return;  // the same in every wave
    const int64_t from = (int64_t)share * p.per;
    const int kb = 2 * p.k - from < p.per ? (int)(2 * p.k - from) : p.per;
    const char* mat = (const char*)(p.a + ((int64_t)cur * p.r + r0) * p.k) + from;
    const char* rows[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) rows[b] = mat + (int64_t)(r0 + 16 * b + i < p.r ? 16 * b + i : 0) * (2 * p.k);
    // a token of another id has this id's first stand in for it, whose row the L1 holds
    const int row = t0 + (mine == cur ? i : (int)__builtin_ctzll(__ballot(mine == cur)));
    const char* tok = (const char*)(p.x + (int64_t)(row < p.m ? row : p.m - 1) * p.k) + from;
    v4f acc[MB];
    thin::product<false, MB, kWaves>(tok, rows, kb, acc);
    join.put(acc);
    const int width = p.r - r0 < 16 * MB ? p.r - r0 : 16 * MB;
    for (int e = threadIdx.x; e < 16 * width; e += kThreads) {
        const int t = e / width, q = e - t * width;
        if (t0 + t < p.m && p.ids[t0 + t] == cur)
            p.part[((int64_t)share * p.m + t0 + t) * p.r + r0 + q] = join.sum(q, t);
    }
}

template <int MB>
__global__ void __launch_bounds__(kThreads) shrink_kernel(Shrink p) {
    __shared__ thin::Join<MB, kWaves> join;
    shrink_body<MB>(join, p, (int)blockIdx.x);
}

// The same and the shared product's shares in one launch: neither needs the
// other, and a launch costs as much as the smaller calls' work.
template <int MB, class C>
__global__ void __launch_bounds__(kThreads) shrink_and_base_kernel(Shrink p, int shrinks, split::Args base) {
    DENSE_LDS(C, ring);
    __shared__ thin::Join<MB, kWaves> join;
    if ((int)blockIdx.x < shrinks)
        shrink_body<MB>(join, p, (int)blockIdx.x);
    else
        split::partial_body<C>(ring, base, (int)blockIdx.x - shrinks);
}

// y for one token and 256 columns: the shared product's shares (or c) plus
// s_i v B_i^T, v joined from its shares in LDS and kept in fp32.
constexpr int kMostRank = 1024;
__global__ void __launch_bounds__(256) join_lora_kernel(const float* part, int shares, const float* vpart, int vshares,
                                                        const uint16_t* c, const uint16_t* b, const int* ids,
                                                        const float* scales, uint16_t* y, int m, int n, int r,
                                                        int adapters) {
    __shared__ __attribute__((aligned(16))) float v[kMostRank];
    const int t = blockIdx.y, col = (int)(blockIdx.x * 256 + threadIdx.x), id = valid_id(ids[t], adapters);
    const int64_t at = (int64_t)t * n + col, values = (int64_t)m * n;
    float base = 0.f;
    if (col < n) {
        if (c) base = __builtin_bit_cast(float, (uint32_t)c[at] << 16);
#pragma unroll 4
        for (int s = 0; s < shares; ++s) base += part[s * values + at];
    }
    if (id != kNone) {  // the same for the whole workgroup
        const float scale = scales[id];
        for (int q = threadIdx.x; q < r; q += 256) {
            float sum = 0.f;
#pragma unroll 4
            for (int s = 0; s < vshares; ++s) sum += vpart[((int64_t)s * m + t) * r + q];
            v[q] = scale * sum;
        }
        __syncthreads();
        if (col < n) {
            const v4i* pb = (const v4i*)(b + ((int64_t)id * n + col) * r);
            float s = 0.f;
#pragma unroll 4
            for (int q = 0; q < r / 8; ++q) {
                float fb[8];
                unpack8(pb[q], fb);
#pragma unroll
                for (int j = 0; j < 8; ++j) s += v[8 * q + j] * fb[j];
            }
            base += s;
        }
    }
    if (col < n) y[at] = thin::to_bf16(base);
}

// The smallest id above `cur` among the tile's rows (one per thread), kNone if
// there is none.
__device__ __forceinline__ int next_id(int mine, int cur, int* slot) {
    int next = mine > cur ? mine : kNone;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        const int other = __shfl_xor(next, o);
        next = other < next ? other : next;
    }
    __syncthreads();  // the last call's readers are done
    if (lane_id() == 0) slot[wave_id()] = next;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kThreads / 64; ++q) next = slot[q] < next ? slot[q] : next;
    return uni(next);
}

// The order in which tiles of 64 rows take the tokens of a span of kSpan: as
// they come where they come in runs of one id, sorted by id where they do not,
// so that a tile meets few ids either way (every id of a tile costs a pass).
// A bitonic sort of id and place in LDS, by each workgroup of the first product
// for itself; the second product takes the order from memory and its rows of x
// and v by it (an offset per load and lane, about 2 % of a call in runs).  8192
// tokens in any order over 128 adapters of rank 64 at 7168 -> 2048 take
// 343 us beside a given c and 683 with the shared product, and took 1779 and
// 2402 unsorted (in 256 runs: 168 and 384); 512 over 32 of rank 16 at 4096 ->
// 4096 36 and 76, and took 97 and 154.  Which it is depends on the span's ids
// alone, and a token's result not on its place in a tile.
constexpr int kSpan = 1024;
constexpr int kRuns = 32;  // groups of four consecutive tokens with a change of id, at most, unsorted

struct Tokens {
    int* keys;  // LDS: id or 2^20, and the place in the span
    int base, at, span;

    // tile: rows [m0, m0 + 64).  span: kSpan, or 64 where lines are so long that
    // a span's offsets would pass 31 bits.
    __device__ __forceinline__ Tokens(int* keys_, const int* ids, int m0, int m, int adapters, int span_)
        : keys(keys_), base(m0 & -span_), at(m0 & (span_ - 1)), span(span_) {
        const int tid = (int)threadIdx.x;
#pragma unroll
        for (int e = 0; e < kSpan / kThreads; ++e) {
            const int i = e * kThreads + tid, t = base + i;
            const int id = t < m && i < span ? valid_id(ids[t], adapters) : kNone;
            keys[i] = (id == kNone ? 1 << 20 : id) << 10 | i;
        }
        __syncthreads();
        bool change = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = 4 * tid + e;
            change |= i + 1 < span && (keys[i] ^ keys[i + 1]) >> 10 != 0;
        }
        if (__syncthreads_count(change) <= kRuns) return;
        for (int size = 2; size <= kSpan; size *= 2)
            for (int step = size / 2; step > 0; step /= 2) {
#pragma unroll
                for (int e = 0; e < kSpan / 2 / kThreads; ++e) {
                    const int q = e * kThreads + tid, i = 2 * q - (q & (step - 1));
                    const int a = keys[i], b = keys[i + step];
                    if ((a > b) == ((i & size) == 0)) keys[i] = b, keys[i + step] = a;
                }
                __syncthreads();
            }
    }
    __device__ __forceinline__ int row(int q) const { return keys[at + q] & (kSpan - 1); }  // of the span
    __device__ __forceinline__ int id(int q) const {
        const int v = keys[at + q] >> 10;
        return v == 1 << 20 ? kNone : v;
    }
};

// Many tokens: 64 tokens by 64 ranks on the tile engine, whose loads take whole
// lines, K shared out over workgroups (`per` K tiles each); part [shares][m][r]
// fp32.  One pass over K for each of the 64 tokens' ids.
template <class C>
__global__ void __launch_bounds__(kThreads) shrink_tile_kernel(const uint16_t* xp, const uint16_t* a, const int* ids,
                                                               float* part, int2* order, int m, int k, int r,
                                                               int adapters, int per, int tiles_m, int span) {
    DENSE_LDS(C, ring);
    Ctx<C> x = make_ctx<C>(ring);
    __shared__ int slot[kThreads / 64], keys[kSpan];
    const int m0 = (int)blockIdx.x % tiles_m * C::BM, share = (int)blockIdx.x / tiles_m, r0 = blockIdx.y * C::BN;
    const int wm = x.w >> 1, wn = x.w & 1;
    const Tokens tok(keys, ids, m0, m, adapters, span);
    int mine = kNone;
    if ((int)threadIdx.x < C::BM) {
        mine = tok.id(threadIdx.x);
        if (share == 0 && r0 == 0 && m0 + (int)threadIdx.x < m)
            order[m0 + threadIdx.x] = make_int2(tok.base + tok.row(threadIdx.x), mine);
    }
    int rows_id[C::MB], rows[C::MB];
#pragma unroll
    for (int mb = 0; mb < C::MB; ++mb) {
        const int q = wm * (C::BM / 2) + 16 * mb + (x.lane & 15);
        rows_id[mb] = tok.id(q);
        rows[mb] = tok.row(q);
    }
    x.ra.init(wm * (C::BM / 2), x.lane);
    x.rb.init(wn * (C::BN / 2), x.lane);
    const FloatRows out(part + (int64_t)share * m * r, tok.base, span, m, r);
    const int first = share * per, all = (k + 63) / 64 - first;
    for (int cur = next_id(mine, -1, slot); cur != kNone; cur = next_id(mine, cur, slot)) {
        x.KT = all < 0 ? 0 : all > per ? per : all;
        x.la.init(Mat{xp, (int64_t)k * 2, m}, tok.base, k * 2, x.w, x.lane, span);
        x.la.gather(x.w, [&](int q) { return tok.row(q); });
        x.lb.init(Mat{a + (int64_t)cur * r * k, (int64_t)k * 2, r}, r0, k * 2, x.w, x.lane);
        x.la.range(first, x.KT);
        x.lb.range(first, x.KT);
        run(x);
        wait_vm_lgkm0<0>();  // the pipeline's last (empty) loads, before the stages are used again
#pragma unroll
        for (int mb = 0; mb < C::MB; ++mb) {
            claim(x.acc[mb]);
#pragma unroll
            for (int nb = 0; nb < C::NB; nb += 2) {
                const int col = r0 + wn * (C::BN / 2) + 16 * nb + pair_column(x.lane);
                float o[8];
                pair_columns(x.acc[mb][nb], x.acc[mb][nb + 1], o);
                out.store(rows[mb], rows_id[mb] == cur && col < r ? col : -1, o);
            }
        }
    }
}

// v from the shares: eight ranks a thread; tokens without an adapter have none.
__global__ void __launch_bounds__(256) join_shrink_kernel(const float* part, int shares, const int* ids,
                                                          const float* scales, uint16_t* v, int m, int r, int adapters) {
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8, values = (int64_t)m * r;
    if (at >= values) return;
    const int id = valid_id(ids[at / r], adapters);
    if (id == kNone) return;
    float o[8];
    split::sum8(part, shares, values, at, o);
    const float scale = scales[id];
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] *= scale;
    *(v4i*)(v + at) = pack8(o);
}

// BASE: the shared product x w^T; otherwise c is given.
template <class C, bool BASE>
__global__ void __launch_bounds__(kThreads) lora_tile_kernel(const uint16_t* xp, const uint16_t* w, const uint16_t* c,
                                                             const uint16_t* b, const uint16_t* v,
                                                             const int2* tokens, uint16_t* y, int m, int n, int k,
                                                             int r, int tiles_m, int tiles_n, int span) {
    DENSE_LDS(C, ring);
    Ctx<C> x = make_ctx<C>(ring);
    __shared__ int slot[kThreads / 64], place[C::BM], place_id[C::BM];
    int tm, tn;
    order::coords(order::xcd_list(blockIdx.x, gridDim.x, tiles_m * tiles_n).first, tiles_m, tiles_n, tm, tn);
    const int m0 = tm * C::BM, n0 = tn * C::BN, wm = x.w >> 1, wn = x.w & 1;
    span = span < C::BM ? C::BM : span;
    const int base = m0 & -span;  // rows are counted from here
    int mine = kNone;
    if (const int q = (int)threadIdx.x; q < C::BM) {
        // places past the last token: a row past the span's last, and no id
        const int2 t = m0 + q >= m ? make_int2(m, kNone) : tokens ? tokens[m0 + q] : make_int2(m0 + q, kNone);
        mine = t.y;
        place[q] = t.x - base;
        place_id[q] = mine;
    }
    __syncthreads();
    int rows_id[C::MB], rows[C::MB];  // of the lane's accumulator rows
#pragma unroll
    for (int mb = 0; mb < C::MB; ++mb) {
        const int q = wm * (C::BM / 2) + 16 * mb + (x.lane & 15);
        rows[mb] = place[q];
        rows_id[mb] = place_id[q];
    }
    const auto row_of = [&](int q) { return place[q]; };
    x.ra.init(wm * (C::BM / 2), x.lane);
    x.rb.init(wn * (C::BN / 2), x.lane);
    if constexpr (BASE) {
        x.KT = (k + 63) / 64;
        x.la.init(Mat{xp, (int64_t)k * 2, m}, base, k * 2, x.w, x.lane, span);
        x.la.gather(x.w, row_of);
        x.lb.init(Mat{w, (int64_t)k * 2, n}, n0, k * 2, x.w, x.lane);
        run(x);
        wait_vm<0>();  // the pipeline's last (empty) loads, before their stage is used again
    } else {
#pragma unroll
        for (int mb = 0; mb < C::MB; ++mb)
#pragma unroll
            for (int nb = 0; nb < C::NB; ++nb) x.acc[mb][nb] = (v4f){0.f, 0.f, 0.f, 0.f};
    }

    // the adapters: v [m, r] and b_i [n, r] are further K tiles
    for (int cur = next_id(mine, -1, slot); cur != kNone; cur = next_id(mine, cur, slot)) {
        x.KT = (r + 63) / 64;
        x.la.init(Mat{v, (int64_t)r * 2, m}, base, r * 2, x.w, x.lane, span);
        x.la.gather(x.w, row_of);
        x.lb.init(Mat{b + (int64_t)cur * n * r, (int64_t)r * 2, n}, n0, r * 2, x.w, x.lane);
        for (int kt = 0; kt < x.KT; ++kt) {
            // every wave is done with the stage: next_id's barriers, or the one below
            issue<C, 0>(x);
            wait_vm_lgkm0<0>();
            barrier();
#pragma unroll
            for (int nb = 0; nb < C::NB; ++nb) {
                const bf8 b0 = x.rb.template read<0, 0>(x.lds.b[0], nb), b1 = x.rb.template read<1, 0>(x.lds.b[0], nb);
#pragma unroll
                for (int mb = 0; mb < C::MB; ++mb) {
                    asm volatile("" : "+a"(x.acc[mb][nb]));  // in its AGPRs up to here and after, or the loop spills
                    const bf8 a0 = x.ra.template read<0, 0>(x.lds.a[0], mb), a1 = x.ra.template read<1, 0>(x.lds.a[0], mb);
                    v4f t = (v4f){0.f, 0.f, 0.f, 0.f};
                    t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b0, a0, t, 0, 0, 0);
                    t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b1, a1, t, 0, 0, 0);
                    const bool keep = rows_id[mb] == cur;
#pragma unroll
                    for (int e = 0; e < 4; ++e) x.acc[mb][nb][e] += keep ? t[e] : 0.f;
                    asm volatile("" : "+a"(x.acc[mb][nb]));
                }
                __builtin_amdgcn_sched_barrier(0);  // one column block at a time, for the same reason
            }
            wait_vm_lgkm0<0>();
            barrier();
        }
    }

    const Rows out(y, base, span, m, n), in(c, base, span, m, n);
#pragma unroll
    for (int mb = 0; mb < C::MB; ++mb) {
        claim(x.acc[mb]);
        const int rr = rows[mb];
#pragma unroll
        for (int nb = 0; nb < C::NB; nb += 2) {
            const int col = n0 + wn * (C::BN / 2) + 16 * nb + pair_column(x.lane);
            float o[8];
            pair_columns(x.acc[mb][nb], x.acc[mb][nb + 1], o);
            if constexpr (!BASE) {
                float base[8];
                unpack8(in.load(rr, col), base);
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] += base[e];
            }
            out.store(rr, col, pack8(o));
        }
    }
}

// MB: up to 64 ranks a workgroup.  base: the shared product too.
template <int MB>
static hipError_t launch_shrink_as(Shrink p, const split::Args* base, hipStream_t st) {
    p.groups = (p.m + 15) / 16;
    p.rblocks = (p.r + 16 * MB - 1) / (16 * MB);
    const int blocks = shrink_blocks(p.m, p.k, p.r, p.adapters);
    using C = Cfg<64, 64, 4, KC, KC>;
    if (base && shrink_with_base(blocks)) {
        split::Args b = *base;
        const int more = split::partial_blocks<C>(b);
        hipLaunchKernelGGL((shrink_and_base_kernel<MB, C>), dim3(blocks + more), dim3(kThreads), 0, st, p, blocks, b);
        return hipGetLastError();
    }
    if (blocks > 0) hipLaunchKernelGGL((shrink_kernel<MB>), dim3(blocks), dim3(kThreads), 0, st, p);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess || !base ? e : split::launch_partial<C>(*base, st);
}

static hipError_t launch_shrink(const Shrink& p, const split::Args* base, hipStream_t st) {
    switch (shrink_mb(p.r)) {
        case 1: return launch_shrink_as<1>(p, base, st);
        case 2: return launch_shrink_as<2>(p, base, st);
        default: return launch_shrink_as<4>(p, base, st);
    }
}

// A span's rows of `cols` values stay below 2^31 bytes.
static int span_for(int64_t cols) { return cols <= (1 << 19) ? kSpan : 64; }

// Tiles whose rows are tokens in the order `tokens` gives.
template <int BM, int BN, int NS>
using Gathered = Cfg<BM, BN, NS, KC, KC, false, false, false, true>;

struct Second {
    const uint16_t *x, *w, *c, *b, *v;
    const int2* tokens;
    uint16_t* y;
    int m, n, k, r, span;
};

template <class C, bool BASE>
static hipError_t launch_tile(const Second& p, hipStream_t st) {
    const int tm = (p.m + C::BM - 1) / C::BM, tn = (p.n + C::BN - 1) / C::BN;
    hipLaunchKernelGGL((lora_tile_kernel<C, BASE>), dim3(tm * tn), dim3(kThreads), 0, st, p.x, p.w, p.c, p.b, p.v,
                       p.tokens, p.y, p.m, p.n, p.k, p.r, tm, tn, p.span);
    return hipGetLastError();
}

static hipError_t launch_second(const Second& p, hipStream_t st) {
    if (p.c) return launch_tile<Gathered<64, 64, 2>, false>(p, st);
    switch (second_choice(p.m, p.n, p.k)) {
        case kTile256: return launch_tile<Gathered<256, 256, 2>, true>(p, st);
        case kTile128: return launch_tile<Gathered<128, 128, 2>, true>(p, st);
        case kTile128D: return launch_tile<Gathered<128, 128, 4>, true>(p, st);
        default: return launch_tile<Gathered<64, 64, 4>, true>(p, st);
    }
}
}  // namespace lora

using namespace lora;

// Workspace: few tokens, v's shares and the shared product's; many, v in bf16,
// the tokens' order (row of the span and id), and v's shares.
static int64_t front_bytes(int m, int k, int r) {
    const int64_t v = ceil_div((int64_t)m * r * (m <= kJoinMost ? 4 * shrink_shares(k) : 2), 256) * 256;
    return v + (m <= kJoinMost ? 0 : ceil_div((int64_t)m * 8, 256) * 256);
}
int64_t lora_workspace_bytes(int m, int n, int k, int r, bool shared) {
    if (m > kJoinMost) return front_bytes(m, k, r) + (int64_t)shrink_plan(m, k, r).shares * m * r * 4;
    return front_bytes(m, k, r) + (shared ? (int64_t)base_plan(m, n, k).shares * m * n * 4 : 0);
}

hipError_t launch_lora(const uint16_t* x, const uint16_t* w, const uint16_t* c, const uint16_t* a, const uint16_t* b,
                       const int* ids, const float* scales, void* ws, uint16_t* y, int m, int n, int k, int r,
                       int adapters, hipStream_t st) {
    float* part = (float*)((char*)ws + front_bytes(m, k, r));
    hipError_t e = hipSuccess;
    if (m <= kJoinMost) {
        float* v = (float*)ws;
        const split::Plan plan = c ? split::Plan{0, 0, 1} : base_plan(m, n, k);
        const split::Args base{{x, x}, {w, w}, part, m, n, 2 * k, plan, 0, 0};
        e = launch_shrink(Shrink{x, a, ids, v, m, k, r, adapters, shrink_per(k), shrink_shares(k), 0, 0},
                          c ? nullptr : &base, st);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(join_lora_kernel, dim3((n + 255) / 256, m), dim3(256), 0, st, part, plan.shares, v,
                           shrink_shares(k), c, b, ids, scales, y, m, n, r, adapters);
        return hipGetLastError();
    }
    uint16_t* v = (uint16_t*)ws;
    int2* order = (int2*)((char*)ws + ceil_div((int64_t)m * r * 2, 256) * 256);
    const int span = span_for(larger(n, k));
    if (adapters > 0) {
        using C = Gathered<64, 64, 4>;
        const split::Plan plan = shrink_plan(m, k, r);
        const int tiles = (int)ceil_div(m, C::BM);
        hipLaunchKernelGGL((shrink_tile_kernel<C>), dim3(tiles * plan.shares, (unsigned)ceil_div(r, C::BN)), dim3(kThreads),
                           0, st, x, a, ids, part, order, m, k, r, adapters, plan.per, tiles, span);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        hipLaunchKernelGGL(join_shrink_kernel, dim3((unsigned)ceil_div((int64_t)m * r, 2048)), dim3(256), 0, st, part,
                           plan.shares, ids, scales, v, m, r, adapters);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    return launch_second(Second{x, w, c, b, v, adapters > 0 ? order : nullptr, y, m, n, k, r, span}, st);
}

}  // namespace dmm
