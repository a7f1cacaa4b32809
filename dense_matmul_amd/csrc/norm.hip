// norm.hip -- layer norm for gfx950, forward and backward, over rows of bf16
// or fp32:
//   y = (x - mu) r w + b,   mu = mean(x),  r = (mean((x - mu)^2) + eps)^-1/2
//   dx = r (g - mean(g) - xh mean(g xh)),  g = dy w,  xh = (x - mu) r
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// Both passes are bound by memory: each reads its rows once, holds them in
// registers as fp32 (so the variance is of centred values, with no
// cancellation) and writes once.  A row belongs to one wave up to 2048
// columns, to a workgroup of 256 up to 8192, of 1024 up to 16384; each thread
// holds NV vectors of eight consecutive columns, TPR vectors apart.
// Workgroups are persistent: the weight (and in the backward pass the running
// sums of dw and db) stay in registers over all rows of a workgroup, and the
// next row is loaded before the present one is reduced.
// The weight's and bias's gradients are joined in two fixed steps, workgroup
// partials in a caller's workspace and then a sum over them in order, so the
// result does not depend on timing.
//
// Measured on one MI355X: forward 32768 x 7168 bf16 184 us, 5.1 TB/s of the
// bytes that must move (a 4 GiB copy: 4.7-4.8), the same with mean and rstd
// kept; fp32 16384 x 7168 179 us; backward 16384 x 7168 bf16 139 us, 5.1 TB/s,
// fp32 266 us, 5.3; 16 x 1024 forward 6 us, a launch and one row's latency; 1117 x
// 1160 fp32 backward 8 + 3 us, a few rows a wave and then the join's latency.
#include "common.h"

namespace dmm {
namespace norm {

// Workgroups of the backward pass at most: what the registers let run at once
// (two workgroups a compute unit of one wave per row, one of the wider ones).
constexpr int max_parts(int TPR) { return TPR == 64 ? 512 : 256; }

// Eight consecutive values as they lie in memory, and as fp32.  What a row's
// computation does not need yet (the next row, the weight, the bias) is kept
// in this form: for bf16 that is half the registers.
template <class T>
struct Raw;
template <>
struct Raw<uint16_t> {
    v4i q;
    __device__ __forceinline__ void load(const uint16_t* p) { q = *(const v4i*)p; }
    __device__ __forceinline__ void zero() { q = (v4i){0, 0, 0, 0}; }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            v[2 * t] = __builtin_bit_cast(float, (uint32_t)q[t] << 16);
            v[2 * t + 1] = __builtin_bit_cast(float, (uint32_t)q[t] & 0xffff0000u);
        }
    }
};
template <>
struct Raw<float> {
    v4f a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = ((const v4f*)p)[0];
        b = ((const v4f*)p)[1];
    }
    __device__ __forceinline__ void zero() { a = b = (v4f){0.f, 0.f, 0.f, 0.f}; }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            v[t] = a[t];
            v[4 + t] = b[t];
        }
    }
};
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
    *(v4i*)p = (v4i){pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    ((v4f*)p)[0] = (v4f){v[0], v[1], v[2], v[3]};
    ((v4f*)p)[1] = (v4f){v[4], v[5], v[6], v[7]};
}

// Sums of N values over the TPR threads of a row, in every one of them.
// slot: LDS of N x 16 floats of this row's own, free when the last call's
// readers are past a barrier; consecutive calls alternate between two.
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* slot) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] += __shfl_xor(v[n], o);
    if constexpr (TPR > 64) {
        const int w = (threadIdx.x % TPR) >> 6;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int n = 0; n < N; ++n) slot[16 * n + w] = v[n];
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            v[n] = 0.f;
#pragma unroll
            for (int i = 0; i < TPR / 64; ++i) v[n] += slot[16 * n + i];
        }
    }
}

// The vectors of one row that a thread holds.
template <class T, int TPR, int NV>
__device__ __forceinline__ void fetch(const T* p, int64_t row, int rows, int cols, int t, Raw<T> (&v)[NV]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int col = 8 * (i * TPR + t);
        v[i].zero();
        if (col < cols && row < rows) v[i].load(p + row * cols + col);
    }
}

// NT threads, NT / TPR rows at a time.
template <class T, int TPR, int NV, int NT>
__global__ void __launch_bounds__(NT) forward_kernel(const T* x, const T* w, const T* b, T* y, float* mean, float* rstd,
                                                     int rows, int cols, float eps) {
    constexpr int RPB = NT / TPR;
    __shared__ float slots[2][RPB][16];
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    Raw<T> wv[NV], bv[NV], nx[NV];
    const int step = gridDim.x * RPB;
    int row = blockIdx.x * RPB + sub;
    const float inv = 1.f / (float)cols;
    fetch<T, TPR, NV>(x, row, rows, cols, t, nx);
    fetch<T, TPR, NV>(w, 0, 1, cols, t, wv);
    fetch<T, TPR, NV>(b, 0, b ? 1 : 0, cols, t, bv);
    // every thread of a workgroup makes the same number of rounds
    const int rounds = (rows - (int)blockIdx.x * RPB + step - 1) / step;
    for (int k = 0; k < rounds; ++k, row += step) {
        float xv[NV][8];
#pragma unroll
        for (int i = 0; i < NV; ++i) nx[i].get(xv[i]);
        fetch<T, TPR, NV>(x, k + 1 < rounds ? row + step : rows, rows, cols, t, nx);
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) s[0] += xv[i][e];
        row_sum<TPR>(s, slots[0][sub]);
        // divided: the reciprocal's rounding would leave a row of one value off its
        // mean by a last place, and rstd is 1 / sqrt(eps) there
        const float mu = s[0] / (float)cols;
        s[0] = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (8 * (i * TPR + t) < cols)
#pragma unroll
                for (int e = 0; e < 8; ++e) s[0] += (xv[i][e] - mu) * (xv[i][e] - mu);
        row_sum<TPR>(s, slots[1][sub]);
        const float r = 1.f / sqrtf(s[0] * inv + eps);
        if (row < rows) {
            if (t == 0 && mean) {
                mean[row] = mu;
                rstd[row] = r;
            }
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (8 * (i * TPR + t) < cols) {
                    float o[8], wf[8], bf[8];
                    wv[i].get(wf);
                    bv[i].get(bf);
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = (xv[i][e] - mu) * r * wf[e] + bf[e];
                    store8(y + (int64_t)row * cols + 8 * (i * TPR + t), o);
                }
        }
    }
}

// part: [gridDim.x][2][cols], the sums of dy xh and of dy over the rows of
// one workgroup.
template <class T, int TPR, int NV, int NT>
__global__ void __launch_bounds__(NT) backward_kernel(const T* dy, const T* x, const T* w, const float* mean,
                                                      const float* rstd, T* dx, float* part, int rows, int cols) {
    constexpr int RPB = NT / TPR;
    // the next row ahead, where the registers hold it beside the running sums
    constexpr bool AHEAD = TPR < 1024 && (sizeof(T) == 2 || NV <= 2);
    __shared__ float slots[2][RPB][2 * 16];
    __shared__ float join[RPB > 1 ? NT * 8 : 1];
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    Raw<T> wv[NV], nx[NV], ng[NV];
    float dw[NV][8], db[NV][8];
    const int step = gridDim.x * RPB;
    const float inv = 1.f / (float)cols;
    int row = blockIdx.x * RPB + sub;
    float nmu = 0.f, nr = 0.f;
    const auto load = [&](int r) {
        fetch<T, TPR, NV>(x, r, rows, cols, t, nx);
        fetch<T, TPR, NV>(dy, r, rows, cols, t, ng);
        if (r < rows) {
            nmu = mean[r];
            nr = rstd[r];
        }
    };
    if constexpr (AHEAD) load(row);
    fetch<T, TPR, NV>(w, 0, 1, cols, t, wv);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[i][e] = db[i][e] = 0.f;
    const int rounds = (rows - (int)blockIdx.x * RPB + step - 1) / step;
    for (int k = 0; k < rounds; ++k, row += step) {
        const bool live = row < rows;
        if constexpr (!AHEAD) load(row);
        const float mu = nmu, r = nr;
        float xh[NV][8], g[NV][8];
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            nx[i].get(xh[i]);
            ng[i].get(g[i]);
        }
        if constexpr (AHEAD) load(k + 1 < rounds ? row + step : rows);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (8 * (i * TPR + t) < cols && live) {
                float wf[8];
                wv[i].get(wf);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    xh[i][e] = (xh[i][e] - mu) * r;
                    dw[i][e] += g[i][e] * xh[i][e];
                    db[i][e] += g[i][e];
                    g[i][e] *= wf[e];
                    s[0] += g[i][e];
                    s[1] += g[i][e] * xh[i][e];
                }
            }
        row_sum<TPR>(s, slots[k & 1][sub]);
        if (live)
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (8 * (i * TPR + t) < cols) {
                    float o[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = r * (g[i][e] - s[0] * inv - xh[i][e] * (s[1] * inv));
                    store8(dx + (int64_t)row * cols + 8 * (i * TPR + t), o);
                }
    }
    float* mine = part + (int64_t)blockIdx.x * 2 * cols;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            float(&v)[8] = which ? db[i] : dw[i];
            if constexpr (RPB > 1) {  // the workgroup's rows, in order
                __syncthreads();
#pragma unroll
                for (int e = 0; e < 8; ++e) join[e * NT + threadIdx.x] = v[e];
                __syncthreads();
                if (sub == 0)
#pragma unroll
                    for (int q = 1; q < RPB; ++q)
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] += join[e * NT + q * TPR + t];
            }
            if (sub == 0 && 8 * (i * TPR + t) < cols) store8(mine + which * cols + 8 * (i * TPR + t), v);
        }
}

// dw and db (grid y = 0, 1) from the workgroups' partials: 32 columns per
// workgroup, 32 runs of partials side by side, each run's loads in flight
// together, joined in order.
template <class T>
__global__ void __launch_bounds__(1024) join_kernel(const float* part, T* dw, T* db, int parts, int cols) {
    __shared__ float s[32][33];
    constexpr int RUN = max_parts(64) / 32;
    const int c = threadIdx.x & 31, q = threadIdx.x >> 5, col = blockIdx.x * 32 + c;
    const int per = (parts + 31) / 32;  // at most RUN
    float v[RUN];
#pragma unroll
    for (int i = 0; i < RUN; ++i) {
        const int p = q * per + i;
        v[i] = i < per && p < parts && col < cols ? part[((int64_t)p * 2 + blockIdx.y) * cols + col] : 0.f;
    }
#pragma unroll
    for (int i = 1; i < RUN; ++i) v[0] += v[i];
    s[q][c] = v[0];
    __syncthreads();
    // 32 lanes to a column: the tree's order is fixed
    const int cc = threadIdx.x >> 5, out = blockIdx.x * 32 + cc;
    float sum = s[threadIdx.x & 31][cc];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
    if ((threadIdx.x & 31) == 0 && out < cols) {
        T* to = blockIdx.y ? db : dw;
        if constexpr (sizeof(T) == 4)
            to[out] = sum;
        else
            to[out] = (T)(pack_bf16(sum, 0.f) & 0xffff);
    }
}

template <class T, int TPR, int NV, int NT>
static hipError_t forward(const T* x, const T* w, const T* b, T* y, float* mean, float* rstd, int rows, int cols,
                          float eps, hipStream_t st) {
    constexpr int RPB = NT / TPR;
    const int want = (rows + RPB - 1) / RPB, most = TPR == 1024 ? 512 : 2048;
    hipLaunchKernelGGL((forward_kernel<T, TPR, NV, NT>), dim3(want < most ? want : most), dim3(NT), 0, st, x, w, b, y,
                       mean, rstd, rows, cols, eps);
    return hipGetLastError();
}

constexpr int backward_parts(int rows, int TPR, int NT) {
    const int groups = (rows + NT / TPR - 1) / (NT / TPR);
    return groups < max_parts(TPR) ? groups : max_parts(TPR);
}

template <class T, int TPR, int NV, int NT>
static hipError_t backward(const T* dy, const T* x, const T* w, const float* mean, const float* rstd, T* dx, float* part,
                           int rows, int cols, hipStream_t st) {
    hipLaunchKernelGGL((backward_kernel<T, TPR, NV, NT>), dim3(backward_parts(rows, TPR, NT)), dim3(NT), 0, st, dy, x, w,
                       mean, rstd, dx, part, rows, cols);
    return hipGetLastError();
}

// threads per row, vectors per thread and threads per workgroup for a width;
// WG: the workgroup of the rows of 256 threads
#define NORM_BY_WIDTH(F, T, WG, ...)                                   \
    (cols <= 512    ? F<T, 64, 1, 256>(__VA_ARGS__)                    \
     : cols <= 1024 ? F<T, 64, 2, 256>(__VA_ARGS__)                    \
     : cols <= 2048 ? F<T, 64, 4, 256>(__VA_ARGS__)                    \
     : cols <= 4096 ? F<T, 256, 2, WG>(__VA_ARGS__)                    \
     : cols <= 8192 ? F<T, 256, 4, WG>(__VA_ARGS__)                    \
                    : F<T, 1024, 2, 1024>(__VA_ARGS__))
}  // namespace norm

int norm_backward_parts(int rows, int cols) {
    return cols <= 2048   ? norm::backward_parts(rows, 64, 256)
           : cols <= 8192 ? norm::backward_parts(rows, 256, 512)
                          : norm::backward_parts(rows, 1024, 1024);
}

template <class T>
static hipError_t norm_forward(const void* x, const void* w, const void* b, void* y, float* mean, float* rstd, int rows,
                               int cols, float eps, hipStream_t st) {
    return NORM_BY_WIDTH(norm::forward, T, 256, (const T*)x, (const T*)w, (const T*)b, (T*)y, mean, rstd, rows, cols, eps, st);
}

hipError_t launch_layer_norm(int fp32, const void* x, const void* w, const void* b, void* y, float* mean, float* rstd,
                             int rows, int cols, float eps, hipStream_t st) {
    return fp32 ? norm_forward<float>(x, w, b, y, mean, rstd, rows, cols, eps, st)
                : norm_forward<uint16_t>(x, w, b, y, mean, rstd, rows, cols, eps, st);
}

template <class T>
static hipError_t norm_backward(const void* dy, const void* x, const void* w, const float* mean, const float* rstd,
                                void* dx, void* dw, void* db, float* part, int rows, int cols, hipStream_t st) {
    const int parts = norm_backward_parts(rows, cols);
    hipError_t e = hipSuccess;
    if (parts > 0)
        e = NORM_BY_WIDTH(norm::backward, T, 512, (const T*)dy, (const T*)x, (const T*)w, mean, rstd, (T*)dx, part, rows,
                          cols, st);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((norm::join_kernel<T>), dim3((cols + 31) / 32, db ? 2 : 1), dim3(1024), 0, st, part, (T*)dw,
                       (T*)db, parts, cols);
    return hipGetLastError();
}

hipError_t launch_layer_norm_backward(int fp32, const void* dy, const void* x, const void* w, const float* mean,
                                      const float* rstd, void* dx, void* dw, void* db, float* part, int rows, int cols,
                                      hipStream_t st) {
    return fp32 ? norm_backward<float>(dy, x, w, mean, rstd, dx, dw, db, part, rows, cols, st)
                : norm_backward<uint16_t>(dy, x, w, mean, rstd, dx, dw, db, part, rows, cols, st);
}

}  // namespace dmm
