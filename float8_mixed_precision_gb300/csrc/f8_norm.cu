// Layer norm and RMS norm around a Float8 linear: forward (with the amax of
// its output, for the cast that follows) and backward with the reduction of
// the weight's and the bias's gradients.
//
//   forward   mu = mean x, r = 1/sqrt(mean (x - mu)^2 + eps), y = (x - mu) r w + b
//   backward  xh = (x - mu) r, g = dy w, c1 = mean g xh, c2 = mean g,
//             dx = r (g - c2 - xh c1), dw = sum_rows dy xh, db = sum_rows dy
// (RMS: mu = 0, c2 = 0).  Everything between the loads and the stores is fp32;
// the one rounding is that of the stored value.
//
// Both are bound by HBM: 2 values moved per element forward, 3 backward.  A
// row belongs to a group of TPR threads that keeps it in registers between the
// loads and the store, so each value moves once; the variance is taken from
// the differences to the mean (two reductions over registers), not from the
// sum of squares.
//
// The backward's sums over rows stay in registers too: a group walks its rows
// with a stride of the grid, each thread adding dy xh and dy of the columns it
// owns, and writes one row of partial sums at the end; a second kernel adds
// the partial rows in order.  No atomics, so equal inputs give equal bits.
//
// Rows wider than the register path's 16384 columns take kernels that walk the
// row once per reduction, with the column sums in a kernel of their own.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "f8_internal.h"
#include "f8_ptx.cuh"

namespace f8 {
namespace {

constexpr int kBf16 = 0;

// ------------------------------------------------------------ elements
template <typename T, int VEC>
struct Raw;
template <>
struct Raw<__nv_bfloat16, 8> {
    using type = uint4;
};
template <>
struct Raw<float, 4> {
    using type = uint4;
};
template <>
struct Raw<__nv_bfloat16, 1> {
    using type = uint16_t;
};
template <>
struct Raw<float, 1> {
    using type = uint32_t;
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t bf_pack(float lo, float hi)
{
    __nv_bfloat162 h = __float22bfloat162_rn(make_float2(lo, hi));
    return *reinterpret_cast<uint32_t *>(&h);
}

template <typename T>
__device__ __forceinline__ void unpack(uint4 v, float *f);
template <>
__device__ __forceinline__ void unpack<__nv_bfloat16>(uint4 v, float *f)
{
    f[0] = bf_lo(v.x), f[1] = bf_hi(v.x), f[2] = bf_lo(v.y), f[3] = bf_hi(v.y);
    f[4] = bf_lo(v.z), f[5] = bf_hi(v.z), f[6] = bf_lo(v.w), f[7] = bf_hi(v.w);
}
template <>
__device__ __forceinline__ void unpack<float>(uint4 v, float *f)
{
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
}
template <typename T>
__device__ __forceinline__ void unpack(uint16_t v, float *f)
{
    f[0] = __uint_as_float(static_cast<uint32_t>(v) << 16);
}
template <typename T>
__device__ __forceinline__ void unpack(uint32_t v, float *f)
{
    f[0] = __uint_as_float(v);
}

template <typename T>
__device__ __forceinline__ void pack(const float *f, uint4 &v);
template <>
__device__ __forceinline__ void pack<__nv_bfloat16>(const float *f, uint4 &v)
{
    v = make_uint4(bf_pack(f[0], f[1]), bf_pack(f[2], f[3]), bf_pack(f[4], f[5]),
                   bf_pack(f[6], f[7]));
}
template <>
__device__ __forceinline__ void pack<float>(const float *f, uint4 &v)
{
    v = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                   __float_as_uint(f[3]));
}
template <typename T>
__device__ __forceinline__ void pack(const float *f, uint16_t &v)
{
    v = __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
}
template <typename T>
__device__ __forceinline__ void pack(const float *f, uint32_t &v)
{
    v = __float_as_uint(f[0]);
}

// Magnitude bits of the stored bf16 values, as a running maximum over u16 pairs.
__device__ __forceinline__ uint32_t abs_max2(uint32_t m, uint4 v)
{
    m = __vmaxu2(m, v.x & 0x7FFF7FFFu);
    m = __vmaxu2(m, v.y & 0x7FFF7FFFu);
    m = __vmaxu2(m, v.z & 0x7FFF7FFFu);
    return __vmaxu2(m, v.w & 0x7FFF7FFFu);
}
__device__ __forceinline__ uint32_t abs_max2(uint32_t m, uint16_t v)
{
    return __vmaxu2(m, v & 0x7FFFu);
}
__device__ __forceinline__ uint32_t abs_max2(uint32_t m, uint32_t) { return m; }

// VEC consecutive parameters from column `col`, bf16 or fp32.
template <int VEC>
__device__ __forceinline__ void load_param(const void *p, int type, int col, int cols, float *f,
                                           unsigned *status)
{
#pragma unroll
    for (int e = 0; e < VEC; ++e)
        f[e] = 0.0f;
    if (!in_range(col, VEC, cols, status))
        return;
    if (type == kBf16) {
        const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p) + col;
        if (VEC == 8) {
            unpack<__nv_bfloat16>(__ldg(reinterpret_cast<const uint4 *>(q)), f);
        } else if (VEC == 4) {
            const uint2 v = __ldg(reinterpret_cast<const uint2 *>(q));
            f[0] = bf_lo(v.x), f[1] = bf_hi(v.x), f[2] = bf_lo(v.y), f[3] = bf_hi(v.y);
        } else {
            f[0] = __bfloat162float(*q);
        }
    } else {
        const float *q = static_cast<const float *>(p) + col;
        if (VEC >= 4) {
#pragma unroll
            for (int h = 0; h < VEC / 4; ++h)
                unpack<float>(__ldg(reinterpret_cast<const uint4 *>(q) + h), f + 4 * h);
        } else {
            f[0] = __ldg(q);
        }
    }
}

// ------------------------------------------------------------ reductions
// Sum of (a, b) over the TPR threads of a group, in a fixed order; every
// thread gets it.  `red` holds two float2 per warp of the group, used in
// turn, so that one barrier per reduction is enough.
template <int TPR>
struct GroupSum {
    float2 *red;
    int group, buf;

    __device__ __forceinline__ float2 operator()(float a, float b)
    {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
            b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
        }
        if (TPR == 32)
            return make_float2(a, b);
        constexpr int W = TPR / 32;
        float2 *r = red + (group * 2 + buf) * W;
        buf ^= 1;
        const int t = static_cast<int>(threadIdx.x) % TPR;
        if ((t & 31) == 0)
            r[t >> 5] = make_float2(a, b);
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(TPR) : "memory");
        float2 v = make_float2(0.0f, 0.0f);
        if ((t & 31) < W)
            v = r[t & 31];
#pragma unroll
        for (int o = W / 2; o > 0; o >>= 1) {
            v.x += __shfl_xor_sync(0xFFFFFFFFu, v.x, o);
            v.y += __shfl_xor_sync(0xFFFFFFFFu, v.y, o);
        }
        v.x = __shfl_sync(0xFFFFFFFFu, v.x, 0);
        v.y = __shfl_sync(0xFFFFFFFFu, v.y, 0);
        return v;
    }
};

// What a block leaves of max |y|: its maximum into `amax` (mode 1, one
// atomicMax on the fp32 pattern of a zeroed word; the maximum does not depend
// on the order) or as partial `blockIdx.x` (mode 2).
constexpr int kAmaxNone = 0, kAmaxAtomic = 1, kAmaxPartials = 2;

__device__ __forceinline__ void block_amax(uint32_t m2, int mode, unsigned *amax, unsigned *status)
{
    __shared__ unsigned blk;
    if (threadIdx.x == 0)
        blk = 0;
    __syncthreads();
    const unsigned m = __reduce_max_sync(0xFFFFFFFFu, max(m2 & 0xFFFFu, m2 >> 16));
    if ((threadIdx.x & 31) == 0)
        atomicMax(&blk, m);
    __syncthreads();
    if (threadIdx.x == 0) {
        if (blk >= 0x7F80u)
            atomicOr(status, kStatusNonfinite);
        if (mode == kAmaxAtomic)
            atomicMax(amax, blk << 16);
        else
            amax[blockIdx.x] = blk << 16;
    }
}

__host__ __device__ constexpr int block_threads(int tpr) { return tpr < 256 ? 256 : tpr; }

// ------------------------------------------------------------ forward
template <typename T, int VEC, int NV, int TPR>
__global__ void __launch_bounds__(block_threads(TPR))
norm_fwd_kernel(const T *x, const void *__restrict__ w, const void *__restrict__ b, int w_type,
                int rms, int64_t rows, int cols, float eps, T *y, float *__restrict__ mean,
                float *__restrict__ rstd, unsigned *amax, int amax_mode, unsigned *status)
{
    using R = typename Raw<T, VEC>::type;
    constexpr int kGroups = block_threads(TPR) / TPR;
    __shared__ float2 red[2 * block_threads(TPR) / 32];
    griddep_wait();
    griddep_launch_dependents();
    const int group = threadIdx.x / TPR, t = threadIdx.x % TPR;
    GroupSum<TPR> sum{red, group, 0};
    const int nvec = cols / VEC;
    const float inv_c = 1.0f / static_cast<float>(cols);
    const int64_t total = rows * cols;
    uint32_t m2 = 0;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * kGroups + group; row < rows;
         row += static_cast<int64_t>(gridDim.x) * kGroups) {
        R v[NV];
        const int64_t at = row * cols;
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int i = u * TPR + t;
            v[u] = R{};
            if (i < nvec && in_range(at + static_cast<int64_t>(i) * VEC, VEC, total, status))
                v[u] = *reinterpret_cast<const R *>(x + at + static_cast<int64_t>(i) * VEC);
        }
        float mu = 0.0f;
        if (!rms) {
            float s = 0.0f;
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                float f[VEC];
                unpack<T>(v[u], f);
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    s += f[e];
            }
            mu = sum(s, 0.0f).x * inv_c;
        }
        float q = 0.0f;
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            float f[VEC];
            unpack<T>(v[u], f);
            if (u * TPR + t < nvec) {
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    q = fmaf(f[e] - mu, f[e] - mu, q);
            }
        }
        const float r = 1.0f / sqrtf(sum(q, 0.0f).x * inv_c + eps);
        if (t == 0) {
            if (mean != nullptr && !rms)
                mean[row] = mu;
            if (rstd != nullptr)
                rstd[row] = r;
        }
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int i = u * TPR + t;
            if (i < nvec) {
                float f[VEC], fw[VEC], fb[VEC];
                unpack<T>(v[u], f);
                load_param<VEC>(w, w_type, i * VEC, cols, fw, status);
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    f[e] = (f[e] - mu) * r * fw[e];
                if (b != nullptr) {
                    load_param<VEC>(b, w_type, i * VEC, cols, fb, status);
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        f[e] += fb[e];
                }
                R o;
                pack<T>(f, o);
                m2 = abs_max2(m2, o);
                if (in_range(at + static_cast<int64_t>(i) * VEC, VEC, total, status))
                    *reinterpret_cast<R *>(y + at + static_cast<int64_t>(i) * VEC) = o;
            }
        }
    }
    if (amax_mode != kAmaxNone)
        block_amax(m2, amax_mode, amax, status);
}

// Any width: the row is walked once per reduction and once for the output.
constexpr int kWideThreads = 1024;

template <typename T>
__device__ __forceinline__ float elem(const T *p);
template <>
__device__ __forceinline__ float elem<__nv_bfloat16>(const __nv_bfloat16 *p)
{
    return __bfloat162float(*p);
}
template <>
__device__ __forceinline__ float elem<float>(const float *p)
{
    return *p;
}

template <typename T>
__global__ void __launch_bounds__(kWideThreads)
norm_fwd_wide_kernel(const T *x, const void *__restrict__ w, const void *__restrict__ b, int w_type,
                     int rms, int64_t rows, int64_t cols, float eps, T *y,
                     float *__restrict__ mean, float *__restrict__ rstd, unsigned *amax,
                     int amax_mode, unsigned *status)
{
    using R = typename Raw<T, 1>::type;
    __shared__ float2 red[2 * kWideThreads / 32];
    griddep_wait();
    griddep_launch_dependents();
    GroupSum<kWideThreads> sum{red, 0, 0};
    const float inv_c = 1.0f / static_cast<float>(cols);
    const int64_t total = rows * cols;
    uint32_t m2 = 0;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const T *xr = x + row * cols;
        float mu = 0.0f;
        if (!rms) {
            float s = 0.0f;
            for (int64_t c = threadIdx.x; c < cols; c += kWideThreads)
                if (in_range(row * cols + c, 1, total, status))
                    s += elem(xr + c);
            mu = sum(s, 0.0f).x * inv_c;
        }
        float q = 0.0f;
        for (int64_t c = threadIdx.x; c < cols; c += kWideThreads)
            if (in_range(row * cols + c, 1, total, status)) {
                const float d = elem(xr + c) - mu;
                q = fmaf(d, d, q);
            }
        const float r = 1.0f / sqrtf(sum(q, 0.0f).x * inv_c + eps);
        if (threadIdx.x == 0) {
            if (mean != nullptr && !rms)
                mean[row] = mu;
            if (rstd != nullptr)
                rstd[row] = r;
        }
        for (int64_t c = threadIdx.x; c < cols; c += kWideThreads) {
            if (!in_range(row * cols + c, 1, total, status))
                continue;
            float fw, fb = 0.0f;
            load_param<1>(static_cast<const char *>(w), w_type, static_cast<int>(c),
                          static_cast<int>(cols), &fw, status);
            if (b != nullptr)
                load_param<1>(b, w_type, static_cast<int>(c), static_cast<int>(cols), &fb, status);
            const float f = fmaf((elem(xr + c) - mu) * r, fw, fb);
            R o;
            pack<T>(&f, o);
            m2 = abs_max2(m2, o);
            *reinterpret_cast<R *>(y + row * cols + c) = o;
        }
    }
    if (amax_mode != kAmaxNone)
        block_amax(m2, amax_mode, amax, status);
}

// ------------------------------------------------------------ backward
// parts: [gridDim.x * groups][2][cols] fp32 partial sums of dw and db.
template <typename T, int VEC, int NV, int TPR>
__global__ void __launch_bounds__(block_threads(TPR))
norm_bwd_kernel(const T *dy, const T *x, const void *__restrict__ w, int w_type,
                const float *__restrict__ mean, const float *__restrict__ rstd, int rms,
                int64_t rows, int cols, T *dx, float *__restrict__ parts, unsigned *status)
{
    using R = typename Raw<T, VEC>::type;
    constexpr int kGroups = block_threads(TPR) / TPR;
    __shared__ float2 red[2 * block_threads(TPR) / 32];
    griddep_wait();
    griddep_launch_dependents();
    const int group = threadIdx.x / TPR, t = threadIdx.x % TPR;
    GroupSum<TPR> sum{red, group, 0};
    const int nvec = cols / VEC;
    const float inv_c = 1.0f / static_cast<float>(cols);
    const int64_t total = rows * cols;
    float aw[NV * VEC], ab[NV * VEC];
#pragma unroll
    for (int e = 0; e < NV * VEC; ++e)
        aw[e] = ab[e] = 0.0f;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kGroups + group;
    for (int64_t row = unit; row < rows; row += static_cast<int64_t>(gridDim.x) * kGroups) {
        R vx[NV], vd[NV];
        const int64_t at = row * cols;
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int i = u * TPR + t;
            vx[u] = vd[u] = R{};
            if (i < nvec && in_range(at + static_cast<int64_t>(i) * VEC, VEC, total, status)) {
                vx[u] = *reinterpret_cast<const R *>(x + at + static_cast<int64_t>(i) * VEC);
                vd[u] = *reinterpret_cast<const R *>(dy + at + static_cast<int64_t>(i) * VEC);
            }
        }
        const float mu = rms ? 0.0f : mean[row];
        const float r = rstd[row];
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int i = u * TPR + t;
            if (i < nvec) {
                float fx[VEC], fd[VEC], fw[VEC];
                unpack<T>(vx[u], fx);
                unpack<T>(vd[u], fd);
                load_param<VEC>(w, w_type, i * VEC, cols, fw, status);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float xh = (fx[e] - mu) * r;
                    const float g = fd[e] * fw[e];
                    s1 = fmaf(g, xh, s1);
                    s2 += g;
                    aw[u * VEC + e] = fmaf(fd[e], xh, aw[u * VEC + e]);
                    ab[u * VEC + e] += fd[e];
                }
            }
        }
        if (dx == nullptr)
            continue;
        const float2 c = sum(s1, s2);
        const float c1 = c.x * inv_c, c2 = rms ? 0.0f : c.y * inv_c;
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int i = u * TPR + t;
            if (i < nvec) {
                float fx[VEC], fd[VEC], fw[VEC];
                unpack<T>(vx[u], fx);
                unpack<T>(vd[u], fd);
                load_param<VEC>(w, w_type, i * VEC, cols, fw, status);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float xh = (fx[e] - mu) * r;
                    fx[e] = r * (fmaf(-xh, c1, fd[e] * fw[e]) - c2);
                }
                R o;
                pack<T>(fx, o);
                if (in_range(at + static_cast<int64_t>(i) * VEC, VEC, total, status))
                    *reinterpret_cast<R *>(dx + at + static_cast<int64_t>(i) * VEC) = o;
            }
        }
    }
    if (parts != nullptr) {
        float *p = parts + unit * 2 * cols;
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int i = u * TPR + t;
            if (i < nvec) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    p[i * VEC + e] = aw[u * VEC + e];
                    p[cols + i * VEC + e] = ab[u * VEC + e];
                }
            }
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kWideThreads)
norm_bwd_wide_kernel(const T *dy, const T *x, const void *__restrict__ w, int w_type,
                     const float *__restrict__ mean, const float *__restrict__ rstd, int rms,
                     int64_t rows, int64_t cols, T *dx, unsigned *status)
{
    using R = typename Raw<T, 1>::type;
    __shared__ float2 red[2 * kWideThreads / 32];
    griddep_wait();
    griddep_launch_dependents();
    GroupSum<kWideThreads> sum{red, 0, 0};
    const float inv_c = 1.0f / static_cast<float>(cols);
    const int64_t total = rows * cols;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const T *xr = x + row * cols, *dr = dy + row * cols;
        const float mu = rms ? 0.0f : mean[row];
        const float r = rstd[row];
        float s1 = 0.0f, s2 = 0.0f;
        for (int64_t c = threadIdx.x; c < cols; c += kWideThreads) {
            if (!in_range(row * cols + c, 1, total, status))
                continue;
            float fw;
            load_param<1>(w, w_type, static_cast<int>(c), static_cast<int>(cols), &fw, status);
            const float g = elem(dr + c) * fw;
            s1 = fmaf(g, (elem(xr + c) - mu) * r, s1);
            s2 += g;
        }
        const float2 s = sum(s1, s2);
        const float c1 = s.x * inv_c, c2 = rms ? 0.0f : s.y * inv_c;
        for (int64_t c = threadIdx.x; c < cols; c += kWideThreads) {
            if (!in_range(row * cols + c, 1, total, status))
                continue;
            float fw;
            load_param<1>(w, w_type, static_cast<int>(c), static_cast<int>(cols), &fw, status);
            const float xh = (elem(xr + c) - mu) * r;
            const float f = r * (fmaf(-xh, c1, elem(dr + c) * fw) - c2);
            R o;
            pack<T>(&f, o);
            *reinterpret_cast<R *>(dx + row * cols + c) = o;
        }
    }
}

// Partial column sums for the wide rows: block (x, y) takes 256 columns and
// every gridDim.y-th row.
template <typename T>
__global__ void __launch_bounds__(256)
norm_cols_wide_kernel(const T *__restrict__ dy, const T *__restrict__ x,
                      const float *__restrict__ mean, const float *__restrict__ rstd, int rms,
                      int64_t rows, int64_t cols, float *__restrict__ parts, unsigned *status)
{
    griddep_wait();
    griddep_launch_dependents();
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (c >= cols)
        return;
    float aw = 0.0f, ab = 0.0f;
    const int64_t total = rows * cols;
    for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
        if (!in_range(row * cols + c, 1, total, status))
            continue;
        const float d = elem(dy + row * cols + c);
        const float mu = rms ? 0.0f : mean[row];
        aw = fmaf(d, (elem(x + row * cols + c) - mu) * rstd[row], aw);
        ab += d;
    }
    float *p = parts + static_cast<int64_t>(blockIdx.y) * 2 * cols;
    p[c] = aw;
    p[cols + c] = ab;
}

// dw and db from the partial rows, added in order: 32 columns per block, 8
// threads per column, each every eighth partial row.
__global__ void __launch_bounds__(256)
norm_reduce_kernel(const float *__restrict__ parts, int nparts, int64_t cols, int w_type,
                   void *__restrict__ dw, void *__restrict__ db, unsigned *status)
{
    griddep_wait();
    griddep_launch_dependents();
    void *out = blockIdx.y == 0 ? dw : db;
    if (out == nullptr)
        return;
    __shared__ float acc[8][33];
    const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    float s = 0.0f;
    if (c < cols) {
        const float *p = parts + static_cast<int64_t>(blockIdx.y) * cols + c;
#pragma unroll 4
        for (int i = k; i < nparts; i += 8)
            s += p[static_cast<int64_t>(i) * 2 * cols];
    }
    acc[k][lane] = s;
    __syncthreads();
    if (k == 0 && c < cols && in_range(c, 1, cols, status)) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            s += acc[i][lane];
        if (w_type == kBf16)
            static_cast<__nv_bfloat16 *>(out)[c] = __float2bfloat16_rn(s);
        else
            static_cast<float *>(out)[c] = s;
    }
}

// ------------------------------------------------------------ launches
struct FwdArgs {
    const void *x, *w, *b;
    int w_type, rms;
    int64_t rows, cols;
    float eps;
    void *y;
    float *mean, *rstd;
    unsigned *amax;
    int amax_mode;
};

struct BwdArgs {
    const void *dy, *x, *w;
    int w_type, rms;
    const float *mean, *rstd;
    int64_t rows, cols;
    void *dx, *dw, *db;
    float *parts;
};

// Resident blocks: 2048 threads an SM by the register use of these kernels.
int64_t grid_for(int64_t rows, int tpr, const DeviceInfo &dev, int per_sm)
{
    const int groups = block_threads(tpr) / tpr;
    return std::max<int64_t>(1, std::min<int64_t>((rows + groups - 1) / groups,
                                                  static_cast<int64_t>(dev.sm_count) * per_sm));
}

template <typename T, int VEC, int NV, int TPR>
cudaError_t fwd_launch(const FwdArgs &a, const DeviceInfo &dev, cudaStream_t st, int *nparts)
{
    const int64_t grid = grid_for(a.rows, TPR, dev, 2048 / block_threads(TPR));
    if (nparts != nullptr)
        *nparts = static_cast<int>(grid);
    return launch_pdl(norm_fwd_kernel<T, VEC, NV, TPR>, dim3(static_cast<unsigned>(grid)),
                      dim3(block_threads(TPR)), 0, st, static_cast<const T *>(a.x), a.w, a.b,
                      a.w_type, a.rms, a.rows, static_cast<int>(a.cols), a.eps,
                      static_cast<T *>(a.y), a.mean, a.rstd, a.amax, a.amax_mode, dev.status);
}

constexpr int kMaxBwdBlocksPerSm = 4;
constexpr int kMaxWideParts = 64;

template <typename T, int VEC, int NV, int TPR>
cudaError_t bwd_launch(const BwdArgs &a, const DeviceInfo &dev, cudaStream_t st, int *nparts)
{
    const int per_sm = std::max(1, std::min(kMaxBwdBlocksPerSm, 1024 / block_threads(TPR)));
    const int64_t grid = grid_for(a.rows, TPR, dev, per_sm);
    *nparts = static_cast<int>(grid) * (block_threads(TPR) / TPR);
    return launch_pdl(norm_bwd_kernel<T, VEC, NV, TPR>, dim3(static_cast<unsigned>(grid)),
                      dim3(block_threads(TPR)), 0, st, static_cast<const T *>(a.dy),
                      static_cast<const T *>(a.x), a.w, a.w_type, a.mean, a.rstd, a.rms, a.rows,
                      static_cast<int>(a.cols), static_cast<T *>(a.dx), a.parts, dev.status);
}

// Threads per row by the row's vectors: the smallest group whose registers
// hold the row.
template <typename T, int VEC, int NV>
cudaError_t fwd_pick(const FwdArgs &a, const DeviceInfo &dev, cudaStream_t st, int *nparts)
{
    const int64_t n = a.cols / VEC;
    if (n <= 32 * NV)
        return fwd_launch<T, VEC, NV, 32>(a, dev, st, nparts);
    if (n <= 128 * NV)
        return fwd_launch<T, VEC, NV, 128>(a, dev, st, nparts);
    if (n <= 256 * NV)
        return fwd_launch<T, VEC, NV, 256>(a, dev, st, nparts);
    if (n <= 512 * NV)
        return fwd_launch<T, VEC, NV, 512>(a, dev, st, nparts);
    return fwd_launch<T, VEC, NV, 1024>(a, dev, st, nparts);
}

template <typename T, int VEC, int NV>
cudaError_t bwd_pick(const BwdArgs &a, const DeviceInfo &dev, cudaStream_t st, int *nparts)
{
    const int64_t n = a.cols / VEC;
    if (n <= 32 * NV)
        return bwd_launch<T, VEC, NV, 32>(a, dev, st, nparts);
    if (n <= 128 * NV)
        return bwd_launch<T, VEC, NV, 128>(a, dev, st, nparts);
    if (n <= 256 * NV)
        return bwd_launch<T, VEC, NV, 256>(a, dev, st, nparts);
    if (n <= 512 * NV)
        return bwd_launch<T, VEC, NV, 512>(a, dev, st, nparts);
    return bwd_launch<T, VEC, NV, 1024>(a, dev, st, nparts);
}

constexpr int64_t kRegCols = 16384;  // 16 elements in each of 1024 threads

template <typename T>
cudaError_t fwd_type(const FwdArgs &a, const DeviceInfo &dev, cudaStream_t st, int *nparts)
{
    constexpr int VEC = 16 / sizeof(T);
    if (a.cols <= kRegCols)
        return a.cols % VEC == 0 ? fwd_pick<T, VEC, 16 / VEC>(a, dev, st, nparts)
                                 : fwd_pick<T, 1, 16>(a, dev, st, nparts);
    const int64_t grid = std::min<int64_t>(a.rows, 2 * dev.sm_count);
    if (nparts != nullptr)
        *nparts = static_cast<int>(grid);
    return launch_pdl(norm_fwd_wide_kernel<T>, dim3(static_cast<unsigned>(grid)), dim3(kWideThreads),
                      0, st, static_cast<const T *>(a.x), a.w, a.b, a.w_type, a.rms, a.rows, a.cols,
                      a.eps, static_cast<T *>(a.y), a.mean, a.rstd, a.amax, a.amax_mode, dev.status);
}

template <typename T>
cudaError_t bwd_type(const BwdArgs &a, const DeviceInfo &dev, cudaStream_t st)
{
    constexpr int VEC = 16 / sizeof(T);
    int nparts = 0;
    cudaError_t e = cudaSuccess;
    if (a.cols <= kRegCols) {
        e = a.cols % VEC == 0 ? bwd_pick<T, VEC, 16 / VEC>(a, dev, st, &nparts)
                              : bwd_pick<T, 1, 16>(a, dev, st, &nparts);
    } else {
        // the column sums first: dx may be one of the inputs
        if (a.parts != nullptr) {
            nparts = static_cast<int>(std::min<int64_t>(a.rows, kMaxWideParts));
            e = launch_pdl(norm_cols_wide_kernel<T>,
                           dim3(static_cast<unsigned>((a.cols + 255) / 256), nparts), dim3(256), 0,
                           st, static_cast<const T *>(a.dy), static_cast<const T *>(a.x), a.mean,
                           a.rstd, a.rms, a.rows, a.cols, a.parts, dev.status);
        }
        if (e == cudaSuccess && a.dx != nullptr)
            e = launch_pdl(norm_bwd_wide_kernel<T>,
                           dim3(static_cast<unsigned>(std::min<int64_t>(a.rows, 2 * dev.sm_count))),
                           dim3(kWideThreads), 0, st, static_cast<const T *>(a.dy),
                           static_cast<const T *>(a.x), a.w, a.w_type, a.mean, a.rstd, a.rms,
                           a.rows, a.cols, static_cast<T *>(a.dx), dev.status);
    }
    if (e != cudaSuccess || a.parts == nullptr)
        return e;
    return launch_pdl(norm_reduce_kernel, dim3(static_cast<unsigned>((a.cols + 31) / 32), 2),
                      dim3(256), 0, st, static_cast<const float *>(a.parts), nparts, a.cols,
                      a.w_type, a.dw, a.db, dev.status);
}

f8_status check_norm(f8_dtype x_type, f8_dtype w_type, f8_norm kind, int64_t rows, int64_t cols)
{
    if ((x_type != F8_BF16 && x_type != F8_F32) || (w_type != F8_BF16 && w_type != F8_F32) ||
        (kind != F8_LAYER_NORM && kind != F8_RMS_NORM) || rows < 0 || cols < 0)
        return F8_ERR_INVALID;
    if (cols > INT32_MAX / 2 || (cols > 0 && rows > INT64_MAX / 8 / cols))
        return F8_ERR_SHAPE;
    return F8_OK;
}

f8_status norm_fwd(const void *x, f8_dtype x_type, const void *w, const void *b, f8_dtype w_type,
                   f8_norm kind, int64_t rows, int64_t cols, float eps, void *y, float *mean,
                   float *rstd, unsigned *amax, int amax_mode, const DeviceInfo &dev,
                   cudaStream_t st, int *nparts)
{
    const FwdArgs a{x,   w, b,    w_type, kind == F8_RMS_NORM, rows, cols,
                    eps, y, mean, rstd,   amax,                amax_mode};
    return from_cuda(x_type == F8_BF16 ? fwd_type<__nv_bfloat16>(a, dev, st, nparts)
                                       : fwd_type<float>(a, dev, st, nparts));
}

f8_status check_norm_fwd(const void *x, const void *w, const void *b, int64_t rows, int64_t cols,
                         float eps, const void *y, const float *mean, const float *rstd)
{
    if (!(eps >= 0.0f))
        return F8_ERR_INVALID;
    if (rows > 0 && cols > 0 && (x == nullptr || w == nullptr || y == nullptr))
        return F8_ERR_INVALID;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(b, 16) || !aligned(y, 16) ||
        !aligned(mean, 4) || !aligned(rstd, 4))
        return F8_ERR_ALIGN;
    return F8_OK;
}

} // namespace
} // namespace f8

using namespace f8;

extern "C" {

f8_status f8_norm_fwd(const void *x, f8_dtype x_type, const void *w, const void *b,
                      f8_dtype w_type, f8_norm kind, int64_t rows, int64_t cols, float eps,
                      void *y, float *mean, float *rstd, float *amax_out, void *stream)
{
    F8_TRY(check_norm(x_type, w_type, kind, rows, cols));
    if (amax_out != nullptr && x_type != F8_BF16)
        return F8_ERR_INVALID;
    F8_TRY(check_norm_fwd(x, w, b, rows, cols, eps, y, mean, rstd));
    if (!aligned(amax_out, 4))
        return F8_ERR_ALIGN;
    const DeviceInfo *dev;
    F8_TRY(get_device(&dev));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (amax_out != nullptr)
        F8_TRY_CUDA(cudaMemsetAsync(amax_out, 0, sizeof(float), st));
    if (rows == 0 || cols == 0)
        return F8_OK;
    return norm_fwd(x, x_type, w, b, w_type, kind, rows, cols, eps, y, mean, rstd,
                    reinterpret_cast<unsigned *>(amax_out),
                    amax_out != nullptr ? kAmaxAtomic : kAmaxNone, *dev, st, nullptr);
}

f8_status f8_quantize_norm(const void *x, const void *w, const void *b, f8_dtype w_type,
                           f8_norm kind, int64_t rows, int64_t cols, float eps, void *y,
                           float *mean, float *rstd, float *amax_out, float *scale_out, uint8_t *q,
                           uint8_t *q_t, void *workspace, size_t workspace_bytes, void *stream)
{
    F8_TRY(check_norm(F8_BF16, w_type, kind, rows, cols));
    if (amax_out == nullptr || workspace == nullptr ||
        workspace_bytes < sizeof(unsigned) * kMaxAmaxPartials)
        return F8_ERR_INVALID;
    F8_TRY(check_norm_fwd(x, w, b, rows, cols, eps, y, mean, rstd));
    if (!aligned(q, 16) || !aligned(q_t, 16) || !aligned(amax_out, 4) || !aligned(scale_out, 4) ||
        !aligned(workspace, 16))
        return F8_ERR_ALIGN;
    if (rows == 0 || cols == 0)  // as for an empty tensor: amax 0 and its scale
        return f8_quantize(y, rows, cols, amax_out, scale_out, q, q_t, workspace, workspace_bytes,
                           stream);
    const DeviceInfo *dev;
    F8_TRY(get_device(&dev));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    unsigned *parts = static_cast<unsigned *>(workspace);
    int np = 0;
    F8_TRY(norm_fwd(x, F8_BF16, w, b, w_type, kind, rows, cols, eps, y, mean, rstd, parts,
                    kAmaxPartials, *dev, st, &np));
    return from_cuda(launch_cast_transpose(y, rows, cols, nullptr, parts, np, amax_out, scale_out, q,
                                           q_t, F8_E4M3, *dev, st));
}

size_t f8_norm_bwd_workspace_bytes(int64_t rows, int64_t cols)
{
    if (rows <= 0 || cols <= 0)
        return 0;
    const DeviceInfo *dev = device_info();
    const int64_t sms = dev != nullptr ? dev->sm_count : 152;
    // at most one partial row per warp of the resident blocks, or kMaxWideParts
    const int64_t groups = cols <= kRegCols ? sms * kMaxBwdBlocksPerSm * 8 : kMaxWideParts;
    return static_cast<size_t>(std::min<int64_t>(((rows + 7) / 8) * 8, groups)) * 2 *
           static_cast<size_t>(cols) * sizeof(float);
}

f8_status f8_norm_bwd(const void *dy, const void *x, f8_dtype x_type, const void *w,
                      f8_dtype w_type, const float *mean, const float *rstd, f8_norm kind,
                      int64_t rows, int64_t cols, void *dx, void *dw, void *db, void *workspace,
                      size_t workspace_bytes, void *stream)
{
    F8_TRY(check_norm(x_type, w_type, kind, rows, cols));
    const bool sums = dw != nullptr || db != nullptr;
    if (rows > 0 && cols > 0 &&
        (dy == nullptr || x == nullptr || w == nullptr || rstd == nullptr ||
         (kind == F8_LAYER_NORM && mean == nullptr)))
        return F8_ERR_INVALID;
    if (sums && rows > 0 && cols > 0 &&
        (workspace == nullptr || workspace_bytes < f8_norm_bwd_workspace_bytes(rows, cols)))
        return F8_ERR_INVALID;
    if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(w, 16) || !aligned(mean, 4) ||
        !aligned(rstd, 4) || !aligned(dx, 16) || !aligned(dw, 16) || !aligned(db, 16) ||
        !aligned(workspace, 16))
        return F8_ERR_ALIGN;
    const DeviceInfo *dev;
    F8_TRY(get_device(&dev));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (rows == 0 || cols == 0) {  // a sum over no rows
        const size_t bytes = static_cast<size_t>(cols) * (w_type == F8_BF16 ? 2 : 4);
        if (dw != nullptr && bytes)
            F8_TRY_CUDA(cudaMemsetAsync(dw, 0, bytes, st));
        if (db != nullptr && bytes)
            F8_TRY_CUDA(cudaMemsetAsync(db, 0, bytes, st));
        return F8_OK;
    }
    if (dx == nullptr && !sums)
        return F8_OK;
    const BwdArgs a{dy,   x,  w,  w_type, kind == F8_RMS_NORM, mean, rstd, rows, cols, dx, dw,
                    db, sums ? static_cast<float *>(workspace) : nullptr};
    return from_cuda(x_type == F8_BF16 ? bwd_type<__nv_bfloat16>(a, *dev, st)
                                       : bwd_type<float>(a, *dev, st));
}

} // extern "C"
