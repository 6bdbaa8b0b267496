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
// Rows wider than a warp holds come through a ring of shared-memory slots that
// bulk copies fill some rows ahead: the registers that hold a row, its
// parameters and its column sums leave too few threads to have enough loads in
// flight of their own.  With plain loads 8192 x 4096 took 34 us forward and
// 85 us backward, through the ring at once 27 and 51 us.
//
// The backward's sums over rows stay in registers too: a group walks its rows
// with a stride of the grid, each thread adding dy xh and dy of the columns it
// owns; a block's groups are joined at the end and leave one row of partial
// sums; a second kernel adds the partial rows in order.  No atomics, so equal
// inputs give equal bits.
//
// Rows wider than the 16384 columns that registers hold take kernels that walk
// the row once per reduction, with the column sums in a kernel of their own.
//
// Measured, bf16, layer norm: forward 8192 x 4096 25.1 us, 5.3 TB/s; backward
// with both parameters' gradients 39.9 us, 5.1 TB/s; a plain copy runs at 6.8.
// RMS norm 21.1 and 39.8: its backward does layer norm's work, sums that only the
// bias needs included.  Farther from the copy rate: widths between the groups'
// (8192 x 2560 24.0 and 36.5 us, of 12.4 and 18.6 for the bytes), odd ones
// (1999 x 5003 26 and 31, of 5.9 and 8.9), narrow ones (65536 x 128 21 and 37, of
// 4.9 and 7.4) and the backward above 8192 columns (4096 x 16384 115 of 59).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>

#include "f8_internal.h"
#include "f8_ptx.cuh"
#include "f8_ring.h"

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

// ------------------------------------------------------------ rows by bulk copies
// The ring kernels bring rows into shared memory with bulk copies, several
// rows ahead, so that the loads in flight do not depend on how many threads
// the registers leave room for: a group of TPR threads walks its rows (stride:
// all groups of the grid) over `stages` slots, and its thread 0 refills a slot
// once the group has taken the row into registers.  A copy covers the row's
// 16-byte pieces, so a row may start inside one (widths that are no multiple
// of 8); the piece that would reach past the last row's end is read directly.
// Such rows are taken from their slot and stored element by element, since an
// element's place in its 16 bytes differs from row to row while a thread's
// columns, parameters and sums do not: 1999 x 5003 bf16 backward 32 us, where
// 2000 x 5000 takes 23.
constexpr int kMaxStages = 8;

struct RowCopy {
    int64_t first;   // element at the slot's start
    int shift;       // elements before the row in the slot
    uint32_t bytes;  // copied
    int tail;        // elements of the row past the copied ones
};

template <typename T>
__device__ __forceinline__ RowCopy row_copy(int64_t row, int64_t rows, int64_t cols)
{
    constexpr int64_t P = 16 / sizeof(T);
    const int64_t b = row * cols, e = b + cols, total = rows * cols;
    RowCopy c;
    c.first = b / P * P;
    c.shift = static_cast<int>(b - c.first);
    const int64_t stop = min((e + P - 1) / P * P, total / P * P);
    c.bytes = static_cast<uint32_t>((stop - c.first) * static_cast<int64_t>(sizeof(T)));
    c.tail = static_cast<int>(max(e - max(stop, b), static_cast<int64_t>(0)));
    return c;
}

// N tensors' rows in one slot, each `pitch` bytes.  WHOLE: every row is whole
// 16-byte pieces.
template <typename T, int N, bool WHOLE>
struct Ring {
    uint8_t *slots;
    uint64_t *full;
    int stages;
    uint32_t pitch;
    int64_t rows, cols;
    const T *src[N];
    int issued;  // copies, by the thread that issues them
    bool ok;     // no wait has run out

    __device__ __forceinline__ T *row(int slot, int which) const
    {
        return reinterpret_cast<T *>(slots + (slot * N + which) * pitch);
    }
    __device__ __forceinline__ void fill(int slot, int64_t r)
    {
        ++issued;
        if (WHOLE) {
            const uint32_t bytes = static_cast<uint32_t>(cols) * sizeof(T);
            mbar_arrive_expect_tx(&full[slot], N * bytes);
#pragma unroll
            for (int i = 0; i < N; ++i)
                bulk_load(row(slot, i), src[i] + r * cols, bytes, &full[slot]);
            return;
        }
        const RowCopy c = row_copy<T>(r, rows, cols);
        mbar_arrive_expect_tx(&full[slot], N * c.bytes);
        if (c.bytes > 0) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                bulk_load(row(slot, i), src[i] + c.first, c.bytes, &full[slot]);
        }
    }
    // A wait that runs out sets the status.  The thread then goes on without
    // waiting, so that all keep to the barriers (what it stores is of no use); the
    // one that issues the copies issues no more, since the slot's phase is not over.
    __device__ __forceinline__ void wait(int slot, uint32_t parity, uint64_t limit_ns,
                                         unsigned *status)
    {
        if (ok && !mbar_wait(&full[slot], parity, nullptr, limit_ns)) {
            ok = false;
            atomicOr(status, kStatusTimeout);
        }
    }
    // The issuing thread's copies land before the block leaves, or takes the slots'
    // memory for something else.
    __device__ __forceinline__ void drain() const
    {
        if (!ok)
            ring_drain(issued, stages, [&](int slot, uint32_t parity) {
                mbar_wait(&full[slot], parity, nullptr, kDrainLimitNs);
            });
    }
};

template <int TPR>
__device__ __forceinline__ void group_sync(int group)
{
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(TPR) : "memory");
}

// The row's elements past the copied ones (of the tensor's last row only),
// into the slot by the group's first threads.
template <typename T, int N, int TPR>
__device__ __forceinline__ void fill_tail(const Ring<T, N, false> &ring, int slot, int64_t r, int group,
                                          int t)
{
    const RowCopy c = row_copy<T>(r, ring.rows, ring.cols);
    if (c.tail == 0)
        return;
    if (t < c.tail) {
        const int64_t at = (r + 1) * ring.cols - c.tail + t;
#pragma unroll
        for (int i = 0; i < N; ++i)
            ring.row(slot, i)[at - c.first] = ring.src[i][at];
    }
    group_sync<TPR>(group);
}

// Sum of a, and of b with PAIR, over the group, in a fixed order; two floats
// per warp and use in `red`, the uses alternating between two halves, so one
// barrier each.
template <int TPR, bool PAIR>
__device__ __forceinline__ float2 ring_sum(float a, float b, float *red, int group, int &buf)
{
    constexpr int W = TPR / 32;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
        if (PAIR)
            b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
    }
    float *r = red + (group * 2 + buf) * 2 * W;
    buf ^= 1;
    const int t = static_cast<int>(threadIdx.x) % TPR;
    if ((t & 31) == 0) {
        r[t >> 5] = a;
        if (PAIR)
            r[W + (t >> 5)] = b;
    }
    group_sync<TPR>(group);
    a = b = 0.0f;
#pragma unroll
    for (int w = 0; w < W; w += 4) {
        const float4 v = *reinterpret_cast<const float4 *>(r + w);
        a += (v.x + v.y) + (v.z + v.w);
        if (PAIR) {
            const float4 u = *reinterpret_cast<const float4 *>(r + W + w);
            b += (u.x + u.y) + (u.z + u.w);
        }
    }
    return make_float2(a, b);
}

// The slot's columns of one thread as VEC-wide vectors u * TPR + t.
template <typename T, int VEC, int NV, int TPR>
__device__ __forceinline__ void take(const T *row, int shift, int nvec, int t,
                                     typename Raw<T, VEC>::type (&v)[NV])
{
    using R = typename Raw<T, VEC>::type;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const int i = u * TPR + t;
        v[u] = R{};
        if (i < nvec)
            v[u] = VEC == 1 ? reinterpret_cast<const R *>(row + shift)[i]
                            : reinterpret_cast<const R *>(row)[i];
    }
}

// Values in pairs: two neighbouring elements of a vector, or (VEC 1) the
// elements of two vectors.
template <typename T, int VEC, int NV>
__device__ __forceinline__ void to_pairs(const typename Raw<T, VEC>::type (&v)[NV],
                                         float2 (&f)[NV * VEC / 2])
{
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        float x[VEC];
        unpack<T>(v[u], x);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int i = u * VEC + e;
            if (i & 1)
                f[i / 2].y = x[e];
            else
                f[i / 2].x = x[e];
        }
    }
}

// The thread's parameters into L2 ahead of the rows' copies, behind which their
// loads would otherwise wait for as long as the slots take to fill.
template <int VEC, int NV, int TPR>
__device__ __forceinline__ void prefetch_params(const void *p, int type, int cols, int t)
{
    if (p == nullptr)
        return;
    const int bytes = type == kBf16 ? 2 : 4;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const int i = u * TPR + t;
        if (i < cols / VEC)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char *>(p) + i * VEC * bytes));
    }
}

template <int VEC, int NV, int TPR, int TYPE>
__device__ __forceinline__ void param_values(const void *p, int cols, int t, float (&x)[NV * VEC],
                                             unsigned *status)
{
#pragma unroll
    for (int u = 0; u < NV; ++u)
        if (u * TPR + t < cols / VEC)
            load_param<VEC>(p, TYPE, (u * TPR + t) * VEC, cols, &x[u * VEC], status);
}

template <int VEC, int NV, int TPR>
__device__ __forceinline__ void param_pairs(const void *p, int type, int cols, int t,
                                            float2 (&f)[NV * VEC / 2], unsigned *status)
{
    float x[NV * VEC] = {};
    if (p != nullptr) {
        if (type == kBf16)
            param_values<VEC, NV, TPR, kBf16>(p, cols, t, x, status);
        else
            param_values<VEC, NV, TPR, kBf16 + 1>(p, cols, t, x, status);
    }
#pragma unroll
    for (int i = 0; i < NV * VEC / 2; ++i)
        f[i] = make_float2(x[2 * i], x[2 * i + 1]);
}

// The pairs of vector u as an array of VEC floats.
template <int VEC, int NV>
__device__ __forceinline__ void pair_vector(const float2 (&f)[NV * VEC / 2], int u, float (&x)[VEC])
{
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const int k = u * VEC + e;
        x[e] = (k & 1) ? f[k / 2].y : f[k / 2].x;
    }
}

// Forward on the ring.  w and b stay in registers as fp32; the arithmetic takes
// two elements per instruction.  FULL: the row is as wide as the group's
// registers, so no vector has to be asked for.
template <typename T, int VEC, int NV, int TPR, bool FULL>
__global__ void __launch_bounds__(block_threads(TPR), 768 / block_threads(TPR))
norm_fwd_ring_kernel(const T *x, const void *__restrict__ w, const void *__restrict__ b, int w_type,
                     int rms, int64_t rows, int cols, float eps, T *y, float *__restrict__ mean,
                     float *__restrict__ rstd, unsigned *amax, int amax_mode, int stages,
                     uint32_t pitch, uint64_t limit_ns, unsigned *status)
{
    using R = typename Raw<T, VEC>::type;
    constexpr int kGroups = block_threads(TPR) / TPR;
    constexpr int P = NV * VEC / 2;
    extern __shared__ __align__(16) uint8_t dyn[];
    __shared__ __align__(16) float red[4 * block_threads(TPR) / 32];
    __shared__ __align__(8) uint64_t full[kGroups * kMaxStages];
    const int group = threadIdx.x / TPR, t = threadIdx.x % TPR;
    Ring<T, 1, (VEC > 1)> ring{dyn + static_cast<size_t>(group) * stages * pitch,
                    full + group * kMaxStages, stages, pitch, rows, cols, {x}, 0, true};
    if (t == 0) {
        for (int i = 0; i < stages; ++i)
            mbar_init(&ring.full[i], 1);
        fence_mbar_init();
    }
    griddep_wait();
    griddep_launch_dependents();
    prefetch_params<VEC, NV, TPR>(w, w_type, cols, t);
    prefetch_params<VEC, NV, TPR>(b, w_type, cols, t);
    const int64_t step = static_cast<int64_t>(gridDim.x) * kGroups;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kGroups + group;
    __syncthreads();
    if (t == 0)
        for (int i = 0; i < stages; ++i)
            if (row0 + i * step < rows)
                ring.fill(i, row0 + i * step);
    float2 fw[P], fb[P];
    param_pairs<VEC, NV, TPR>(w, w_type, cols, t, fw, status);
    param_pairs<VEC, NV, TPR>(b, w_type, cols, t, fb, status);
    const int nvec = FULL ? NV * TPR : cols / VEC;
    const float inv_c = 1.0f / static_cast<float>(cols);
    const int64_t total = rows * cols;
    uint32_t m2 = 0;
    int buf = 0, slot = 0;
    uint32_t parity = 0;
    const int64_t ahead = stages * step;
    R *out = reinterpret_cast<R *>(y + row0 * cols) + t;
    const int64_t out_step = step * nvec;
    for (int64_t row = row0; row < rows; row += step, out += out_step) {
        ring.wait(slot, parity, limit_ns, status);
        int shift = 0;
        if constexpr (VEC == 1) {
            shift = row_copy<T>(row, rows, cols).shift;
            fill_tail<T, 1, TPR>(ring, slot, row, group, t);
        }
        R v[NV];
        take<T, VEC, NV, TPR>(ring.row(slot, 0), shift, nvec, t, v);
        float2 f[P];
        to_pairs<T, VEC, NV>(v, f);
        // elements past the row are 0 and take part in the first sum only
        float mu = 0.0f;
        if (!rms) {
            float2 s = f[0];
#pragma unroll
            for (int i = 1; i < P; ++i)
                s = __fadd2_rn(s, f[i]);
            mu = ring_sum<TPR, false>(s.x + s.y, 0.0f, red, group, buf).x * inv_c;
        }
        float2 q = make_float2(0.0f, 0.0f);
        const float2 nmu = make_float2(-mu, -mu);
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            if (u * TPR + t < nvec) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const int k = u * VEC + e;
                    if (VEC > 1) {
                        if ((k & 1) == 0) {
                            f[k / 2] = __fadd2_rn(f[k / 2], nmu);
                            q = __ffma2_rn(f[k / 2], f[k / 2], q);
                        }
                    } else if (k & 1) {
                        f[k / 2].y -= mu;
                        q.y = fmaf(f[k / 2].y, f[k / 2].y, q.y);
                    } else {
                        f[k / 2].x -= mu;
                        q.x = fmaf(f[k / 2].x, f[k / 2].x, q.x);
                    }
                }
            }
        }
        const float r =
            1.0f / sqrtf(ring_sum<TPR, false>(q.x + q.y, 0.0f, red, group, buf).x * inv_c + eps);
        // every thread has taken its part of the row: the slot can be refilled
        if (t == 0) {
            if (ring.ok && row + ahead < rows)
                ring.fill(slot, row + ahead);
            if (mean != nullptr && !rms)
                mean[row] = mu;
            if (rstd != nullptr)
                rstd[row] = r;
        }
        const float2 r2 = make_float2(r, r);
#pragma unroll
        for (int i = 0; i < P; ++i)
            f[i] = __ffma2_rn(__fmul2_rn(f[i], r2), fw[i], fb[i]);
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int i = u * TPR + t;
            if (i < nvec) {
                float o[VEC];
                pair_vector<VEC, NV>(f, u, o);
                R p;
                pack<T>(o, p);
                if (amax_mode != kAmaxNone)
                    m2 = abs_max2(m2, p);
                if (in_range(row * cols + i * VEC, VEC, total, status))
                    out[u * TPR] = p;
            }
        }
        if (++slot == stages) {
            slot = 0;
            parity ^= 1u;
        }
    }
    if (t == 0)
        ring.drain();
    if (amax_mode != kAmaxNone)
        block_amax(m2, amax_mode, amax, status);
}

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

// ------------------------------------------------------------ backward on the ring
// As the forward, with rows of dy beside those of x in a slot.  A block has
// 512 threads in as many groups as its rows' width leaves; their column sums
// are joined in shared memory at the end, so there is one partial row per
// block.  Elements past the row are 0 and add nothing anywhere.
// 512 threads of 128 registers (the row, dy and the two sums of 16 columns, and
// w) fill an SM; what bounds it is a row's chain of shared-memory reads,
// reduction and stores with two rows in work: about 2000 cycles a row of 4096,
// of which the wait for its copy is 150.
constexpr int kBwdThreads = 512;

template <typename T, int VEC, int NV, int TPR, bool FULL>
__global__ void __launch_bounds__(kBwdThreads, 1)
norm_bwd_ring_kernel(const T *dy, const T *x, const void *__restrict__ w, int w_type,
                     const float *__restrict__ mean, const float *__restrict__ rstd, int rms,
                     int64_t rows, int cols, T *dx, float *__restrict__ parts, int stages,
                     uint32_t pitch, uint64_t limit_ns, unsigned *status)
{
    using R = typename Raw<T, VEC>::type;
    constexpr int kGroups = kBwdThreads / TPR;
    constexpr int P = NV * VEC / 2;
    extern __shared__ __align__(16) uint8_t dyn[];
    __shared__ __align__(16) float red[4 * kBwdThreads / 32];
    __shared__ __align__(8) uint64_t full[kGroups * kMaxStages];
    const int group = threadIdx.x / TPR, t = threadIdx.x % TPR;
    Ring<T, 2, (VEC > 1)> ring{dyn + static_cast<size_t>(group) * stages * 2 * pitch,
                    full + group * kMaxStages, stages, pitch, rows, cols, {x, dy}, 0, true};
    if (t == 0) {
        for (int i = 0; i < stages; ++i)
            mbar_init(&ring.full[i], 1);
        fence_mbar_init();
    }
    griddep_wait();
    griddep_launch_dependents();
    prefetch_params<VEC, NV, TPR>(w, w_type, cols, t);
    const int64_t step = static_cast<int64_t>(gridDim.x) * kGroups;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kGroups + group;
    __syncthreads();
    if (t == 0)
        for (int i = 0; i < stages; ++i)
            if (row0 + i * step < rows)
                ring.fill(i, row0 + i * step);
    float2 fw[P], aw[P], ab[P];
    param_pairs<VEC, NV, TPR>(w, w_type, cols, t, fw, status);
#pragma unroll
    for (int i = 0; i < P; ++i)
        aw[i] = ab[i] = make_float2(0.0f, 0.0f);
    const int nvec = FULL ? NV * TPR : cols / VEC;
    const float inv_c = 1.0f / static_cast<float>(cols);
    const int64_t total = rows * cols;
    int buf = 0, slot = 0;
    uint32_t parity = 0;
    // the next row's statistics are on their way while a row is worked on
    float mu_next = 0.0f, r_next = 0.0f;
    if (row0 < rows) {
        mu_next = rms ? 0.0f : mean[row0];
        r_next = rstd[row0];
    }
    const int64_t ahead = stages * step;
    R *out = reinterpret_cast<R *>(dx + row0 * cols) + t;
    const int64_t out_step = step * nvec;
    for (int64_t row = row0; row < rows; row += step, out += out_step) {
        const float mu = mu_next, r = r_next;
        if (row + step < rows) {
            mu_next = rms ? 0.0f : mean[row + step];
            r_next = rstd[row + step];
        }
        ring.wait(slot, parity, limit_ns, status);
        int shift = 0;
        if constexpr (VEC == 1) {
            shift = row_copy<T>(row, rows, cols).shift;
            fill_tail<T, 2, TPR>(ring, slot, row, group, t);
        }
        R vx[NV], vd[NV];
        take<T, VEC, NV, TPR>(ring.row(slot, 0), shift, nvec, t, vx);
        take<T, VEC, NV, TPR>(ring.row(slot, 1), shift, nvec, t, vd);
        float2 xh[P], g[P];
        to_pairs<T, VEC, NV>(vx, xh);
        to_pairs<T, VEC, NV>(vd, g);
        const float2 r2 = make_float2(r, r), nmu = make_float2(-mu, -mu);
        float2 s1 = make_float2(0.0f, 0.0f), s2 = s1;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            xh[i] = __fmul2_rn(__fadd2_rn(xh[i], nmu), r2);
            aw[i] = __ffma2_rn(g[i], xh[i], aw[i]);
            ab[i] = __fadd2_rn(ab[i], g[i]);
            g[i] = __fmul2_rn(g[i], fw[i]);
            s1 = __ffma2_rn(g[i], xh[i], s1);
            s2 = __fadd2_rn(s2, g[i]);
        }
        const float2 c = ring_sum<TPR, true>(s1.x + s1.y, s2.x + s2.y, red, group, buf);
        if (t == 0 && ring.ok && row + ahead < rows)
            ring.fill(slot, row + ahead);
        if (dx != nullptr) {
            const float k1 = -r * (c.x * inv_c), k2 = rms ? 0.0f : -r * (c.y * inv_c);
            const float2 n1 = make_float2(k1, k1), n2 = make_float2(k2, k2);
#pragma unroll
            for (int i = 0; i < P; ++i)
                g[i] = __ffma2_rn(g[i], r2, __ffma2_rn(xh[i], n1, n2));
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                const int i = u * TPR + t;
                if (i < nvec) {
                    float o[VEC];
                    pair_vector<VEC, NV>(g, u, o);
                    R p;
                    pack<T>(o, p);
                    if (in_range(row * cols + i * VEC, VEC, total, status))
                        out[u * TPR] = p;
                }
            }
        }
        if (++slot == stages) {
            slot = 0;
            parity ^= 1u;
        }
    }
    if (t == 0)
        ring.drain();
    if (parts == nullptr)
        return;
    // the groups' sums joined in group order, through the slots' memory
    if (kGroups > 1) {
        float4 *ex = reinterpret_cast<float4 *>(dyn);
        __syncthreads();
        if (group > 0) {
            float4 *mine = ex + (group - 1) * P * TPR + t;
#pragma unroll
            for (int i = 0; i < P; i += 2) {
                mine[i * TPR] = make_float4(aw[i].x, aw[i].y, aw[i + 1].x, aw[i + 1].y);
                mine[(i + 1) * TPR] = make_float4(ab[i].x, ab[i].y, ab[i + 1].x, ab[i + 1].y);
            }
        }
        __syncthreads();
        if (group > 0)
            return;
#pragma unroll
        for (int j = 0; j < kGroups - 1; ++j) {
            const float4 *o = ex + j * P * TPR + t;
#pragma unroll
            for (int i = 0; i < P; i += 2) {
                const float4 u = o[i * TPR], v = o[(i + 1) * TPR];
                aw[i] = __fadd2_rn(aw[i], make_float2(u.x, u.y));
                aw[i + 1] = __fadd2_rn(aw[i + 1], make_float2(u.z, u.w));
                ab[i] = __fadd2_rn(ab[i], make_float2(v.x, v.y));
                ab[i + 1] = __fadd2_rn(ab[i + 1], make_float2(v.z, v.w));
            }
        }
    }
    float *p = parts + static_cast<int64_t>(blockIdx.x) * 2 * cols;
    auto put = [&](float *to, const float2(&f)[P]) {
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int i = u * TPR + t;
            if (i < nvec) {
                float o[VEC];
                pair_vector<VEC, NV>(f, u, o);
                if constexpr (VEC == 1) {
                    to[i] = o[0];
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; e += 4)
                        *reinterpret_cast<float4 *>(to + i * VEC + e) =
                            make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                }
            }
        }
    };
    put(p, aw);
    put(p + cols, ab);
}

// ------------------------------------------------------------ backward
// Rows of up to 512 columns by a warp each, and those of more than 8192 by 1024
// threads.  parts: [gridDim.x][2][cols] fp32 partial sums of dw and db.
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
    if (parts == nullptr)
        return;
    if constexpr (kGroups > 1) {  // joined in group order, as on the ring
        constexpr int Q = NV * VEC / 4;
        __shared__ float4 ex[(kGroups - 1) * 2 * Q * TPR];
        auto at = [&](int g, int i) -> float4 & { return ex[((g - 1) * 2 * Q + i) * TPR + t]; };
        if (group > 0) {
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                at(group, i) = make_float4(aw[4 * i], aw[4 * i + 1], aw[4 * i + 2], aw[4 * i + 3]);
                at(group, Q + i) = make_float4(ab[4 * i], ab[4 * i + 1], ab[4 * i + 2], ab[4 * i + 3]);
            }
        }
        __syncthreads();
        if (group > 0)
            return;
        for (int g = 1; g < kGroups; ++g) {
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                const float4 a = at(g, i), b = at(g, Q + i);
                aw[4 * i] += a.x, aw[4 * i + 1] += a.y, aw[4 * i + 2] += a.z, aw[4 * i + 3] += a.w;
                ab[4 * i] += b.x, ab[4 * i + 1] += b.y, ab[4 * i + 2] += b.z, ab[4 * i + 3] += b.w;
            }
        }
    }
    float *p = parts + static_cast<int64_t>(blockIdx.x) * 2 * cols;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const int i = u * TPR + t;
        if (i < nvec) {
            if constexpr (VEC == 1) {
                p[i] = aw[u];
                p[cols + i] = ab[u];
            } else {
#pragma unroll
                for (int e = u * VEC; e < (u + 1) * VEC; e += 4) {
                    const int c = i * VEC + e - u * VEC;
                    *reinterpret_cast<float4 *>(p + c) = make_float4(aw[e], aw[e + 1], aw[e + 2], aw[e + 3]);
                    *reinterpret_cast<float4 *>(p + cols + c) =
                        make_float4(ab[e], ab[e + 1], ab[e + 2], ab[e + 3]);
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

// dw and db from the partial rows, in a fixed order: 32 columns per block, 32
// threads per column, each every 32nd partial row.
constexpr int kReduceThreads = 1024;

__global__ void __launch_bounds__(kReduceThreads)
norm_reduce_kernel(const float *__restrict__ parts, int nparts, int64_t cols, int w_type,
                   void *__restrict__ dw, void *__restrict__ db, unsigned *status)
{
    griddep_wait();
    griddep_launch_dependents();
    void *out = blockIdx.y == 0 ? dw : db;
    if (out == nullptr)
        return;
    __shared__ float acc[32][33];
    const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    float s = 0.0f;
    if (c < cols) {
        const float *p = parts + static_cast<int64_t>(blockIdx.y) * cols + c;
#pragma unroll 8
        for (int i = k; i < nparts; i += 32)
            s += p[static_cast<int64_t>(i) * 2 * cols];
    }
    acc[k][lane] = s;
    __syncthreads();
    // warp k adds the 32 sums of column k
    s = acc[lane][k];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + k;
    if (lane == 0 && col < cols && in_range(col, 1, cols, status)) {
        if (w_type == kBf16)
            static_cast<__nv_bfloat16 *>(out)[col] = __float2bfloat16_rn(s);
        else
            static_cast<float *>(out)[col] = s;
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

// At most `per_sm` blocks an SM.  The kernels without a ring ask for more than
// their registers let run at once (forward 58 to 64, 108 for fp32 rows of up to 1024
// columns: four or two blocks of 256 threads, of eight asked for; backward 80 to
// 128: three or two, of four), so their blocks run in two waves or more.
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

// Ring launches.  Shared memory for the rows: what leaves room for the blocks
// that the registers allow per SM.
constexpr int kRingBytes = 200 * 1024;

template <auto Kernel>
cudaError_t allow_ring(const DeviceInfo &dev)
{
    static std::once_flag once[64];
    static cudaError_t err[64];
    const int d = dev.ordinal & 63;
    std::call_once(once[d], [&] {
        err[d] = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    });
    return err[d];
}

struct RingPlan {
    int grid, stages;
    uint32_t pitch;
    size_t smem;
};

// Blocks and slots for `groups` groups a block, `per_sm` blocks an SM and
// `tensors` rows a slot.
RingPlan ring_plan(int64_t rows, int64_t cols, int esize, int groups, int per_sm, int tensors,
                   const DeviceInfo &dev)
{
    RingPlan p;
    p.grid = static_cast<int>(std::max<int64_t>(
        1, std::min<int64_t>((rows + groups - 1) / groups,
                             static_cast<int64_t>(dev.sm_count) * per_sm)));
    // up to 15 bytes before and after the row
    p.pitch = static_cast<uint32_t>((cols * esize + 15 + 15) / 16 * 16);
    const int64_t per_group = (rows + static_cast<int64_t>(p.grid) * groups - 1) /
                              (static_cast<int64_t>(p.grid) * groups);
    const int64_t fit = kRingBytes / per_sm / (static_cast<int64_t>(groups) * tensors * p.pitch);
    p.stages = static_cast<int>(std::min<int64_t>(std::min<int64_t>(fit, kMaxStages), per_group));
    p.smem = static_cast<size_t>(groups) * p.stages * tensors * p.pitch;
    return p;
}

constexpr int fwd_blocks(int tpr) { return 768 / block_threads(tpr); }

template <typename T, int VEC, int NV, int TPR, bool FULL = false>
cudaError_t fwd_ring(const FwdArgs &a, const DeviceInfo &dev, cudaStream_t st, int *nparts)
{
    if constexpr (VEC > 1 && !FULL)
        if (a.cols == NV * VEC * TPR)
            return fwd_ring<T, VEC, NV, TPR, true>(a, dev, st, nparts);
    const RingPlan p = ring_plan(a.rows, a.cols, sizeof(T), block_threads(TPR) / TPR,
                                 fwd_blocks(TPR), 1, dev);
    const cudaError_t e = allow_ring<norm_fwd_ring_kernel<T, VEC, NV, TPR, FULL>>(dev);
    if (e != cudaSuccess)
        return e;
    if (nparts != nullptr)
        *nparts = p.grid;
    return launch_pdl(norm_fwd_ring_kernel<T, VEC, NV, TPR, FULL>, dim3(p.grid), dim3(block_threads(TPR)),
                      p.smem, st, static_cast<const T *>(a.x), a.w, a.b, a.w_type, a.rms, a.rows,
                      static_cast<int>(a.cols), a.eps, static_cast<T *>(a.y), a.mean, a.rstd, a.amax,
                      a.amax_mode, p.stages, p.pitch, wait_limit_ns(), dev.status);
}

template <typename T, int VEC, int NV, int TPR, bool FULL = false>
cudaError_t bwd_ring(const BwdArgs &a, const DeviceInfo &dev, cudaStream_t st, int *nparts)
{
    if constexpr (VEC > 1 && !FULL)
        if (a.cols == NV * VEC * TPR)
            return bwd_ring<T, VEC, NV, TPR, true>(a, dev, st, nparts);
    const RingPlan p = ring_plan(a.rows, a.cols, sizeof(T), kBwdThreads / TPR, 1, 2, dev);
    const cudaError_t e = allow_ring<norm_bwd_ring_kernel<T, VEC, NV, TPR, FULL>>(dev);
    if (e != cudaSuccess)
        return e;
    *nparts = p.grid;
    // the join at the end needs what the other groups' threads have added up
    const size_t smem = std::max<size_t>(p.smem, sizeof(float) * 2 * NV * VEC * (kBwdThreads - TPR));
    return launch_pdl(norm_bwd_ring_kernel<T, VEC, NV, TPR, FULL>, dim3(p.grid), dim3(kBwdThreads), smem,
                      st, static_cast<const T *>(a.dy), static_cast<const T *>(a.x), a.w, a.w_type,
                      a.mean, a.rstd, a.rms, a.rows, static_cast<int>(a.cols),
                      static_cast<T *>(a.dx), a.parts, p.stages, p.pitch, wait_limit_ns(),
                      dev.status);
}

constexpr int kMaxBwdBlocksPerSm = 4;
constexpr int kMaxWideParts = 64;

template <typename T, int VEC, int NV, int TPR>
cudaError_t bwd_launch(const BwdArgs &a, const DeviceInfo &dev, cudaStream_t st, int *nparts)
{
    const int per_sm = std::max(1, std::min(kMaxBwdBlocksPerSm, 1024 / block_threads(TPR)));
    const int64_t grid = grid_for(a.rows, TPR, dev, per_sm);
    *nparts = static_cast<int>(grid);
    return launch_pdl(norm_bwd_kernel<T, VEC, NV, TPR>, dim3(static_cast<unsigned>(grid)),
                      dim3(block_threads(TPR)), 0, st, static_cast<const T *>(a.dy),
                      static_cast<const T *>(a.x), a.w, a.w_type, a.mean, a.rstd, a.rms, a.rows,
                      static_cast<int>(a.cols), static_cast<T *>(a.dx), a.parts, dev.status);
}

// Threads per row by its width: the smallest group that holds the row at 16
// elements a thread (32 in the forward's widest).  Up to 512 columns, forward in
// whole vectors up to 1024, a warp has
// the row and needs no barrier, and many warps have loads in flight: 65536 x
// 512 bf16 29 us forward and 55 us backward, on the ring 88 and 101; 65537 x
// 511 57 and 104, on the ring 159 and 157; 32768 x 1024 forward 27, on the ring
// 51.  Above, the ring (measured at the head of this file) up to what its
// registers hold; up to 1024 columns 8 elements a thread, since half the threads
// would have none of 16: 32768 x 1024 backward 47 us against 57, x 1023 forward
// 64 against 91 and backward 61 against 87.
template <typename T, int VEC>
cudaError_t fwd_pick(const FwdArgs &a, const DeviceInfo &dev, cudaStream_t st, int *nparts)
{
    constexpr int NV = 16 / VEC;
    if (a.cols <= 512)
        return fwd_launch<T, VEC, NV, 32>(a, dev, st, nparts);
    if (a.cols <= 1024) {
        if constexpr (VEC > 1)
            return fwd_launch<T, VEC, 2 * NV, 32>(a, dev, st, nparts);
        else
            return fwd_ring<T, VEC, NV / 2, 128>(a, dev, st, nparts);
    }
    if (a.cols <= 2048)
        return fwd_ring<T, VEC, NV, 128>(a, dev, st, nparts);
    if (a.cols <= 4096)
        return fwd_ring<T, VEC, NV, 256>(a, dev, st, nparts);
    if (a.cols <= 8192)
        return fwd_ring<T, VEC, NV, 512>(a, dev, st, nparts);
    return fwd_ring<T, VEC, 2 * NV, 512>(a, dev, st, nparts);
}

template <typename T, int VEC>
cudaError_t bwd_pick(const BwdArgs &a, const DeviceInfo &dev, cudaStream_t st, int *nparts)
{
    constexpr int NV = 16 / VEC;
    if (a.cols <= 512)
        return bwd_launch<T, VEC, NV, 32>(a, dev, st, nparts);
    if (a.cols <= 1024)
        return bwd_ring<T, VEC, NV / 2, 128>(a, dev, st, nparts);
    if (a.cols <= 2048)
        return bwd_ring<T, VEC, NV, 128>(a, dev, st, nparts);
    if (a.cols <= 4096)
        return bwd_ring<T, VEC, NV, 256>(a, dev, st, nparts);
    if (a.cols <= 8192)
        return bwd_ring<T, VEC, NV, 512>(a, dev, st, nparts);
    return bwd_launch<T, VEC, NV, 1024>(a, dev, st, nparts);
}

constexpr int64_t kRegCols = 16384;  // 16 elements in each of 1024 threads, 32 in each of 512

template <typename T>
cudaError_t fwd_type(const FwdArgs &a, const DeviceInfo &dev, cudaStream_t st, int *nparts)
{
    constexpr int VEC = 16 / sizeof(T);
    if (a.cols <= kRegCols)
        return a.cols % VEC == 0 ? fwd_pick<T, VEC>(a, dev, st, nparts)
                                 : fwd_pick<T, 1>(a, dev, st, nparts);
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
        e = a.cols % VEC == 0 ? bwd_pick<T, VEC>(a, dev, st, &nparts)
                              : bwd_pick<T, 1>(a, dev, st, &nparts);
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
                      dim3(kReduceThreads), 0, st, static_cast<const float *>(a.parts), nparts, a.cols,
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
    // at most one partial row per resident block, or kMaxWideParts
    const int64_t parts = cols <= kRegCols ? sms * kMaxBwdBlocksPerSm : kMaxWideParts;
    return static_cast<size_t>(std::min<int64_t>(rows, parts)) * 2 * static_cast<size_t>(cols) *
           sizeof(float);
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
