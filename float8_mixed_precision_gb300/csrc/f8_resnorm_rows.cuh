// Rows of several tensors brought into shared memory some rows ahead by bulk copies,
// cut into column slices over the blocks of a cluster, and the sums over such rows.
// For kernels whose block keeps its slice's columns in registers, eight a thread.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "f8_ptx.cuh"
#include "f8_ring.h"

namespace f8 {
namespace rows {

constexpr int kE = 8;            // columns of a thread
constexpr int kMaxStages = 8;
constexpr int kMaxCluster = 4;

// The elements [begin, begin + n) of a tensor of `total` as the 16-byte pieces that
// hold them; the piece that would reach past the tensor's end is not copied.
template <typename T>
struct Window {
    int64_t first;   // element at the window's start
    int shift;       // elements before the wanted ones
    uint32_t bytes;  // copied
    int tail;        // wanted elements past the copied ones

    __device__ __forceinline__ Window(int64_t begin, int n, int64_t total)
    {
        constexpr int64_t P = 16 / sizeof(T);
        const int64_t end = begin + n;
        first = begin / P * P;
        shift = static_cast<int>(begin - first);
        const int64_t stop = min((end + P - 1) / P * P, total / P * P);
        bytes = static_cast<uint32_t>(max(stop - first, int64_t{0}) * static_cast<int64_t>(sizeof(T)));
        tail = static_cast<int>(max(end - max(stop, begin), int64_t{0}));
    }
};

// Bytes of a slice of n columns in a slot: up to 15 before and after it.
template <typename T>
__host__ __device__ constexpr uint32_t slice_pitch(int n)
{
    return static_cast<uint32_t>((n * static_cast<int>(sizeof(T)) + 15 + 15) / 16 * 16);
}

// This block's columns: slice `rank` of the cluster's `ranks`.
struct Slice {
    int first, n;  // column and count
};

// NA tensors of TA and NR of TR; a slot holds a slice of each.  Of the pointers, NULL
// ones are left out.
template <typename TA, int NA, typename TR, int NR>
struct Slots {
    uint8_t *mem;
    uint64_t *full;
    int stages;
    int64_t cols, total;
    Slice slice;
    const TA *a[NA];
    const TR *r[NR];
    uint32_t issued;  // by thread 0
    bool ok;          // no wait has run out

    __device__ __forceinline__ uint32_t pitch_a() const { return slice_pitch<TA>(slice.n); }
    __device__ __forceinline__ uint32_t pitch_r() const { return slice_pitch<TR>(slice.n); }
    __device__ __forceinline__ uint32_t slot_bytes() const { return NA * pitch_a() + NR * pitch_r(); }
    __device__ __forceinline__ uint8_t *at_a(int slot, int i) const
    {
        return mem + slot * slot_bytes() + i * pitch_a();
    }
    __device__ __forceinline__ uint8_t *at_r(int slot, int i) const
    {
        return mem + slot * slot_bytes() + NA * pitch_a() + i * pitch_r();
    }
    __device__ __forceinline__ int64_t begin(int64_t row) const { return row * cols + slice.first; }

    // by one thread, once every thread is done with the slot
    __device__ __forceinline__ void fill(int64_t row)
    {
        const int slot = ring_slot(issued, stages);
        ++issued;
        const Window<TA> wa(begin(row), slice.n, total);
        const Window<TR> wr(begin(row), slice.n, total);
        uint32_t bytes = 0;
#pragma unroll
        for (int i = 0; i < NA; ++i)
            bytes += a[i] != nullptr ? wa.bytes : 0u;
#pragma unroll
        for (int i = 0; i < NR; ++i)
            bytes += r[i] != nullptr ? wr.bytes : 0u;
        mbar_arrive_expect_tx(&full[slot], bytes);
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (a[i] != nullptr && wa.bytes > 0)
                bulk_load(at_a(slot, i), a[i] + wa.first, wa.bytes, &full[slot]);
#pragma unroll
        for (int i = 0; i < NR; ++i)
            if (r[i] != nullptr && wr.bytes > 0)
                bulk_load(at_r(slot, i), r[i] + wr.first, wr.bytes, &full[slot]);
    }

    // Waits for the block's seq-th row.  A wait that runs out sets the status; the
    // thread then goes on without waiting, so that all keep to the barriers (what it
    // stores is of no use), and issues no more copies.
    __device__ __forceinline__ void wait(uint32_t seq, uint64_t limit_ns, unsigned *status)
    {
        if (ok && !mbar_wait(&full[ring_slot(seq, stages)], ring_parity(seq, stages), nullptr, limit_ns)) {
            ok = false;
            atomicOr(status, kStatusTimeout);
        }
    }

    // The elements past the copied ones (of the tensors' last row only), into the slot;
    // all threads, with a barrier where there are any.
    __device__ __forceinline__ void tails(uint32_t seq, int64_t row)
    {
        const Window<TA> wa(begin(row), slice.n, total);
        const Window<TR> wr(begin(row), slice.n, total);
        if (wa.tail == 0 && wr.tail == 0)
            return;
        const int slot = ring_slot(seq, stages), t = threadIdx.x;
        const int64_t end = begin(row) + slice.n;
        if (t < wa.tail) {
            const int64_t e = end - wa.tail + t;
#pragma unroll
            for (int i = 0; i < NA; ++i)
                if (a[i] != nullptr)
                    reinterpret_cast<TA *>(at_a(slot, i))[e - wa.first] = a[i][e];
        }
        if (t < wr.tail) {
            const int64_t e = end - wr.tail + t;
#pragma unroll
            for (int i = 0; i < NR; ++i)
                if (r[i] != nullptr)
                    reinterpret_cast<TR *>(at_r(slot, i))[e - wr.first] = r[i][e];
        }
        __syncthreads();
    }

    // Thread 0's copies land before the block leaves.
    __device__ __forceinline__ void drain() const
    {
        if (!ok)
            ring_drain(issued, stages, [&](int slot, uint32_t parity) {
                mbar_wait(&full[slot], parity, nullptr, kDrainLimitNs);
            });
    }
};

__device__ __forceinline__ float2 bf2(uint32_t w)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t pack2(float2 f)
{
    __nv_bfloat162 h = __float22bfloat162_rn(f);
    return *reinterpret_cast<uint32_t *>(&h);
}

// A thread's eight columns as pairs.  VEC: columns 8t .. 8t + 7; else t + j T, the
// pair i being columns j = 2i and 2i + 1.  Columns past the slice are 0.
template <bool VEC, typename T>
__device__ __forceinline__ void take(const uint8_t *slot, int shift, int n, float2 (&f)[kE / 2])
{
    const int t = threadIdx.x;
#pragma unroll
    for (int i = 0; i < kE / 2; ++i)
        f[i] = make_float2(0.0f, 0.0f);
    if constexpr (VEC) {
        if (kE * t >= n)
            return;
        const uint4 *p = reinterpret_cast<const uint4 *>(slot + static_cast<size_t>(kE) * t * sizeof(T));
        const uint4 v = p[0];
        if constexpr (sizeof(T) == 2) {
            f[0] = bf2(v.x), f[1] = bf2(v.y), f[2] = bf2(v.z), f[3] = bf2(v.w);
        } else {
            const uint4 w = p[1];
            f[0] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
            f[1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
            f[2] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
            f[3] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
        }
    } else {
        const T *p = reinterpret_cast<const T *>(slot) + shift;
#pragma unroll
        for (int j = 0; j < kE; ++j) {
            const int c = t + j * static_cast<int>(blockDim.x);
            if (c < n) {
                const float v = sizeof(T) == 2 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[c])
                                               : reinterpret_cast<const float *>(p)[c];
                if (j & 1)
                    f[j / 2].y = v;
                else
                    f[j / 2].x = v;
            }
        }
    }
}

// The same columns of a parameter row in global memory, bf16 or fp32; 0 past the
// slice, `none` throughout where there is no parameter.
template <bool VEC>
__device__ __forceinline__ void take_param(const void *p, int f32, int64_t at, int n, float none,
                                           float2 (&f)[kE / 2])
{
    const int t = threadIdx.x;
#pragma unroll
    for (int i = 0; i < kE / 2; ++i)
        f[i] = make_float2(none, none);
    if (p == nullptr)
        return;
#pragma unroll
    for (int i = 0; i < kE / 2; ++i)
        f[i] = make_float2(0.0f, 0.0f);
    if constexpr (VEC) {
        if (kE * t >= n)
            return;
        if (f32) {
            const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at + kE * t);
            const float4 v = __ldg(q), w = __ldg(q + 1);
            f[0] = make_float2(v.x, v.y), f[1] = make_float2(v.z, v.w);
            f[2] = make_float2(w.x, w.y), f[3] = make_float2(w.z, w.w);
        } else {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p) + at + kE * t));
            f[0] = bf2(v.x), f[1] = bf2(v.y), f[2] = bf2(v.z), f[3] = bf2(v.w);
        }
    } else {
#pragma unroll
        for (int j = 0; j < kE; ++j) {
            const int c = t + j * static_cast<int>(blockDim.x);
            if (c < n) {
                const float v = f32 ? __ldg(static_cast<const float *>(p) + at + c)
                                    : __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[at + c]);
                if (j & 1)
                    f[j / 2].y = v;
                else
                    f[j / 2].x = v;
            }
        }
    }
}

// The thread's columns to `p` (the slice's first element), rounded to T.  `seen`
// gathers the largest magnitude of the stored bf16 values.
template <bool VEC, typename T>
__device__ __forceinline__ void give(T *p, int n, const float2 (&f)[kE / 2], uint32_t *seen, bool inside)
{
    const int t = threadIdx.x;
    if (!inside)
        return;
    if constexpr (VEC) {
        if (kE * t >= n)
            return;
        uint4 *q = reinterpret_cast<uint4 *>(p + kE * t);
        if constexpr (sizeof(T) == 2) {
            const uint4 v = make_uint4(pack2(f[0]), pack2(f[1]), pack2(f[2]), pack2(f[3]));
            if (seen != nullptr) {
                const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                            __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
                *seen = __vmaxu2(*seen, m);
            }
            q[0] = v;
        } else {
            q[0] = make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x),
                              __float_as_uint(f[1].y));
            q[1] = make_uint4(__float_as_uint(f[2].x), __float_as_uint(f[2].y), __float_as_uint(f[3].x),
                              __float_as_uint(f[3].y));
        }
    } else {
#pragma unroll
        for (int j = 0; j < kE; ++j) {
            const int c = t + j * static_cast<int>(blockDim.x);
            if (c < n) {
                const float v = (j & 1) ? f[j / 2].y : f[j / 2].x;
                if constexpr (sizeof(T) == 2) {
                    const __nv_bfloat16 h = __float2bfloat16_rn(v);
                    if (seen != nullptr)
                        *seen = __vmaxu2(*seen, static_cast<uint32_t>(__bfloat16_as_ushort(h)) & 0x7FFFu);
                    p[c] = h;
                } else {
                    p[c] = v;
                }
            }
        }
    }
}

// The thread's columns of one row of a gradient in type `f32` (else bf16).
template <bool VEC>
__device__ __forceinline__ void give_param(void *p, int f32, int64_t at, int n, const float2 (&f)[kE / 2])
{
    if (f32)
        give<VEC>(static_cast<float *>(p) + at, n, f, nullptr, true);
    else
        give<VEC>(static_cast<__nv_bfloat16 *>(p) + at, n, f, nullptr, true);
}

// Sum of (a, b) over the cluster's blocks in a fixed order (block, warp, lane tree);
// every thread gets it.  Each warp leaves its part in every block of the cluster, so
// one barrier a sum; the two halves of `red` [2][kMaxCluster][32] are used in turn.
struct ClusterSum {
    float2 *red;
    int half;
    uint32_t rank, ranks;

    __device__ __forceinline__ float2 operator()(float a, float b)
    {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
            b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
        }
        const int w = static_cast<int>(blockDim.x) >> 5;
        float2 *r = red + half * kMaxCluster * 32;
        half ^= 1;
        const uint32_t mine = rank * w + (threadIdx.x >> 5);
        if (ranks == 1) {
            if ((threadIdx.x & 31) == 0)
                r[mine] = make_float2(a, b);
            __syncthreads();
        } else {
            // lane k writes to block k
            if ((threadIdx.x & 31) < ranks) {
                const uint32_t to = cluster_map(smem_addr(r + mine), threadIdx.x & 31);
                asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(a), "f"(b) : "memory");
            }
            cluster_sync();
        }
        // the parts by the lanes, then the tree again: the same order in every warp
        const int parts = w * static_cast<int>(ranks);
        a = b = 0.0f;
        for (int i = threadIdx.x & 31; i < parts; i += 32) {
            a += r[i].x;
            b += r[i].y;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
            b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
        }
        return make_float2(a, b);
    }
};

} // namespace rows
} // namespace f8
