// Rows of several tensors brought into shared memory some rows ahead by bulk copies,
// cut into column slices over the blocks of a cluster, and the sums over such rows.
// For kernels whose block keeps its slice's columns in registers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "f8_ptx.cuh"
#include "f8_ring.h"

namespace f8 {
namespace rows {

constexpr int kMaxStages = 8;
constexpr int kMaxCluster = 4;
constexpr int kMaxWarps = 20;  // of a block
constexpr int kMaxParts = 64;  // warps of a cluster
constexpr int kPartsPitch = kMaxParts + 16;  // half the banks further on
constexpr int kSumFloats = 2 * 4 * kPartsPitch;

// How a block's threads lie over its columns.
constexpr int kFull = 0;    // E / 8 vectors of eight each, all within the row, one block a row
constexpr int kVec = 1;     // the same for any whole vectors, of a cluster's slice
constexpr int kRagged = 2;  // element by element
constexpr int kShift = 3;   // vectors on the tensors' own 16-byte boundaries, whatever the width

// Where a thread's vectors of kShift lie.  A row starts s = (row cols) mod 8 elements
// into a vector of the tensor (bf16 and fp32 alike: 16 and 32 bytes), and rows eight
// apart have the same s, so a unit that walks every eighth row keeps its threads on
// their columns.  Position p of such a row is its column p - s; vector u of the thread
// has the positions from slice.first + 8 (u T + t), of which [lo, hi) are columns.  A
// block's slice is in positions too.
template <int MODE, int E>
struct Place {
    int n;      // columns (positions) of the slice
    int first;  // and their first
    __device__ __forceinline__ void set(int slice_first, int slice_n, int, int)
    {
        first = slice_first;
        n = slice_n;
    }
};
template <int E>
struct Place<kShift, E> {
    int n, first, s;
    uint32_t m[E / 2];  // of each pair's elements, 16 set bits where it is a column
    bool all[E / 8];    // the vector is columns only
    __device__ __forceinline__ void set(int slice_first, int slice_n, int shift, int cols)
    {
        n = slice_n;
        first = slice_first;
        s = shift;
#pragma unroll
        for (int u = 0; u < E / 8; ++u) {
            const int c = 8 * (u * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x));
            const int lo = s - (first + c), hi = c < n ? s + cols - (first + c) : 0;
            all[u] = lo <= 0 && hi >= 8;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                m[4 * u + i] = (2 * i >= lo && 2 * i < hi ? 0xFFFFu : 0u) |
                               (2 * i + 1 >= lo && 2 * i + 1 < hi ? 0xFFFF0000u : 0u);
        }
    }
    __device__ __forceinline__ bool whole(int u) const { return all[u]; }
    __device__ __forceinline__ bool has(int u, int e) const { return ((m[4 * u + e / 2] >> (16 * (e & 1))) & 1u) != 0u; }
};

// Zeros where a thread's vectors are not columns.
template <int E>
__device__ __forceinline__ void mask(const Place<kShift, E> &pl, float2 (&f)[E / 2])
{
#pragma unroll
    for (int u = 0; u < E / 8; ++u) {
        if (pl.whole(u))
            continue;
#pragma unroll
        for (int i = 4 * u; i < 4 * u + 4; ++i) {
            f[i].x = __int_as_float(__float_as_int(f[i].x) & (static_cast<int>(pl.m[i] << 16) >> 16));
            f[i].y = __int_as_float(__float_as_int(f[i].y) & (static_cast<int>(pl.m[i]) >> 16));
        }
    }
}

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
        first = begin & ~(P - 1);
        shift = static_cast<int>(begin - first);
        const int64_t stop = min((end + P - 1) & ~(P - 1), total & ~(P - 1));
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

// The columns of one block of a cluster.
struct Slice {
    int first, n;  // column and count
};

// mbar_wait for what is due within a microsecond or two: it reads the global timer
// only after some tries, which would cost more than the wait.
__device__ __forceinline__ bool wait_soon(uint64_t *bar, uint32_t parity, uint64_t limit_ns)
{
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
        if (mbar_try_wait(bar, parity))
            return true;
    return mbar_wait(bar, parity, nullptr, limit_ns);
}

// A row's slot, the phase of its copies, and its memory.
struct Cursor {
    int slot;
    uint32_t parity;
    uint8_t *at;
};

// NA tensors of TA and NR of TR; a slot holds a slice of each.  Of the pointers, NULL
// ones are left out.
template <typename TA, int NA, typename TR, int NR, int MODE>
struct Slots {
    uint8_t *mem;
    uint64_t *full;
    int stages;
    int64_t cols, total;
    Slice slice;
    int shift;  // of kShift
    const TA *a[NA];
    const TR *r[NR];
    uint32_t pitch_a, pitch_r;
    // thread 0's copies
    uint32_t issued;
    int next;
    bool ok;  // no wait has run out
    unsigned *status;

    __device__ __forceinline__ void start(uint8_t *memory, uint64_t *bars, int n, int64_t columns, int64_t rows,
                                          const Slice &s, int s0, unsigned *word)
    {
        status = word;
        shift = s0;
        mem = memory;
        full = bars;
        stages = n;
        cols = columns;
        total = rows * columns;
        slice = s;
        pitch_a = slice_pitch<TA>(s.n);
        pitch_r = slice_pitch<TR>(s.n);
        next = 0;
        issued = 0u;
        ok = true;
    }
    __device__ __forceinline__ uint32_t slot_bytes() const { return NA * pitch_a + NR * pitch_r; }
    __device__ __forceinline__ uint8_t *at_a(const Cursor &c, int i) const { return c.at + i * pitch_a; }
    __device__ __forceinline__ uint8_t *at_r(const Cursor &c, int i) const
    {
        return c.at + NA * pitch_a + i * pitch_r;
    }
    __device__ __forceinline__ int64_t begin(int64_t row) const
    {
        return row * cols + slice.first - (MODE == kShift ? shift : 0);
    }
    // Elements of a slice from b that lie in whole 16-byte pieces of the tensor.
    template <typename T>
    __device__ __forceinline__ int whole(int64_t b) const
    {
        constexpr int64_t P = 16 / sizeof(T);
        return static_cast<int>(max(min(static_cast<int64_t>(slice.n), (total & ~(P - 1)) - b), int64_t{0}));
    }

    // by one thread, once every thread is done with the slot
    __device__ __forceinline__ void fill(int64_t row)
    {
        uint8_t *to = mem + next * slot_bytes();
        uint64_t *bar = &full[next];
        ++issued;
        if (++next == stages)
            next = 0;
        const int64_t b = begin(row);
        int64_t fa = b, fr = b;
        uint32_t ba = slice.n * sizeof(TA), br = slice.n * sizeof(TR);
        if constexpr (MODE == kRagged) {
            const Window<TA> wa(b, slice.n, total);
            const Window<TR> wr(b, slice.n, total);
            fa = wa.first, fr = wr.first, ba = wa.bytes, br = wr.bytes;
        }
        if constexpr (MODE == kShift) {
            ba = whole<TA>(b) * sizeof(TA);
            br = whole<TR>(b) * sizeof(TR);
        }
        if (ba > 0 && !in_range(fa, ba / sizeof(TA), total, status))
            ba = 0u;
        if (br > 0 && !in_range(fr, br / sizeof(TR), total, status))
            br = 0u;
        uint32_t bytes = 0;
#pragma unroll
        for (int i = 0; i < NA; ++i)
            bytes += a[i] != nullptr ? ba : 0u;
#pragma unroll
        for (int i = 0; i < NR; ++i)
            bytes += r[i] != nullptr ? br : 0u;
        mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (a[i] != nullptr && ba > 0)
                bulk_load(to + i * pitch_a, a[i] + fa, ba, bar);
#pragma unroll
        for (int i = 0; i < NR; ++i)
            if (r[i] != nullptr && br > 0)
                bulk_load(to + NA * pitch_a + i * pitch_r, r[i] + fr, br, bar);
    }

    // Waits for the row at `c`.  A wait that runs out sets the status; the thread
    // then goes on without waiting, so that all keep to the barriers (what it stores is
    // of no use), and issues no more copies.
    __device__ __forceinline__ void wait(const Cursor &c, uint64_t limit_ns, unsigned *status)
    {
        if (ok && !wait_soon(&full[c.slot], c.parity, limit_ns)) {
            ok = false;
            atomicOr(status, kStatusTimeout);
        }
    }
    __device__ __forceinline__ Cursor first() const { return Cursor{0, 0u, mem}; }
    __device__ __forceinline__ void step(Cursor &c) const
    {
        c.at += slot_bytes();
        if (++c.slot == stages) {
            c.slot = 0;
            c.at = mem;
            c.parity ^= 1u;
        }
    }

    // Where a row's slice starts in its window, and the elements past the copied ones
    // (of the tensors' last row only) into the slot; all threads, with a barrier where
    // there are any.
    __device__ __forceinline__ void ragged(const Cursor &c, int64_t row, int &shift_a, int &shift_r)
    {
        const int64_t b = begin(row), end = b + slice.n;
        const Window<TA> wa(b, slice.n, total);
        const Window<TR> wr(b, slice.n, total);
        shift_a = wa.shift;
        shift_r = wr.shift;
        if (wa.tail == 0 && wr.tail == 0)
            return;
        const int t = threadIdx.x;
        if (t < wa.tail) {
            const int64_t e = end - wa.tail + t;
#pragma unroll
            for (int i = 0; i < NA; ++i)
                if (a[i] != nullptr && in_range(e, 1, total, status))
                    reinterpret_cast<TA *>(at_a(c, i))[e - wa.first] = a[i][e];
        }
        if (t < wr.tail) {
            const int64_t e = end - wr.tail + t;
#pragma unroll
            for (int i = 0; i < NR; ++i)
                if (r[i] != nullptr && in_range(e, 1, total, status))
                    reinterpret_cast<TR *>(at_r(c, i))[e - wr.first] = r[i][e];
        }
        __syncthreads();
    }

    // The same for kShift, whose slices start at their vectors.
    __device__ __forceinline__ void tail(const Cursor &c, int64_t row)
    {
        const int64_t b = begin(row);
        const int wa = whole<TA>(b), wr = whole<TR>(b), end = static_cast<int>(min(static_cast<int64_t>(slice.n), total - b));
        if (wa >= end && wr >= end)
            return;
        const int t = threadIdx.x;
        if (wa + t < end) {
#pragma unroll
            for (int i = 0; i < NA; ++i)
                if (a[i] != nullptr && in_range(b + wa + t, 1, total, status))
                    reinterpret_cast<TA *>(at_a(c, i))[wa + t] = a[i][b + wa + t];
        }
        if (wr + t < end) {
#pragma unroll
            for (int i = 0; i < NR; ++i)
                if (r[i] != nullptr && in_range(b + wr + t, 1, total, status))
                    reinterpret_cast<TR *>(at_r(c, i))[wr + t] = r[i][b + wr + t];
        }
        __syncthreads();
    }

    // Thread 0's copies land before the block leaves.
    __device__ __forceinline__ void drain() const
    {
        if (!ok)
            ring_drain(issued, stages, [&](int s, uint32_t p) {
                mbar_wait(&full[s], p, nullptr, kDrainLimitNs);
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

// A thread's E columns as pairs.  In vectors: vector u at column 8 (u T + t); ragged:
// columns t + j T, pair i being j = 2i and 2i + 1.  T is the block's size.  Columns past
// the slice are 0 and are not stored.
__device__ __forceinline__ int vec_col(int u)
{
    return 8 * (u * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x));
}
__device__ __forceinline__ int elem_col(int j)
{
    return static_cast<int>(threadIdx.x) + j * static_cast<int>(blockDim.x);
}
template <int MODE>
__device__ __forceinline__ bool vec_in(int c, int n)
{
    return MODE == kFull || c < n;
}

template <int MODE, int E, typename T>
__device__ __forceinline__ void take(const uint8_t *slot, int shift, const Place<MODE, E> &pl,
                                     float2 (&f)[E / 2])
{
    const int n = pl.n;
    if constexpr (MODE != kRagged) {
#pragma unroll
        for (int u = 0; u < E / 8; ++u) {
            const int c = vec_col(u);
            uint4 v = make_uint4(0u, 0u, 0u, 0u), w = v;
            if (vec_in<MODE>(c, n)) {
                const uint4 *p = reinterpret_cast<const uint4 *>(slot + static_cast<size_t>(c) * sizeof(T));
                v = p[0];
                if (sizeof(T) == 4)
                    w = p[1];
            }
            // beside a row's first and last columns lie its neighbours'
            if constexpr (MODE == kShift && sizeof(T) == 2)
                v = make_uint4(v.x & pl.m[4 * u], v.y & pl.m[4 * u + 1], v.z & pl.m[4 * u + 2], v.w & pl.m[4 * u + 3]);
            if constexpr (sizeof(T) == 2) {
                f[4 * u] = bf2(v.x), f[4 * u + 1] = bf2(v.y);
                f[4 * u + 2] = bf2(v.z), f[4 * u + 3] = bf2(v.w);
            } else {
                f[4 * u] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
                f[4 * u + 1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
                f[4 * u + 2] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
                f[4 * u + 3] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
            }
        }
        if constexpr (MODE == kShift && sizeof(T) == 4)
            mask<E>(pl, f);
    } else {
        const T *p = reinterpret_cast<const T *>(slot) + shift;
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const int c = elem_col(j);
            float v = 0.0f;
            if (c < n)
                v = sizeof(T) == 2 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[c])
                                   : reinterpret_cast<const float *>(p)[c];
            if (j & 1)
                f[j / 2].y = v;
            else
                f[j / 2].x = v;
        }
    }
}

// The thread's columns of a row of parameters.  Those in bf16 stay packed.
template <int E, bool BF>
struct Param {
    float2 f[E / 2];
    __device__ __forceinline__ float2 pair(int i) const { return f[i]; }
    __device__ __forceinline__ void set(int i, float2 v) { f[i] = v; }
    __device__ __forceinline__ void word(int i, uint32_t bf) { f[i] = bf2(bf); }
};
template <int E>
struct Param<E, true> {
    uint32_t w[E / 2];
    __device__ __forceinline__ float2 pair(int i) const { return bf2(w[i]); }
    __device__ __forceinline__ void set(int i, float2 v) { w[i] = pack2(v); }
    __device__ __forceinline__ void word(int i, uint32_t bf) { w[i] = bf; }
};

// The slice of a row of parameters in global memory that begins at element `row` of
// `total`, of type T; 0 past the slice.
template <int MODE, int E, typename T, typename P>
__device__ __forceinline__ void take_typed(const T *p, int64_t row, const Place<MODE, E> &pl, P &out, int64_t total,
                                           unsigned *status)
{
    const int64_t at = row + pl.first;
    if constexpr (MODE == kFull || MODE == kVec) {
#pragma unroll
        for (int u = 0; u < E / 8; ++u) {
            const int c = vec_col(u);
            if (!vec_in<MODE>(c, pl.n) || !in_range(at + c, 8, total, status))
                continue;
            const uint4 *q = reinterpret_cast<const uint4 *>(p + at + c);
            const uint4 v = __ldg(q);
            if constexpr (sizeof(T) == 4) {
                const uint4 w = __ldg(q + 1);
                out.set(4 * u, make_float2(__uint_as_float(v.x), __uint_as_float(v.y)));
                out.set(4 * u + 1, make_float2(__uint_as_float(v.z), __uint_as_float(v.w)));
                out.set(4 * u + 2, make_float2(__uint_as_float(w.x), __uint_as_float(w.y)));
                out.set(4 * u + 3, make_float2(__uint_as_float(w.z), __uint_as_float(w.w)));
            } else {
                out.word(4 * u, v.x), out.word(4 * u + 1, v.y);
                out.word(4 * u + 2, v.z), out.word(4 * u + 3, v.w);
            }
        }
    } else {
        // all loads on their way before the first is used
        T v[E];
#pragma unroll
        for (int j = 0; j < E; ++j) {
            v[j] = T(0.0f);
            if constexpr (MODE == kShift) {
                if (pl.has(j / 8, j & 7) && in_range(at + vec_col(j / 8) - pl.s + (j & 7), 1, total, status))
                    v[j] = __ldg(p + at + vec_col(j / 8) - pl.s + (j & 7));
            } else {
                if (elem_col(j) < pl.n && in_range(at + elem_col(j), 1, total, status))
                    v[j] = __ldg(p + at + elem_col(j));
            }
        }
#pragma unroll
        for (int i = 0; i < E / 2; ++i)
            out.set(i, make_float2(static_cast<float>(v[2 * i]), static_cast<float>(v[2 * i + 1])));
    }
}
// The same of bf16 or fp32 (BF: bf16); `none` throughout where there is no parameter.
template <int MODE, int E, bool BF>
__device__ __forceinline__ void take_param(const void *p, int f32, int64_t row, const Place<MODE, E> &pl,
                                           float none, Param<E, BF> &out, int64_t total, unsigned *status)
{
#pragma unroll
    for (int i = 0; i < E / 2; ++i)
        out.set(i, p == nullptr ? make_float2(none, none) : make_float2(0.0f, 0.0f));
    if (p == nullptr)
        return;
    if (!BF && f32)
        take_typed<MODE, E>(static_cast<const float *>(p), row, pl, out, total, status);
    else
        take_typed<MODE, E>(static_cast<const __nv_bfloat16 *>(p), row, pl, out, total, status);
}

// One value to `p`, rounded to T.
template <typename T>
__device__ __forceinline__ void give_one(T *p, float v, uint32_t *seen)
{
    if constexpr (sizeof(T) == 2) {
        const __nv_bfloat16 h = __float2bfloat16_rn(v);
        if (seen != nullptr)
            *seen = __vmaxu2(*seen, static_cast<uint32_t>(__bfloat16_as_ushort(h)) & 0x7FFFu);
        *p = h;
    } else {
        *p = v;
    }
}

// The thread's columns to `p` (the slice's first element), rounded to T.  `seen`
// gathers the largest magnitude of the stored bf16 values.
template <int MODE, int E, typename T>
__device__ __forceinline__ void give(T *p, const Place<MODE, E> &pl, const float2 (&f)[E / 2],
                                     uint32_t *seen = nullptr)
{
    const int n = pl.n;
    if constexpr (MODE != kRagged) {
#pragma unroll
        for (int u = 0; u < E / 8; ++u) {
            const int c = vec_col(u);
            if (!vec_in<MODE>(c, n))
                continue;
            if constexpr (MODE == kShift) {
                if (!pl.whole(u)) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (pl.has(u, e))
                            give_one(p + c + e, (e & 1) ? f[4 * u + e / 2].y : f[4 * u + e / 2].x, seen);
                    continue;
                }
            }
            uint4 *q = reinterpret_cast<uint4 *>(p + c);
            const float2 *g = f + 4 * u;
            if constexpr (sizeof(T) == 2) {
                const uint4 v = make_uint4(pack2(g[0]), pack2(g[1]), pack2(g[2]), pack2(g[3]));
                if (seen != nullptr) {
                    const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                                __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
                    *seen = __vmaxu2(*seen, m);
                }
                q[0] = v;
            } else {
                q[0] = make_uint4(__float_as_uint(g[0].x), __float_as_uint(g[0].y), __float_as_uint(g[1].x),
                                  __float_as_uint(g[1].y));
                q[1] = make_uint4(__float_as_uint(g[2].x), __float_as_uint(g[2].y), __float_as_uint(g[3].x),
                                  __float_as_uint(g[3].y));
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const int c = elem_col(j);
            if (c >= n)
                continue;
            give_one(p + c, (j & 1) ? f[j / 2].y : f[j / 2].x, seen);
        }
    }
}

// Floats from one row of sums to the next: kShift's are laid out by position, which
// keeps its vectors whole; element by element each 32-byte piece would be written eight
// times.
__host__ __device__ __forceinline__ int64_t sums_pitch(int64_t cols)
{
    return cols % 8 == 0 ? cols : (cols + 7 + 7) / 8 * 8;
}

// The thread's columns of a row of sums that begins at element `at` of `total`.
template <int MODE, int E>
__device__ __forceinline__ void give_sums(float *sums, int64_t at, int64_t total, const Place<MODE, E> &pl,
                                          const float2 (&f)[E / 2], unsigned *status)
{
    if (pl.n > 0 && !in_range(at + pl.first, pl.n, total, status))
        return;
    float *row = sums + at;
    if constexpr (MODE == kShift) {
#pragma unroll
        for (int u = 0; u < E / 8; ++u) {
            const int c = vec_col(u);
            if (c < pl.n) {
                float4 *q = reinterpret_cast<float4 *>(row + pl.first + c);
                q[0] = make_float4(f[4 * u].x, f[4 * u].y, f[4 * u + 1].x, f[4 * u + 1].y);
                q[1] = make_float4(f[4 * u + 2].x, f[4 * u + 2].y, f[4 * u + 3].x, f[4 * u + 3].y);
            }
        }
    } else {
        give<MODE, E>(row + pl.first, pl, f);
    }
}
// Or of one of a gradient of `total` elements, of type `f32` (else bf16), not of kShift's.
template <int MODE, int E>
__device__ __forceinline__ void give_param(void *p, int f32, int64_t row, const Place<MODE, E> &pl,
                                           const float2 (&f)[E / 2], int64_t total, unsigned *status)
{
    static_assert(MODE != kShift, "these leave sums");
    if (pl.n > 0 && !in_range(row + pl.first, pl.n, total, status))
        return;
    if (f32)
        give<MODE, E>(static_cast<float *>(p) + row + pl.first, pl, f);
    else
        give<MODE, E>(static_cast<__nv_bfloat16 *>(p) + row + pl.first, pl, f);
}

// Sums over the block, or over the cluster's blocks, in a fixed order; every thread
// gets them.  Each warp leaves its parts, in a cluster by a store to every block that
// counts on that block's mbarrier: a cluster barrier's release would wait for the
// rows' stores to global memory each time (8192 columns over two blocks, backward: 3.0 us
// a row).  The two halves of `red` [2][4][kPartsPitch] and of `bars` are used in turn; a
// half is written again only once every warp has left its part of the sum between,
// which it does after reading this one.  `red` starts as zeros: parts are read four at
// a time.
template <int MODE>
struct Sum {
    float *red;
    uint64_t *bars;
    int half;
    uint32_t rank, ranks, phases;
    bool ok;  // no wait has run out
    uint64_t limit_ns;
    unsigned *status;

    __device__ __forceinline__ void start(float *memory, uint64_t *barriers, uint32_t r, uint32_t n,
                                          uint64_t limit, unsigned *word)
    {
        red = memory;
        bars = barriers;
        half = 0;
        rank = r;
        ranks = n;
        phases = 0u;
        ok = true;
        limit_ns = limit;
        status = word;
    }
    __device__ __forceinline__ bool single() const { return MODE == kFull || ranks == 1; }
    // The part of this warp, by the lanes of `mine`, into `to` of half h.
    __device__ __forceinline__ void leave(float *to, float v, bool mine, int h)
    {
        const uint32_t w = threadIdx.x >> 5;
        if (single()) {
            if (mine)
                to[w] = v;
        } else if (mine) {
            const uint32_t part = smem_addr(to + rank * (blockDim.x >> 5) + w), bar = smem_addr(&bars[h]);
            for (uint32_t k = 0; k < ranks; ++k)
                asm volatile(
                    "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(
                        cluster_map(part, k)),
                    "r"(__float_as_uint(v)), "r"(cluster_map(bar, k))
                    : "memory");
        }
    }
    // All parts of half h are there; `count` a warp.  A wait that runs out sets the
    // status; the thread then goes on without waiting (what it forms is of no use).
    __device__ __forceinline__ void meet(int h, uint32_t count)
    {
        if (single()) {
            __syncthreads();
            return;
        }
        if (threadIdx.x == 0)
            mbar_arrive_expect_tx(&bars[h], count * ranks * (blockDim.x >> 5) * 4u);
        if (ok && !wait_soon(&bars[h], (phases >> h) & 1u, limit_ns)) {
            ok = false;
            atomicOr(status, kStatusTimeout);
        }
        phases ^= 1u << h;
        __syncwarp();
    }
    __device__ __forceinline__ float total(const float *from) const
    {
        float2 s = make_float2(0.0f, 0.0f);
        if (single()) {
#pragma unroll
            for (int i = 0; i < kMaxWarps; i += 4) {
                const float4 v = *reinterpret_cast<const float4 *>(from + i);
                s = __fadd2_rn(s, __fadd2_rn(make_float2(v.x, v.y), make_float2(v.z, v.w)));
            }
        } else {
            const int parts = static_cast<int>(ranks * (blockDim.x >> 5));
#pragma unroll 4
            for (int i = 0; i < parts; i += 4) {
                const float4 v = *reinterpret_cast<const float4 *>(from + i);
                s = __fadd2_rn(s, __fadd2_rn(make_float2(v.x, v.y), make_float2(v.z, v.w)));
            }
        }
        return s.x + s.y;
    }
    __device__ __forceinline__ float *next(int &h)
    {
        h = half;
        half ^= 1;
        return red + h * 4 * kPartsPitch;
    }
    static __device__ __forceinline__ float warp(float a)
    {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
        return a;
    }

    __device__ __forceinline__ float operator()(float a)
    {
        a = warp(a);
        int h;
        float *r = next(h);
        leave(r, a, (threadIdx.x & 31) == 0, h);
        meet(h, 1);
        return total(r);
    }
    // of a and b: the lower lanes gather a, the upper ones b
    __device__ __forceinline__ float2 operator()(float a, float b)
    {
        const bool upper = (threadIdx.x & 16) != 0;
        float v = upper ? b : a;
        v += __shfl_xor_sync(0xFFFFFFFFu, upper ? a : b, 16);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1)
            v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        int h;
        float *r = next(h);
        leave(r + (upper ? kPartsPitch : 0), v, (threadIdx.x & 15) == 0, h);
        meet(h, 2);
        return make_float2(total(r), total(r + kPartsPitch));
    }
    // Of four values: a group of eight lanes gathers one each, on the way to the other
    // warps and back.
    __device__ __forceinline__ float4 operator()(float a, float b, float c, float d)
    {
        const int group = (threadIdx.x & 31) >> 3;
        const bool up2 = (group & 2) != 0, up1 = (group & 1) != 0;
        float u = up2 ? c : a, v = up2 ? d : b;
        u += __shfl_xor_sync(0xFFFFFFFFu, up2 ? a : c, 16);
        v += __shfl_xor_sync(0xFFFFFFFFu, up2 ? b : d, 16);
        float s = up1 ? v : u;
        s += __shfl_xor_sync(0xFFFFFFFFu, up1 ? u : v, 8);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1)
            s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        int h;
        float *r = next(h) + group * kPartsPitch;
        leave(r, s, (threadIdx.x & 7) == 0, h);
        meet(h, 4);
        const int parts = static_cast<int>(ranks * (blockDim.x >> 5));
        s = 0.0f;
        for (int i = 2 * (threadIdx.x & 7); i < parts; i += 16) {
            const float2 w = *reinterpret_cast<const float2 *>(r + i);
            s += w.x + w.y;
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1)
            s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        return make_float4(__shfl_sync(0xFFFFFFFFu, s, 0), __shfl_sync(0xFFFFFFFFu, s, 8),
                           __shfl_sync(0xFFFFFFFFu, s, 16), __shfl_sync(0xFFFFFFFFu, s, 24));
    }
    // Mean of the row and sum of the squared differences to it, from a full block's
    // warps of 32 E values each: a warp takes its own mean and its values' differences
    // to that, and the warps are joined by their means' differences to the row's.  As
    // exact as two passes, with one barrier.  x becomes x - mean.
    template <int E>
    __device__ __forceinline__ float2 moments(float2 (&x)[E / 2], float inv_w)
    {
        constexpr float kCount = 32.0f * E;
        float2 s = x[0];
#pragma unroll
        for (int i = 1; i < E / 2; ++i)
            s = __fadd2_rn(s, x[i]);
        const float mean = warp(s.x + s.y) * (1.0f / kCount);
        float2 q = make_float2(0.0f, 0.0f);
        const float2 nm = make_float2(-mean, -mean);
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            const float2 d = __fadd2_rn(x[i], nm);
            q = __ffma2_rn(d, d, q);
        }
        const float m2 = warp(q.x + q.y);
        int h;
        float *r = next(h);
        leave(r, mean, (threadIdx.x & 31) == 0, h);
        leave(r + kPartsPitch, m2, (threadIdx.x & 31) == 0, h);
        meet(h, 2);
        const int w = static_cast<int>(blockDim.x >> 5);
        const float mu = total(r) * inv_w;
        float2 all = make_float2(0.0f, 0.0f);
        const float2 nu = make_float2(-mu, -mu), count = make_float2(kCount, kCount);
        for (int i = 0; i < w; i += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(r + i);
            const float4 q4 = *reinterpret_cast<const float4 *>(r + kPartsPitch + i);
            float2 p = __fadd2_rn(make_float2(v.x, v.y), nu), o = __fadd2_rn(make_float2(v.z, v.w), nu);
            if (i + 4 > w) {  // places past the last warp hold no mean
                p.y = i + 1 < w ? p.y : 0.0f;
                o.x = i + 2 < w ? o.x : 0.0f;
                o.y = 0.0f;
            }
            all = __fadd2_rn(all, __fadd2_rn(make_float2(q4.x, q4.y), make_float2(q4.z, q4.w)));
            all = __ffma2_rn(__fmul2_rn(p, p), count, all);
            all = __ffma2_rn(__fmul2_rn(o, o), count, all);
        }
#pragma unroll
        for (int i = 0; i < E / 2; ++i)
            x[i] = __fadd2_rn(x[i], nu);
        return make_float2(mu, all.x + all.y);
    }
};

} // namespace rows
} // namespace f8
