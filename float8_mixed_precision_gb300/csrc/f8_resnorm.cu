// The residual stream between two blocks: a block's output normed, gated and added
// to the scaled stream, and the norm in front of the next block; with its backward
// pass and every parameter's gradient.
//
//   forward   u = norm_post(a), r' = scale r + g u, y = norm_pre(r')
//   backward  D = dr' + s2 (dy w2 - mean(dy w2) - e2 mean(dy w2 e2)), dr = scale D,
//             du = g D, da = s1 (du w1 - mean(du w1) - e1 mean(du w1 e1)),
//             dw2 = sum dy e2, db2 = sum dy, dw1 = sum du e1, db1 = sum du,
//             dg = sum over the gate's rows of D u
//
// Everything between the loads and the stores is fp32.  Sums over rows: rows are cut
// into chunks; a chunk leaves one partial row of each parameter's gradient, writes
// the gate gradients whose rows it has whole, and leaves partial rows for the gates
// of its first and last rows where those reach into other chunks.  Partial rows are
// added in order by a kernel of its own.  No atomics: equal inputs give equal bits.
//
// Both are bound by HBM: four values moved per element forward, six backward.  A row's
// values stay in registers between the loads and the stores, 16 a thread forward and 8
// backward (beside four column sums and two parameters), and rows come some ahead through
// shared memory by bulk copies (f8_resnorm_rows.cuh); with the rows read again for each
// reduction 8192 x 4096 took 327 us forward and 482 backward.  What is left is the
// arithmetic, some 600 instructions a warp and row forward, with two rows in work an SM.
//
// Measured, bf16: 8192 x 4096 layer norm forward, gates of 1024 rows, 60 us, 4.5 TB/s;
// RMS norm backward with every gradient 79 us, 5.1 TB/s, with one gate for all rows, and 82
// with gates of 1024; a plain copy runs at 6.8.  1999 x 5003 with an fp32 stream, layer
// norms and gates of 250 rows, backward, 71 us of 26.5 for the bytes: one row is in work an
// SM, and where 8 does not divide the width, of a unit's every eighth row.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <iterator>
#include <mutex>
#include <type_traits>

#include "f8_internal.h"
#include "f8_ptx.cuh"
#include "f8_resnorm_rows.cuh"

namespace f8 {
namespace {

constexpr int kWalkThreads = 512;

__device__ __forceinline__ float elem(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ float elem(const float *p) { return *p; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float f) { *p = __float2bfloat16_rn(f); }
__device__ __forceinline__ void put(float *p, float f) { *p = f; }

// One parameter value of n, bf16 or fp32.
__device__ __forceinline__ float param(const void *p, int f32, int64_t i, int64_t n, unsigned *status)
{
    if (!in_range(i, 1, n, status))
        return 0.0f;
    return f32 ? static_cast<const float *>(p)[i]
               : __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

__device__ __forceinline__ void put_param(void *p, int f32, int64_t i, float v, int64_t n, unsigned *status)
{
    if (!in_range(i, 1, n, status))
        return;
    if (f32)
        static_cast<float *>(p)[i] = v;
    else
        static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

// What both passes know of the call.
struct Call {
    int layer;           // layer norm (else RMS norm)
    int w_f32, g_f32;
    int64_t rows, cols, gate_rows;
    float eps, scale;
    const void *w_pre, *b_pre, *w_post, *b_post, *gate;
    float *stats;        // [4][rows]: mean and 1/deviation of a, then of r'

    __device__ __forceinline__ float stat(int which, int64_t row, unsigned *status) const
    {
        const int64_t i = which * rows + row;
        return in_range(i, 1, 4 * rows, status) ? stats[i] : 0.0f;
    }
    __device__ __forceinline__ void put_stat(int which, int64_t row, float v, unsigned *status) const
    {
        const int64_t i = which * rows + row;
        if (in_range(i, 1, 4 * rows, status))
            stats[i] = v;
    }
    // elements of the gates
    __device__ __forceinline__ int64_t gate_n() const
    {
        return gate != nullptr ? ((rows - 1) / gate_rows + 1) * cols : 0;
    }
};

// Sum over the block, in a fixed order; every thread gets it.  `red` has two halves
// used in turn, so one barrier a sum.
template <int THREADS>
struct BlockSum {
    float *red;  // [2][THREADS / 32]
    int half;

    __device__ __forceinline__ float operator()(float v)
    {
        constexpr int W = THREADS / 32;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        float *r = red + half * W;
        half ^= 1;
        if ((threadIdx.x & 31) == 0)
            r[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w)
            v += r[w];
        return v;
    }
};

// ------------------------------------------------------------ any width
// One block a row, which is walked once per reduction and once for the outputs.
template <typename TA, typename TR>
__global__ void __launch_bounds__(kWalkThreads)
fwd_walk_kernel(const Call c, const TA *a, const TR *r, TR *r_out, TA *y, unsigned *amax,
                unsigned *status)
{
    __shared__ float red[2 * kWalkThreads / 32];
    __shared__ unsigned blk;
    if (threadIdx.x == 0)
        blk = 0u;
    griddep_wait();
    griddep_launch_dependents();
    BlockSum<kWalkThreads> sum{red, 0};
    const float inv_c = 1.0f / static_cast<float>(c.cols);
    const int64_t total = c.rows * c.cols;
    unsigned m = 0u;
    for (int64_t row = blockIdx.x; row < c.rows; row += gridDim.x) {
        const int64_t at = row * c.cols;
        const int64_t gat = c.gate != nullptr ? row / c.gate_rows * c.cols : 0;
        float mu1 = 0.0f, s1 = 1.0f;
        if (c.w_post != nullptr) {
            float t = 0.0f;
            if (c.layer) {
                for (int64_t i = threadIdx.x; i < c.cols; i += kWalkThreads)
                    if (in_range(at + i, 1, total, status))
                        t += elem(a + at + i);
                mu1 = sum(t) * inv_c;
            }
            t = 0.0f;
            for (int64_t i = threadIdx.x; i < c.cols; i += kWalkThreads)
                if (in_range(at + i, 1, total, status)) {
                    const float d = elem(a + at + i) - mu1;
                    t = fmaf(d, d, t);
                }
            s1 = 1.0f / sqrtf(sum(t) * inv_c + c.eps);
        }
        auto stream = [&](int64_t i) {
            if (!in_range(at + i, 1, total, status))
                return 0.0f;
            float u = elem(a + at + i);
            if (c.w_post != nullptr) {
                u = (u - mu1) * s1 * param(c.w_post, c.w_f32, i, c.cols, status);
                if (c.b_post != nullptr)
                    u += param(c.b_post, c.w_f32, i, c.cols, status);
            }
            if (c.gate != nullptr)
                u *= param(c.gate, c.g_f32, gat + i, c.gate_n(), status);
            return fmaf(c.scale, elem(r + at + i), u);
        };
        float mu2 = 0.0f, t = 0.0f;
        if (c.layer) {
            for (int64_t i = threadIdx.x; i < c.cols; i += kWalkThreads)
                t += stream(i);
            mu2 = sum(t) * inv_c;
        }
        t = 0.0f;
        for (int64_t i = threadIdx.x; i < c.cols; i += kWalkThreads) {
            const float d = stream(i) - mu2;
            t = fmaf(d, d, t);
        }
        const float s2 = 1.0f / sqrtf(sum(t) * inv_c + c.eps);
        // a thread reads its own columns only, so r_out may be r and y may be a
        for (int64_t i = threadIdx.x; i < c.cols; i += kWalkThreads) {
            const float v = stream(i);
            float o = (v - mu2) * s2 * param(c.w_pre, c.w_f32, i, c.cols, status);
            if (c.b_pre != nullptr)
                o += param(c.b_pre, c.w_f32, i, c.cols, status);
            if (!in_range(at + i, 1, total, status))
                continue;
            put(r_out + at + i, v);
            put(y + at + i, o);
            if constexpr (sizeof(TA) == 2)
                m = max(m, static_cast<unsigned>(__bfloat16_as_ushort(y[at + i])) & 0x7FFFu);
        }
        if (threadIdx.x == 0) {
            if (c.w_post != nullptr) {
                if (c.layer)
                    c.put_stat(0, row, mu1, status);
                c.put_stat(1, row, s1, status);
            }
            if (c.layer)
                c.put_stat(2, row, mu2, status);
            c.put_stat(3, row, s2, status);
        }
    }
    if (amax != nullptr) {
        __syncthreads();
        m = __reduce_max_sync(0xFFFFFFFFu, m);
        if ((threadIdx.x & 31) == 0)
            atomicMax(&blk, m);
        __syncthreads();
        if (threadIdx.x == 0) {
            if (blk >= 0x7F80u)
                atomicOr(status, kStatusNonfinite);
            atomicMax(amax, blk << 16);  // the maximum does not depend on the order
        }
    }
}

// D = dr' + s2 g - s2 mean(g) - e2 s2 mean(g e2) of one element, g = dy w2, from the
// row's k1 = -s2 mean(g e2) and k2 = -s2 mean(g).
__device__ __forceinline__ float stream_grad(float dr, float g, float e2, float s2, float k1, float k2)
{
    return dr + fmaf(g, s2, fmaf(e2, k1, k2));
}

template <typename TA, typename TR>
__global__ void __launch_bounds__(kWalkThreads)
bwd_walk_kernel(const Call c, const TA *__restrict__ dy, const TR *__restrict__ dr_out,
                const TA *__restrict__ a, const TR *__restrict__ r_out, TA *__restrict__ da,
                TR *__restrict__ dr, float *__restrict__ consts, unsigned *status)
{
    __shared__ float red[2 * kWalkThreads / 32];
    griddep_wait();
    griddep_launch_dependents();
    BlockSum<kWalkThreads> sum{red, 0};
    const float inv_c = 1.0f / static_cast<float>(c.cols);
    const int64_t total = c.rows * c.cols;
    const bool post = c.w_post != nullptr;
    for (int64_t row = blockIdx.x; row < c.rows; row += gridDim.x) {
        const int64_t at = row * c.cols;
        const int64_t gat = c.gate != nullptr ? row / c.gate_rows * c.cols : 0;
        const float mu1 = post && c.layer ? c.stat(0, row, status) : 0.0f;
        const float s1 = post ? c.stat(1, row, status) : 1.0f;
        const float mu2 = c.layer ? c.stat(2, row, status) : 0.0f;
        const float s2 = c.stat(3, row, status);
        float t1 = 0.0f, t2 = 0.0f;
        for (int64_t i = threadIdx.x; i < c.cols; i += kWalkThreads)
            if (in_range(at + i, 1, total, status)) {
                const float g = elem(dy + at + i) * param(c.w_pre, c.w_f32, i, c.cols, status);
                t1 = fmaf(g, (elem(r_out + at + i) - mu2) * s2, t1);
                t2 += g;
            }
        const float k1 = -s2 * (sum(t1) * inv_c);
        const float k2 = c.layer ? -s2 * (sum(t2) * inv_c) : 0.0f;
        auto grad = [&](int64_t i) {
            return stream_grad(dr_out != nullptr ? elem(dr_out + at + i) : 0.0f,
                               elem(dy + at + i) * param(c.w_pre, c.w_f32, i, c.cols, status),
                               (elem(r_out + at + i) - mu2) * s2, s2, k1, k2);
        };
        float d1 = 0.0f, d2 = 0.0f;
        if (post) {
            t1 = t2 = 0.0f;
            for (int64_t i = threadIdx.x; i < c.cols; i += kWalkThreads)
                if (in_range(at + i, 1, total, status)) {
                    float h = grad(i) * param(c.w_post, c.w_f32, i, c.cols, status);
                    if (c.gate != nullptr)
                        h *= param(c.gate, c.g_f32, gat + i, c.gate_n(), status);
                    t1 = fmaf(h, (elem(a + at + i) - mu1) * s1, t1);
                    t2 += h;
                }
            d1 = sum(t1) * inv_c;
            d2 = c.layer ? sum(t2) * inv_c : 0.0f;
        }
        for (int64_t i = threadIdx.x; i < c.cols; i += kWalkThreads) {
            if (!in_range(at + i, 1, total, status))
                continue;
            const float d = grad(i);
            if (dr != nullptr)
                put(dr + at + i, c.scale * d);
            if (da == nullptr)
                continue;
            float h = c.gate != nullptr ? d * param(c.gate, c.g_f32, gat + i, c.gate_n(), status) : d;
            if (post) {
                const float e1 = (elem(a + at + i) - mu1) * s1;
                h = s1 * (fmaf(-e1, d1, h * param(c.w_post, c.w_f32, i, c.cols, status)) - d2);
            }
            put(da + at + i, h);
        }
        if (threadIdx.x == 0 && consts != nullptr && in_range(c.rows + row, 1, 2 * c.rows, status)) {
            consts[row] = k1;
            consts[c.rows + row] = k2;
        }
    }
}

// ------------------------------------------------------------ rows in registers
// A block keeps its row, or its slice of a row that a cluster shares, in registers,
// and rows come some ahead through shared memory.
using rows::Param;
constexpr int kFwdE = 16, kBwdE = 8;  // columns of a thread
constexpr int kThreads = 512;         // of a block at most, but for wide_block()'s

__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }

__device__ __forceinline__ rows::Slice slice_of(int64_t cols, int per, uint32_t rank)
{
    rows::Slice s;
    s.first = per * static_cast<int>(rank);
    s.n = max(0, min(per, static_cast<int>(cols) - s.first));
    return s;
}

// The rows of a unit: every one of a chunk's, or (kShift) every eighth, eight units
// sharing a chunk of a multiple of eight rows.
template <int MODE>
struct Walk {
    static constexpr int kStep = MODE == rows::kShift ? 8 : 1;
    int64_t chunk;  // number
    int64_t first, stop;
    int shift;
    __device__ __forceinline__ Walk(int64_t unit, int64_t rows_of_chunk, int64_t rows, int64_t cols)
    {
        chunk = unit / kStep;
        first = chunk * rows_of_chunk + unit % kStep;
        stop = min((chunk + 1) * rows_of_chunk, rows);
        shift = MODE == rows::kShift ? static_cast<int>((first * cols) & 7) : 0;
    }
    // columns, or the positions that hold them in whole vectors
    __device__ __forceinline__ int64_t width(int64_t cols) const
    {
        return MODE == rows::kShift ? (shift + cols + 7) & ~int64_t{7} : cols;
    }
};

// Mean (0 without `layer`) and 1/deviation of the row; x becomes x - mean.
template <int MODE, int E>
__device__ __forceinline__ void row_stats(float2 (&x)[E / 2], const rows::Place<MODE, E> &pl, bool layer, float inv_c, float eps,
                                          rows::Sum<MODE> &sum, float &mu, float &rstd)
{
    mu = 0.0f;
    if (MODE == rows::kFull && layer) {
        const float2 m = sum.template moments<E>(x, 32.0f * E * inv_c);  // 1 / warps
        mu = m.x;
        rstd = rsqrtf(m.y * inv_c + eps);
        return;
    }
    if (layer) {
        float2 s = x[0];
#pragma unroll
        for (int i = 1; i < E / 2; ++i)
            s = __fadd2_rn(s, x[i]);
        mu = sum(s.x + s.y) * inv_c;
#pragma unroll
        for (int i = 0; i < E / 2; ++i)
            x[i] = __fadd2_rn(x[i], splat(-mu));
    }
    float2 q = splat(0.0f);
    // places past the slice are -mean and do not count
    [[maybe_unused]] const int n = pl.n;
    if constexpr (MODE == rows::kShift) {
        if (layer)
            rows::mask<E>(pl, x);
#pragma unroll
        for (int i = 0; i < E / 2; ++i)
            q = __ffma2_rn(x[i], x[i], q);
    } else if constexpr (MODE != rows::kRagged) {
#pragma unroll
        for (int u = 0; u < E / 8; ++u)
            if (rows::vec_in<MODE>(rows::vec_col(u), n)) {
#pragma unroll
                for (int i = 4 * u; i < 4 * u + 4; ++i)
                    q = __ffma2_rn(x[i], x[i], q);
            }
    } else {
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            if (rows::elem_col(2 * i) < n)
                q.x = fmaf(x[i].x, x[i].x, q.x);
            if (rows::elem_col(2 * i + 1) < n)
                q.y = fmaf(x[i].y, x[i].y, q.y);
        }
    }
    rstd = rsqrtf(sum(q.x + q.y) * inv_c + eps);
}

// The checked build's test of a row's slice: of kShift's, whose first and last vectors
// are shared with other rows, the part that is the tensor's.
template <int MODE>
__device__ __forceinline__ bool inside_of(int64_t at, int n, int64_t total, unsigned *status)
{
    return in_range(at, MODE == rows::kShift ? min(static_cast<int64_t>(n), total - at) : n, total, status);
}

__device__ __forceinline__ void zero_sums(float *red)
{
    for (int i = threadIdx.x; i < rows::kSumFloats; i += blockDim.x)
        red[i] = 0.0f;
}

// A unit (a block, or a cluster by column slices) walks the rows [unit chunk, (unit +
// 1) chunk).  BF: all parameters are bf16 and stay in registers over the rows; fp32
// ones are read again for each row, from L1.
template <typename TA, typename TR, int MODE, bool BF, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS < kThreads ? 2 : 1)
fwd_kernel(const Call c, const TA *a, const TR *r, TR *r_out, TA *y, unsigned *amax, int64_t chunk,
           int ranks, int slice, int stages, uint64_t limit_ns, unsigned *status)
{
    constexpr int E = kFwdE, P = E / 2;
    extern __shared__ __align__(16) uint8_t dyn[];
    __shared__ __align__(16) float red[rows::kSumFloats];
    __shared__ __align__(8) uint64_t full[rows::kMaxStages], meets[2];
    __shared__ unsigned blk;
    const uint32_t rank = MODE != rows::kFull && ranks > 1 ? cluster_ctarank() : 0u;
    const Walk<MODE> walk(blockIdx.x / ranks, chunk, c.rows, c.cols);
    constexpr int kStep = Walk<MODE>::kStep;
    const int64_t first = walk.first, stop = walk.stop;
    const rows::Slice sl = slice_of(walk.width(c.cols), slice, rank);
    rows::Place<MODE, E> pl;
    pl.set(sl.first, sl.n, walk.shift, static_cast<int>(c.cols));
    rows::Slots<TA, 1, TR, 1, MODE> slots;
    slots.start(dyn, full, stages, c.cols, c.rows, sl, walk.shift, status);
    slots.a[0] = a;
    slots.r[0] = r;
    zero_sums(red);
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i)
            mbar_init(&full[i], 1);
        mbar_init(&meets[0], 1);
        mbar_init(&meets[1], 1);
        fence_mbar_init();
        blk = 0u;
    }
    griddep_wait();
    griddep_launch_dependents();
    if (MODE != rows::kFull && ranks > 1)
        cluster_sync();  // a peer's part of a sum may come from here on
    else
        __syncthreads();
    if (threadIdx.x == 0)
        for (int i = 0; i < stages && first + i * kStep < stop; ++i)
            slots.fill(first + i * kStep);
    rows::Sum<MODE> sum;
    sum.start(red, meets, rank, static_cast<uint32_t>(ranks), limit_ns, status);
    const float inv_c = 1.0f / static_cast<float>(c.cols);
    const bool post = c.w_post != nullptr, gated = c.gate != nullptr, layer = c.layer != 0;
    Param<E, BF> w1, b1, g, w2, b2;
    if (BF) {
        rows::take_param<MODE>(c.w_post, 0, 0, pl, 1.0f, w1, c.cols, status);
        rows::take_param<MODE>(c.b_post, 0, 0, pl, 0.0f, b1, c.cols, status);
        rows::take_param<MODE>(c.w_pre, 0, 0, pl, 1.0f, w2, c.cols, status);
        rows::take_param<MODE>(c.b_pre, 0, 0, pl, 0.0f, b2, c.cols, status);
    }
    int64_t gate = gated ? first / c.gate_rows : 0;
    int64_t gate_end = gated ? first : stop, gate_at = 0;
    uint32_t m2 = 0u;
    int64_t at = slots.begin(first);
    rows::Cursor cur = slots.first();
    for (int64_t row = first; row < stop; row += kStep, at += kStep * c.cols) {
        if (gated && row >= gate_end) {
            gate = MODE == rows::kShift ? row / c.gate_rows : gate;
            if (BF)
                rows::take_param<MODE>(c.gate, 0, gate * c.cols, pl, 1.0f, g, c.gate_n(), status);
            gate_at = gate * c.cols;
            ++gate;
            gate_end = min(stop, gate * c.gate_rows);  // within rows + gate_rows
        }
        slots.wait(cur, limit_ns, status);
        int sa = 0, sr = 0;
        if constexpr (MODE == rows::kRagged)
            slots.ragged(cur, row, sa, sr);
        if constexpr (MODE == rows::kShift)
            slots.tail(cur, row);
        float2 x[P], v[P];
        rows::take<MODE, E, TA>(slots.at_a(cur, 0), sa, pl, x);
        float mu1 = 0.0f, s1 = 1.0f;
        if (post) {
            row_stats<MODE, E>(x, pl, layer, inv_c, c.eps, sum, mu1, s1);
            if (!BF)
                rows::take_param<MODE>(c.w_post, c.w_f32, 0, pl, 1.0f, w1, c.cols, status);
            if (!BF)
                rows::take_param<MODE>(c.b_post, c.w_f32, 0, pl, 0.0f, b1, c.cols, status);
#pragma unroll
            for (int i = 0; i < P; ++i)
                x[i] = __ffma2_rn(__fmul2_rn(x[i], splat(s1)), w1.pair(i), b1.pair(i));
        }
        if (gated) {
            if (!BF)
                rows::take_param<MODE>(c.gate, c.g_f32, gate_at, pl, 1.0f, g, c.gate_n(), status);
#pragma unroll
            for (int i = 0; i < P; ++i)
                x[i] = __fmul2_rn(x[i], g.pair(i));
        }
        rows::take<MODE, E, TR>(slots.at_r(cur, 0), sr, pl, v);
#pragma unroll
        for (int i = 0; i < P; ++i)
            x[i] = __ffma2_rn(v[i], splat(c.scale), x[i]);
        const bool inside = inside_of<MODE>(at, sl.n, c.rows * c.cols, status);
        if (inside)
            rows::give<MODE, E>(r_out + at, pl, x);
        float mu2, s2;
        row_stats<MODE, E>(x, pl, layer, inv_c, c.eps, sum, mu2, s2);
        // every thread has taken its columns: the slot may be filled again
        if (threadIdx.x == 0) {
            if (slots.ok && row + stages * kStep < stop)
                slots.fill(row + stages * kStep);
            if (rank == 0) {
                if (post) {
                    if (layer)
                        c.put_stat(0, row, mu1, status);
                    c.put_stat(1, row, s1, status);
                }
                if (layer)
                    c.put_stat(2, row, mu2, status);
                c.put_stat(3, row, s2, status);
            }
        }
        if (!BF)
            rows::take_param<MODE>(c.w_pre, c.w_f32, 0, pl, 1.0f, w2, c.cols, status);
        if (!BF)
            rows::take_param<MODE>(c.b_pre, c.w_f32, 0, pl, 0.0f, b2, c.cols, status);
#pragma unroll
        for (int i = 0; i < P; ++i)
            x[i] = __ffma2_rn(__fmul2_rn(x[i], splat(s2)), w2.pair(i), b2.pair(i));
        if (inside)
            rows::give<MODE, E>(y + at, pl, x, amax != nullptr ? &m2 : nullptr);
        slots.step(cur);
    }
    if (threadIdx.x == 0)
        slots.drain();
    if (amax != nullptr) {
        const unsigned m = __reduce_max_sync(0xFFFFFFFFu, max(m2 & 0xFFFFu, m2 >> 16));
        if ((threadIdx.x & 31) == 0)
            atomicMax(&blk, m);
        __syncthreads();
        if (threadIdx.x == 0) {
            if (blk >= 0x7F80u)
                atomicOr(status, kStatusNonfinite);
            atomicMax(amax, blk << 16);  // the maximum does not depend on the order
        }
    }
    if (MODE != rows::kFull && ranks > 1)
        cluster_sync();  // a peer may still write its part of a sum here
}

// ------------------------------------------------------------ sums over rows
// The gates of a chunk of rows [first, stop): a gate's rows may reach into other
// chunks only at the chunk's ends.
struct Chunks {
    int64_t rows, gate_rows, chunk;
    int64_t room;  // units that the workspace has partial rows for
    __host__ __device__ int64_t first(int64_t i) const { return i * chunk; }
    __host__ __device__ int64_t stop(int64_t i) const
    {
        const int64_t e = (i + 1) * chunk;
        return e < rows ? e : rows;
    }
    __host__ __device__ int64_t gate(int64_t row) const { return row / gate_rows; }
    __host__ __device__ int64_t gate_first(int64_t g) const { return g * gate_rows; }
    __host__ __device__ int64_t gate_stop(int64_t g) const
    {
        return gate_rows >= rows - g * gate_rows ? rows : (g + 1) * gate_rows;
    }
    // whether gate g's rows all lie in chunk i, and which of the chunk's two partial
    // rows takes them where they do not
    __host__ __device__ bool whole(int64_t g, int64_t i) const
    {
        return gate_first(g) >= first(i) && gate_stop(g) <= stop(i);
    }
    __host__ __device__ int slot(int64_t g, int64_t i) const { return gate(first(i)) == g ? 0 : 1; }
};

// Block (x, y): 256 columns, chunk y.  parts: [chunks][4][cols] of dw_pre, db_pre,
// dw_post, db_post; ends: [chunks][2][cols] of dgate.
template <typename TA, typename TR>
__global__ void __launch_bounds__(256)
cols_walk_kernel(const Call c, const Chunks ch, const TA *__restrict__ dy, const TR *__restrict__ dr_out,
                 const TA *__restrict__ a, const TR *__restrict__ r_out,
                 const float *__restrict__ consts, float *__restrict__ parts, float *__restrict__ ends,
                 void *__restrict__ dgate, unsigned *status)
{
    griddep_wait();
    griddep_launch_dependents();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= c.cols)
        return;
    const int64_t chunk = blockIdx.y, first = ch.first(chunk), stop = ch.stop(chunk);
    const int64_t total = c.rows * c.cols;
    const bool post = c.w_post != nullptr, gated = c.gate != nullptr;
    const float w2 = param(c.w_pre, c.w_f32, i, c.cols, status);
    const float w1 = post ? param(c.w_post, c.w_f32, i, c.cols, status) : 1.0f;
    const float b1 = c.b_post != nullptr ? param(c.b_post, c.w_f32, i, c.cols, status) : 0.0f;
    float dw2 = 0.0f, db2 = 0.0f, dw1 = 0.0f, db1 = 0.0f;
    for (int64_t row = first; row < stop;) {
        // rows of one gate: S = sum D e1, T = sum D
        const int64_t g = gated ? ch.gate(row) : 0;
        const int64_t end = gated ? min(stop, ch.gate_stop(g)) : stop;
        float S = 0.0f, T = 0.0f;
        for (; row < end; ++row) {
            const int64_t at = row * c.cols + i;
            if (!in_range(at, 1, total, status) || !in_range(c.rows + row, 1, 2 * c.rows, status))
                continue;
            const float mu1 = post && c.layer ? c.stat(0, row, status) : 0.0f;
            const float s1 = post ? c.stat(1, row, status) : 1.0f;
            const float mu2 = c.layer ? c.stat(2, row, status) : 0.0f;
            const float s2 = c.stat(3, row, status);
            const float v = elem(dy + at), e2 = (elem(r_out + at) - mu2) * s2;
            const float d = stream_grad(dr_out != nullptr ? elem(dr_out + at) : 0.0f, v * w2, e2, s2,
                                        consts[row], consts[c.rows + row]);
            const float e1 = (elem(a + at) - mu1) * s1;
            dw2 = fmaf(v, e2, dw2);
            db2 += v;
            S = fmaf(d, e1, S);
            T += d;
        }
        const float gate = gated ? param(c.gate, c.g_f32, g * c.cols + i, c.gate_n(), status) : 1.0f;
        dw1 = fmaf(gate, S, dw1);
        db1 = fmaf(gate, T, db1);
        if (dgate != nullptr) {
            const float dg = fmaf(S, w1, T * b1);
            const int64_t end_at = (chunk * 2 + ch.slot(g, chunk)) * c.cols + i;
            if (ch.whole(g, chunk))
                put_param(dgate, c.g_f32, g * c.cols + i, dg, c.gate_n(), status);
            else if (in_range(end_at, 1, 2 * ch.room * c.cols, status))
                ends[end_at] = dg;
        }
    }
    if (!in_range(chunk * 4 * c.cols + i, 3 * c.cols + 1, 4 * ch.room * c.cols, status))
        return;
    float *p = parts + chunk * 4 * c.cols + i;
    p[0] = dw2;
    p[c.cols] = db2;
    p[2 * c.cols] = dw1;
    p[3 * c.cols] = db1;
}

// The backward pass in one: a unit (a block, or a cluster by column slices) walks the
// chunk `unit` of rows, with the column sums of all gradients in registers.  FULL:
// with means or biases; without, the sums that only those need are left out.
// Of a gate's rows only S = sum D e1 and T = sum D are kept: they give dgate = w1 S + b1 T,
// and g S and g T for dw1 and db1, whose sums over several gates lie in shared memory.
// With u formed for each row and its three sums, five parameters' columns and five sums
// a thread, 8192 x 4999 layer norm took 214 us against 195.
template <typename TA, typename TR, int MODE, bool FULL, int THREADS>
__global__ void __launch_bounds__(THREADS, 1)
bwd_kernel(const Call c, const Chunks ch, const TA *__restrict__ dy, const TR *__restrict__ dr_out,
           const TA *__restrict__ a, const TR *__restrict__ r_out, TA *__restrict__ da,
           TR *__restrict__ dr, float *__restrict__ parts, float *__restrict__ ends,
           void *__restrict__ dgate, int ranks, int slice, int stages, uint64_t limit_ns, unsigned *status)
{
    constexpr int E = kBwdE, P = E / 2;
    extern __shared__ __align__(16) uint8_t dyn[];
    __shared__ __align__(16) float red[rows::kSumFloats];
    __shared__ __align__(8) uint64_t full[rows::kMaxStages], meets[2];
    const uint32_t rank = MODE != rows::kFull && ranks > 1 ? cluster_ctarank() : 0u;
    const int64_t unit = blockIdx.x / ranks;
    const Walk<MODE> walk(unit, ch.chunk, c.rows, c.cols);
    constexpr int kStep = Walk<MODE>::kStep;
    const int64_t first = walk.first, stop = walk.stop;
    const rows::Slice sl = slice_of(walk.width(c.cols), slice, rank);
    rows::Place<MODE, E> pl;
    pl.set(sl.first, sl.n, walk.shift, static_cast<int>(c.cols));
    rows::Slots<TA, 2, TR, 2, MODE> slots;
    slots.start(dyn, full, stages, c.cols, c.rows, sl, walk.shift, status);
    slots.a[0] = dy;
    slots.a[1] = a;
    slots.r[0] = dr_out;
    slots.r[1] = r_out;
    zero_sums(red);
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i)
            mbar_init(&full[i], 1);
        mbar_init(&meets[0], 1);
        mbar_init(&meets[1], 1);
        fence_mbar_init();
    }
    griddep_wait();
    griddep_launch_dependents();
    if (MODE != rows::kFull && ranks > 1)
        cluster_sync();
    else
        __syncthreads();
    if (threadIdx.x == 0)
        for (int64_t i = 0; i < stages && first + i * kStep < stop; ++i)
            slots.fill(first + i * kStep);
    rows::Sum<MODE> sum;
    sum.start(red, meets, rank, static_cast<uint32_t>(ranks), limit_ns, status);
    const float inv_c = 1.0f / static_cast<float>(c.cols);
    const bool post = c.w_post != nullptr, layer = FULL && c.layer;
    float2 *acc = reinterpret_cast<float2 *>(dyn + stages * slots.slot_bytes()) + threadIdx.x;
    auto acc_at = [&](int i) -> float2 & { return acc[i * blockDim.x]; };
    const int64_t pitch = rows::sums_pitch(c.cols);
    const int64_t parts_n = 4 * ch.room * pitch, ends_n = 2 * ch.room * pitch, mine = unit * 4 * pitch;
    Param<E, false> w2, gw;  // gw: gate w1
    rows::take_param<MODE>(c.w_pre, c.w_f32, 0, pl, 1.0f, w2, c.cols, status);
    float2 dw2[P], db2[P], S[P], T[P];
#pragma unroll
    for (int i = 0; i < P; ++i)
        dw2[i] = db2[i] = S[i] = T[i] = splat(0.0f);
    int64_t gate = 0, gate_end = first;
    bool begun = false;  // acc holds sums
    // What a gate's rows of this unit have given, into place.  Units of kShift share
    // their chunk's gates, of which there are at most two.
    int left = 0;  // which of the unit's two partial rows are written
    auto close = [&](bool last) {
        Param<E, false> w;
        float2 v[P];
        if (dgate != nullptr) {
            rows::take_param<MODE>(c.w_post, c.w_f32, 0, pl, 1.0f, w, c.cols, status);
#pragma unroll
            for (int i = 0; i < P; ++i)
                v[i] = __fmul2_rn(S[i], w.pair(i));
            if (FULL) {
                rows::take_param<MODE>(c.b_post, c.w_f32, 0, pl, 0.0f, w, c.cols, status);
#pragma unroll
                for (int i = 0; i < P; ++i)
                    v[i] = __ffma2_rn(T[i], w.pair(i), v[i]);
            }
            bool whole = false;
            if constexpr (MODE != rows::kShift) {
                whole = ch.whole(gate, walk.chunk);
                if (whole)
                    rows::give_param<MODE, E>(dgate, c.g_f32, gate * c.cols, pl, v, c.gate_n(), status);
            }
            if (!whole) {
                const int to = ch.slot(gate, walk.chunk);
                left |= 1 << to;
                rows::give_sums<MODE, E>(ends, (unit * 2 + to) * pitch, ends_n, pl, v, status);
            }
        }
        rows::take_param<MODE>(c.gate, c.g_f32, gate * c.cols, pl, 1.0f, w, c.gate_n(), status);
        auto join = [&](float2 (&of)[P], int at, int row) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                v[i] = __ffma2_rn(of[i], w.pair(i), begun ? acc_at(at + i) : splat(0.0f));
                if (!last)
                    acc_at(at + i) = v[i];
                of[i] = splat(0.0f);
            }
            if (last)
                rows::give_sums<MODE, E>(parts, mine + row * pitch, parts_n, pl, v, status);
        };
        join(S, 0, 2);
        if (FULL)
            join(T, P, 3);
        begun = true;
    };
    // statistics of the row in phase two, of the one in phase one, and of the one after
    // that, which are on their way
    struct Stats {
        float mu1, s1, mu2, s2;
    };
    auto stats_of = [&](int64_t row) {
        Stats v{0.0f, 1.0f, 0.0f, 0.0f};
        if (row >= stop)
            return v;
        if (post) {
            v.s1 = c.stat(1, row, status);
            if (layer)
                v.mu1 = c.stat(0, row, status);
        }
        v.s2 = c.stat(3, row, status);
        if (layer)
            v.mu2 = c.stat(2, row, status);
        return v;
    };
    Stats now, soon = stats_of(first), later = stats_of(first + kStep);
    rows::Cursor cur = slots.first(), ahead = cur;
    int sa = 0, sr = 0, next_sa = 0, next_sr = 0;
    // A row's two sums depend on one another.  An exchange carries the second sum of a row
    // and the first one of the next; phase two forms phase one's values again from the slot.
    // With an exchange for each and the values kept, 8192 x 5120 layer norm took 141 us
    // against 130, 8192 x 4096 109 against 103, 1999 x 8192 over clusters 95 against 80.
    // Phase one of a row: the sums that D needs, and the gradients of w2 and b2.
    auto one = [&](int64_t row, const Stats &v) {
        slots.wait(ahead, limit_ns, status);
        if constexpr (MODE == rows::kRagged)
            slots.ragged(ahead, row, next_sa, next_sr);
        if constexpr (MODE == rows::kShift)
            slots.tail(ahead, row);
        float2 h[P], e[P];
        rows::take<MODE, E, TA>(slots.at_a(ahead, 0), next_sa, pl, h);
        rows::take<MODE, E, TR>(slots.at_r(ahead, 1), next_sr, pl, e);
        float2 t1 = splat(0.0f), t2 = splat(0.0f);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            e[i] = __fmul2_rn(__fadd2_rn(e[i], splat(-v.mu2)), splat(v.s2));
            dw2[i] = __ffma2_rn(h[i], e[i], dw2[i]);
            if (FULL)
                db2[i] = __fadd2_rn(db2[i], h[i]);
            h[i] = __fmul2_rn(h[i], w2.pair(i));
            t1 = __ffma2_rn(h[i], e[i], t1);
            if (FULL)
                t2 = __fadd2_rn(t2, h[i]);
        }
        slots.step(ahead);
        return make_float2(t1.x + t1.y, t2.x + t2.y);
    };
    float k1 = 0.0f, k2 = 0.0f;
    auto means = [&](float x, float y, const Stats &v) {
        k1 = -v.s2 * (x * inv_c);
        k2 = layer ? -v.s2 * (y * inv_c) : 0.0f;
    };
    if (first < stop) {
        const float2 t = one(first, soon), k = FULL ? sum(t.x, t.y) : make_float2(sum(t.x), 0.0f);
        means(k.x, k.y, soon);
    }
    int64_t at = slots.begin(first);
    for (int64_t row = first; row < stop; row += kStep, at += kStep * c.cols) {
        if (row >= gate_end) {
            gate = ch.gate(row);
            gate_end = min(stop, ch.gate_stop(gate));
            Param<E, false> g;
            rows::take_param<MODE>(c.w_post, c.w_f32, 0, pl, 1.0f, gw, c.cols, status);
            rows::take_param<MODE>(c.gate, c.g_f32, gate * c.cols, pl, 1.0f, g, c.gate_n(), status);
#pragma unroll
            for (int i = 0; i < P; ++i)
                gw.set(i, __fmul2_rn(gw.pair(i), g.pair(i)));
        }
        now = soon;
        soon = later;
        later = stats_of(row + 2 * kStep);
        sa = next_sa;
        sr = next_sr;
        // h becomes D
        float2 h[P], e[P], o[P];
        rows::take<MODE, E, TA>(slots.at_a(cur, 0), sa, pl, h);
        rows::take<MODE, E, TR>(slots.at_r(cur, 1), sr, pl, e);
        if (dr_out != nullptr) {
            rows::take<MODE, E, TR>(slots.at_r(cur, 0), sr, pl, o);
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i)
                o[i] = splat(0.0f);
        }
        const float s2k1 = now.s2 * k1;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            e[i] = __fadd2_rn(e[i], splat(-now.mu2));
            h[i] = __fmul2_rn(h[i], w2.pair(i));
            h[i] = __fadd2_rn(o[i], __ffma2_rn(h[i], splat(now.s2), __ffma2_rn(e[i], splat(s2k1), splat(k2))));
        }
        rows::take<MODE, E, TA>(slots.at_a(cur, 1), sa, pl, e);
        const bool inside = inside_of<MODE>(at, sl.n, c.rows * c.cols, status);
        if (dr != nullptr && inside) {
#pragma unroll
            for (int i = 0; i < P; ++i)
                o[i] = __fmul2_rn(h[i], splat(c.scale));
            rows::give<MODE, E>(dr + at, pl, o);
        }
        // e becomes e1 (a without the norm), h du w1
        float2 t1 = splat(0.0f), t2 = splat(0.0f);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            e[i] = __fmul2_rn(__fadd2_rn(e[i], splat(-now.mu1)), splat(now.s1));
            S[i] = __ffma2_rn(h[i], e[i], S[i]);
            if (FULL)
                T[i] = __fadd2_rn(T[i], h[i]);
            h[i] = __fmul2_rn(h[i], gw.pair(i));
            t1 = __ffma2_rn(h[i], e[i], t1);
            if (FULL)
                t2 = __fadd2_rn(t2, h[i]);
        }
        float2 k, t = make_float2(0.0f, 0.0f);
        if (row + kStep < stop)
            t = one(row + kStep, soon);
        if constexpr (FULL) {
            const float4 both = sum(t1.x + t1.y, t2.x + t2.y, t.x, t.y);
            k = make_float2(both.x, both.y);
            means(both.z, both.w, soon);
        } else {
            const float2 both = sum(t1.x + t1.y, t.x);
            k = make_float2(both.x, 0.0f);
            means(both.y, 0.0f, soon);
        }
        // every thread is done with the row: its slot may be filled again
        if (threadIdx.x == 0 && slots.ok && row + stages * kStep < stop)
            slots.fill(row + stages * kStep);
        if (post) {
            const float d1 = -now.s1 * (k.x * inv_c), d2 = layer ? -now.s1 * (k.y * inv_c) : 0.0f;
#pragma unroll
            for (int i = 0; i < P; ++i)
                h[i] = __ffma2_rn(h[i], splat(now.s1), __ffma2_rn(e[i], splat(d1), splat(d2)));
        }
        if (da != nullptr && inside)
            rows::give<MODE, E>(da + at, pl, h);
        slots.step(cur);
        if (row + kStep >= gate_end)
            close(row + kStep >= stop);
    }
    if (first >= stop) {
        rows::give_sums<MODE, E>(parts, mine + 2 * pitch, parts_n, pl, S, status);
        if (FULL)
            rows::give_sums<MODE, E>(parts, mine + 3 * pitch, parts_n, pl, T, status);
    }
    if (MODE == rows::kShift && dgate != nullptr) {
        // a unit without rows of one of them: close left zeros
        for (int to = 0; to < 2; ++to)
            if ((left & (1 << to)) == 0)
                rows::give_sums<MODE, E>(ends, (unit * 2 + to) * pitch, ends_n, pl, S, status);
    }
    rows::give_sums<MODE, E>(parts, mine, parts_n, pl, dw2, status);
    if (FULL)
        rows::give_sums<MODE, E>(parts, mine + pitch, parts_n, pl, db2, status);
    if (threadIdx.x == 0)
        slots.drain();
    if (MODE != rows::kFull && ranks > 1)
        cluster_sync();
}

// The gradients from the partial rows, in a fixed order: 32 columns a block, a lane
// each, and W warps that take every W-th row.  blockIdx.y names a parameter's
// gradient, or from 4 on gates whose rows may lie in several chunks: kEach's gate y - 4,
// kMany's W gates from W (y - 4) on, a warp each; kBorder's those that reach over the
// borders after the W chunks from W (y - 4) on.  What a chunk has whole it has written, unless
// its rows are shared by `units` (kShift), which all leave partial rows, by position: unit
// i's start `shift` i mod 8 floats in.  W is 8, or
// 32 where the parameters' blocks would not fill the GPU: 8192 x 4096 with 33 gates 105 us
// in all against 134, 16384 x 512 RMS norm with one gate 33.5 us against 37.5.
constexpr int kReduceWarps = 8, kReduceMost = 32;
enum GateSums { kEach, kMany, kBorder };
struct Sums {
    void *out[4];
    void *dgate;
    const float *parts, *ends;
    int nparts, w_f32, g_f32, units;
    GateSums by;
    int shift;
    int64_t cols, pitch, gates;
};

__global__ void __launch_bounds__(32 * kReduceMost)
reduce_kernel(const __grid_constant__ Sums a, const Chunks ch, unsigned *status)
{
    __shared__ float acc[kReduceMost][32];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, k = threadIdx.x >> 5, W = blockDim.x >> 5;
    const int64_t cols = a.cols, c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    void *out;
    int64_t at = 0;
    int f32 = a.w_f32;
    float s = 0.0f;
    if (blockIdx.y < 4) {
        out = a.out[blockIdx.y];
        if (out == nullptr)
            return;
        if (c < cols) {
            const float *p = a.parts + static_cast<int64_t>(blockIdx.y) * a.pitch + c;
#pragma unroll 8
            for (int i = k; i < a.nparts; i += W)
                if (in_range((4ll * i + blockIdx.y) * a.pitch + c + (i * a.shift & 7), 1, 4 * ch.room * a.pitch, status))
                    s += p[static_cast<int64_t>(i) * 4 * a.pitch + (i * a.shift & 7)];
        }
    } else {
        const int64_t y = blockIdx.y - 4;
        int64_t g = a.by == kEach ? y : y * W + k;
        if (a.by == kBorder) {
            // the gate over the border after chunk g, once: at the first that it reaches over
            const int64_t border = g;
            if (border + 1 >= a.nparts)
                return;
            g = ch.gate(ch.stop(border) - 1);
            if (ch.gate_first(g) / ch.chunk != border)
                return;
        }
        if (g >= a.gates)
            return;
        const int64_t first = ch.gate_first(g) / ch.chunk, last = (ch.gate_stop(g) - 1) / ch.chunk;
        if (a.units == 1 && first == last)
            return;
        out = a.dgate;
        at = g * cols;
        f32 = a.g_f32;
        // the gate comes first in every chunk but the one that it begins in
        const int64_t n = a.units, step = a.by == kEach ? W : 1;
        if (c < cols) {
            auto held = [&](const float *p, int64_t i) {
                return in_range(p - a.ends + i * 2 * a.pitch + (i * a.shift & 7), 1, 2 * ch.room * a.pitch, status);
            };
            const float *p = a.ends + (first * n * 2 + ch.slot(g, first)) * a.pitch + c;
#pragma unroll 8
            for (int64_t i = a.by == kEach ? k : 0; i < n; i += step)
                if (held(p, i))
                    s += p[i * 2 * a.pitch + (i * a.shift & 7)];
            p = a.ends + (first + 1) * n * 2 * a.pitch + c;
#pragma unroll 8
            for (int64_t i = a.by == kEach ? k : 0; i < (last - first) * n; i += step)
                if (held(p, i))
                    s += p[i * 2 * a.pitch + (i * a.shift & 7)];
        }
        if (a.by != kEach) {
            if (c < cols)
                put_param(out, f32, at + c, s, a.gates * cols, status);
            return;
        }
    }
    acc[k][lane] = s;
    __syncthreads();
    if (k > 0 || c >= cols)
        return;
#pragma unroll 4
    for (int i = 1; i < W; ++i)
        s += acc[i][lane];
    put_param(out, f32, at + c, s, blockIdx.y < 4 ? cols : a.gates * cols, status);
}

// ------------------------------------------------------------ launches
constexpr int kMaxChunks = 1024;
constexpr int64_t kRegCols = 16384;  // a cluster's registers hold no more

// Columns, or the positions that an odd width's rows reach into, a vector more than
// they fill.
int64_t width_of(int64_t cols) { return cols % 8 == 0 ? cols : cols + 7; }
bool in_registers(int64_t cols) { return width_of(cols) <= kRegCols; }
// Shared memory for a block's ring, of `per_sm` on an SM: beside it lie the sums' and
// bars' 2.7 KB, and the SM's own 1 KB.
constexpr int kRingBytes = 224 * 1024;
int ring_bytes(int per_sm) { return std::min(kRingBytes, (228 / per_sm - 4) * 1024); }

int64_t walk_chunks(int64_t rows, int64_t cols, int sms)
{
    const int64_t strips = (cols + 255) / 256;
    return std::max<int64_t>(1, std::min<int64_t>({(8ll * sms + strips - 1) / strips, (rows + 7) / 8,
                                                   kMaxChunks}));
}

// How rows are laid over the GPU: `ranks` blocks of `threads` to a row, `per_sm`
// blocks an SM.
struct Plan {
    int ranks, threads, per_sm, slice;
};

// 512 threads of 128 registers an SM, of `e` columns each, in blocks that hold a row's
// slice; slices of whole vectors, the last one perhaps shorter.
Plan plan_of(int64_t cols, int e, int most = kThreads)
{
    Plan p;
    p.ranks = 1;
    while (p.ranks * most * e < width_of(cols))
        p.ranks *= 2;
    const int64_t width = width_of(cols);
    p.slice = static_cast<int>((width + 8 * p.ranks - 1) / (8 * p.ranks)) * 8;
    p.threads = (p.slice + 32 * e - 1) / (32 * e) * 32;
    p.per_sm = std::max(1, std::min(16, most / p.threads));
    return p;
}


// Forward, rows of 4097 to 5120 columns go by two blocks of 320 threads an SM at 96
// registers, not one at 128: 8192 x 5120 layer norm 82 us against 109, RMS norm 66 against
// 72, 8192 x 4095 131 against 174 (some 5 us of each are the measuring's).  At 96 registers
// whole vectors' kernels spill 48 to 56 bytes, kShift's 176 to 264.
constexpr int kPairThreads = 320;
bool pair_blocks(int64_t cols)
{
    return width_of(cols) > kThreads / 2 * kFwdE && width_of(cols) <= kPairThreads * kFwdE;
}
Plan fwd_plan(int64_t cols)
{
    Plan p = plan_of(cols, kFwdE);
    if (pair_blocks(cols))
        p.per_sm = 2;
    return p;
}

// Backward, 640 threads of 96 registers an SM where 512 of 128 would hold one block
// little over half of them, or a row take a cluster: 8192 x 2560 layer norm 74 us against
// 93, 8192 x 2047 97 against 117, 8192 x 5120 130 against 213.  Elsewhere the registers
// are worth more: 8192 x 4096 103 us against 111, 8192 x 2048 62 against 68, 8192 x 1536
// (three blocks instead of two) 56 against 56 (some 5 us of each are the measuring's).
constexpr int kWideThreads = 640;
bool wide_block(int64_t cols)
{
    const int64_t threads = (width_of(cols) + kBwdE - 1) / kBwdE;
    return (threads > kThreads / 2 && threads <= kWideThreads / 2) ||
           (threads > kThreads && threads <= kWideThreads);
}
Plan bwd_plan(int64_t cols) { return plan_of(cols, kBwdE, wide_block(cols) ? kWideThreads : kThreads); }

// Most units (blocks, or clusters) of the backward pass: kShift's may be twice as many
// as run at once, so that their chunks have at most two gates.
int64_t bwd_units(int64_t rows, int64_t cols, int sms)
{
    const Plan p = bwd_plan(cols);
    const int64_t most = static_cast<int64_t>(sms) * p.per_sm / p.ranks * (cols % 8 != 0 ? 2 : 1);
    return std::max<int64_t>(8, std::min<int64_t>((rows + 7) / 8 * 8, most));
}

size_t round256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

// The backward pass's workspace: row constants (past kRegCols), partial rows of the
// parameters' gradients, and of the gates at the chunks' ends.
struct Workspace {
    size_t consts, parts, ends, bytes;
    int64_t room;  // units that have partial rows
};

Workspace workspace_of(int64_t rows, int64_t cols, int sms)
{
    const bool walk = !in_registers(cols);
    const size_t n = static_cast<size_t>(walk ? walk_chunks(rows, cols, sms) : bwd_units(rows, cols, sms));
    const size_t row = static_cast<size_t>(rows::sums_pitch(cols)) * sizeof(float);
    Workspace w;
    w.consts = 0;
    w.parts = walk ? round256(2 * static_cast<size_t>(rows) * sizeof(float)) : 0;
    w.ends = w.parts + round256(4 * n * row);
    w.bytes = w.ends + round256(2 * n * row);
    w.room = static_cast<int64_t>(n);
    return w;
}

Call call_of(const f8_residual_norm &n, float *stats)
{
    return Call{n.kind == F8_LAYER_NORM, n.w_type == F8_F32, n.gate_type == F8_F32, n.rows, n.cols,
                n.gate_rows, n.eps, n.scale, n.w_pre, n.b_pre, n.w_post, n.b_post, n.gate, stats};
}

constexpr std::true_type yes;
constexpr std::false_type no;

// f(mode) for the rows' width, ODD that of a width of no whole vectors.
template <int ODD, typename F>
cudaError_t by_mode(int64_t cols, const Plan &p, int e, F f)
{
    if (cols % 8 != 0)
        return f(std::integral_constant<int, ODD>());
    if (p.ranks == 1 && cols == static_cast<int64_t>(p.threads) * e)
        return f(std::integral_constant<int, rows::kFull>());
    return f(std::integral_constant<int, rows::kVec>());
}

bool params_bf16(const Call &c) { return !c.w_f32 && (c.gate == nullptr || !c.g_f32); }

// Units that run at once, and the slots of each: a launch of more would walk its
// last chunks alone.
struct Shape {
    int64_t most;
    int stages;
    size_t smem;
};

template <auto Kernel>
cudaError_t shape_of(const Plan &p, uint32_t slot_bytes, uint32_t more, const DeviceInfo &dev, Shape *out)
{
    static std::once_flag once[64];
    static cudaError_t err[64];
    const int d = dev.ordinal & 63;
    std::call_once(once[d], [&] {
        err[d] = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    });
    if (err[d] != cudaSuccess)
        return err[d];
    const int fit = (ring_bytes(p.per_sm) - static_cast<int>(more)) / static_cast<int>(slot_bytes);
    out->stages = std::max(2, std::min(fit, rows::kMaxStages));
    out->smem = static_cast<size_t>(out->stages) * slot_bytes + more;
    int64_t units = static_cast<int64_t>(dev.sm_count) * p.per_sm / p.ranks;
    if (p.ranks > 2) {
        // clusters of more than a pair may leave SMs of a group over
        static std::mutex mutex;
        static int known[64][rows::kMaxCluster + 1];
        std::lock_guard<std::mutex> lock(mutex);
        int &n = known[d][p.ranks];
        if (n == 0) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(static_cast<unsigned>(units * p.ranks));
            cfg.blockDim = dim3(static_cast<unsigned>(p.threads));
            cfg.dynamicSmemBytes = out->smem;
            cudaLaunchAttribute attr;
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = static_cast<unsigned>(p.ranks);
            attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, Kernel, &cfg);
            if (e != cudaSuccess)
                return e;
            n = std::max(n, 1);
        }
        units = std::min<int64_t>(units, n);
    }
    out->most = std::max<int64_t>(1, units);
    return cudaSuccess;
}

// Rows of a chunk and the units that walk them, for at most `most` units at once (but
// eight, kShift's for one chunk).
template <int MODE>
int64_t chunk_rows(int64_t rows, int64_t most, int64_t *chunk)
{
    if (MODE != rows::kShift) {
        *chunk = (rows + std::min(most, rows) - 1) / std::min(most, rows);
        return (rows + *chunk - 1) / *chunk;
    }
    const int64_t n = std::max<int64_t>(1, std::min(most / 8, (rows + 7) / 8));
    *chunk = (rows + 8 * n - 1) / (8 * n) * 8;
    return (rows + *chunk - 1) / *chunk * 8;
}

template <typename TA, typename TR, int MODE, bool BF, int THREADS>
cudaError_t fwd_rows(const Call &c, const void *a, const void *r, void *r_out, void *y, unsigned *amax,
                     const DeviceInfo &dev, cudaStream_t st)
{
    const Plan p = fwd_plan(c.cols);
    Shape s;
    const cudaError_t e = shape_of<fwd_kernel<TA, TR, MODE, BF, THREADS>>(
        p, rows::slice_pitch<TA>(p.slice) + rows::slice_pitch<TR>(p.slice), 0, dev, &s);
    if (e != cudaSuccess)
        return e;
    int64_t chunk;
    const int64_t units = chunk_rows<MODE>(c.rows, s.most, &chunk);
    return launch_pdl_cluster(fwd_kernel<TA, TR, MODE, BF, THREADS>, dim3(static_cast<unsigned>(units * p.ranks)),
                              dim3(static_cast<unsigned>(p.threads)), s.smem, st,
                              static_cast<unsigned>(p.ranks), c, static_cast<const TA *>(a),
                              static_cast<const TR *>(r), static_cast<TR *>(r_out), static_cast<TA *>(y),
                              amax, chunk, p.ranks, p.slice, s.stages, wait_limit_ns(), dev.status);
}

// Widths of no whole vectors go by the tensors' own vectors (kShift) where all parameters
// are bf16 and stay in registers over the rows, element by element (kRagged) where one is
// fp32: each row then reads them again, which kShift's lanes do in eight scattered pieces.
// RMS / layer norm, fp32 weights, element by element against vectors: 8192 x 4095 181 / 225
// us against 174 / 246, 1999 x 5003 53 / 64 against 55 / 76, 8192 x 1001 45 / 57 against 42 /
// 64, 1999 x 12001 150 / 189 against 153 / 243; bf16 weights in vectors 102 / 127, 33 / 40, 27
// / 33 and 92 / 132.
template <typename TA, typename TR>
cudaError_t fwd(const Call &c, const void *a, const void *r, void *r_out, void *y, unsigned *amax,
                const DeviceInfo &dev, cudaStream_t st)
{
    if (in_registers(c.cols)) {
        const Plan p = fwd_plan(c.cols);
        auto run = [&](auto bf, auto threads) {
            return by_mode<bf.value ? rows::kShift : rows::kRagged>(c.cols, p, kFwdE, [&](auto mode) {
                return fwd_rows<TA, TR, mode.value, bf.value, threads.value>(c, a, r, r_out, y, amax, dev, st);
            });
        };
        constexpr std::integral_constant<int, kThreads> usual;
        constexpr std::integral_constant<int, kPairThreads> pair;
        if (pair_blocks(c.cols))
            return params_bf16(c) ? run(yes, pair) : run(no, pair);
        return params_bf16(c) ? run(yes, usual) : run(no, usual);
    }
    const int64_t grid = std::min<int64_t>(c.rows, 4 * dev.sm_count);
    return launch_pdl(fwd_walk_kernel<TA, TR>, dim3(static_cast<unsigned>(grid)), dim3(kWalkThreads), 0,
                      st, c, static_cast<const TA *>(a), static_cast<const TR *>(r),
                      static_cast<TR *>(r_out), static_cast<TA *>(y), amax, dev.status);
}

template <typename TA, typename TR, int MODE, bool FULL, int THREADS>
cudaError_t bwd_rows(const Call &c, Chunks &ch, int *shared, const void *dy, const void *dr_out, const void *a,
                     const void *r_out, const f8_residual_norm_grads &g, float *parts, float *ends,
                     const DeviceInfo &dev, cudaStream_t st)
{
    const Plan p = bwd_plan(c.cols);
    // dw1's and db1's sums over a unit's gates
    const uint32_t acc = c.gate != nullptr && c.gate_rows < c.rows ? p.threads * kBwdE * (FULL ? 8u : 4u) : 0u;
    Shape s;
    const cudaError_t e = shape_of<bwd_kernel<TA, TR, MODE, FULL, THREADS>>(
        p, 2 * (rows::slice_pitch<TA>(p.slice) + rows::slice_pitch<TR>(p.slice)), acc, dev, &s);
    if (e != cudaSuccess)
        return e;
    int64_t units = chunk_rows<MODE>(c.rows, s.most, &ch.chunk);
    *shared = MODE == rows::kShift ? 8 : 1;
    // kShift's units have room for two gates of their chunk
    if constexpr (MODE == rows::kShift)
        if (c.gate != nullptr && c.gate_rows < ch.chunk)
            units = chunk_rows<MODE>(c.rows, 2 * s.most, &ch.chunk);
    if constexpr (MODE == rows::kShift)
        if (c.gate != nullptr && c.gate_rows < ch.chunk)
            return bwd_rows<TA, TR, rows::kRagged, FULL, THREADS>(c, ch, shared, dy, dr_out, a, r_out, g, parts,
                                                                  ends, dev, st);
    return launch_pdl_cluster(bwd_kernel<TA, TR, MODE, FULL, THREADS>, dim3(static_cast<unsigned>(units * p.ranks)),
                              dim3(static_cast<unsigned>(p.threads)), s.smem, st,
                              static_cast<unsigned>(p.ranks), c, ch, static_cast<const TA *>(dy),
                              static_cast<const TR *>(dr_out), static_cast<const TA *>(a),
                              static_cast<const TR *>(r_out), static_cast<TA *>(g.da),
                              static_cast<TR *>(g.dr), parts, ends, g.dgate, p.ranks, p.slice, s.stages,
                              wait_limit_ns(), dev.status);
}

template <typename TA, typename TR>
cudaError_t bwd(const Call &c, const void *dy, const void *dr_out, const void *a, const void *r_out,
                const f8_residual_norm_grads &g, uint8_t *ws, const DeviceInfo &dev, cudaStream_t st)
{
    const bool sums = g.dw_pre != nullptr || g.db_pre != nullptr || g.dw_post != nullptr ||
                      g.db_post != nullptr || g.dgate != nullptr;
    const Workspace w = workspace_of(c.rows, c.cols, dev.sm_count);
    float *parts = reinterpret_cast<float *>(ws + w.parts);
    float *ends = reinterpret_cast<float *>(ws + w.ends);
    const unsigned strips = static_cast<unsigned>((c.cols + 255) / 256);
    Chunks ch{c.rows, c.gate != nullptr ? c.gate_rows : c.rows, 0, w.room};
    int shared = 1;  // units that share a chunk
    cudaError_t e;
    if (in_registers(c.cols)) {
        const bool full = c.layer || c.b_post != nullptr || g.db_pre != nullptr || g.db_post != nullptr;
        const Plan p = bwd_plan(c.cols);
        auto run = [&](auto all, auto threads) {
            return by_mode<rows::kShift>(c.cols, p, kBwdE, [&](auto mode) {
                return bwd_rows<TA, TR, mode.value, all.value, threads.value>(c, ch, &shared, dy, dr_out, a, r_out,
                                                                              g, parts, ends, dev, st);
            });
        };
        constexpr std::integral_constant<int, kThreads> usual;
        constexpr std::integral_constant<int, kWideThreads> wide;
        if (wide_block(c.cols))
            e = full ? run(yes, wide) : run(no, wide);
        else
            e = full ? run(yes, usual) : run(no, usual);
    } else {
        float *consts = reinterpret_cast<float *>(ws + w.consts);
        const auto *dy_ = static_cast<const TA *>(dy), *a_ = static_cast<const TA *>(a);
        const auto *dr_ = static_cast<const TR *>(dr_out), *r_ = static_cast<const TR *>(r_out);
        const int64_t grid = std::min<int64_t>(c.rows, 4 * dev.sm_count);
        e = launch_pdl(bwd_walk_kernel<TA, TR>, dim3(static_cast<unsigned>(grid)), dim3(kWalkThreads), 0,
                       st, c, dy_, dr_, a_, r_, static_cast<TA *>(g.da), static_cast<TR *>(g.dr), consts,
                       dev.status);
        if (e != cudaSuccess || !sums)
            return e;
        const int64_t want = walk_chunks(c.rows, c.cols, dev.sm_count);
        ch.chunk = (c.rows + want - 1) / want;
        e = launch_pdl(cols_walk_kernel<TA, TR>,
                       dim3(strips, static_cast<unsigned>((c.rows + ch.chunk - 1) / ch.chunk)), dim3(256), 0,
                       st, c, ch, dy_, dr_, a_, r_, static_cast<const float *>(consts), parts, ends,
                       g.dgate, dev.status);
    }
    if (e != cudaSuccess || !sums)
        return e;
    const int64_t n = (c.rows + ch.chunk - 1) / ch.chunk;
    const int64_t gates = (c.rows - 1) / ch.gate_rows + 1;
    Sums out = {};
    out.out[0] = g.dw_pre;
    out.out[1] = g.db_pre;
    out.out[2] = g.dw_post;
    out.out[3] = g.db_post;
    out.dgate = g.dgate;
    out.parts = parts;
    out.ends = ends;
    out.nparts = static_cast<int>(n * shared);
    out.w_f32 = c.w_f32;
    out.g_f32 = c.g_f32;
    out.units = shared;
    out.shift = shared == 1 ? 0 : static_cast<int>(c.cols & 7);
    out.cols = c.cols;
    out.pitch = in_registers(c.cols) ? rows::sums_pitch(c.cols) : c.cols;
    out.gates = gates;
    const unsigned across = static_cast<unsigned>((c.cols + 31) / 32);
    const int W = across * 4 < 2u * dev.sm_count ? kReduceMost : kReduceWarps;
    const bool few = (ch.gate_rows / ch.chunk + 2) * shared <= 2 * W;  // partial rows of a gate
    out.by = shared == 1 && gates > n - 1 ? kBorder : few ? kMany : kEach;
    const int64_t down = g.dgate == nullptr ? 0 : out.by == kEach ? gates : ((out.by == kMany ? gates : n) + W - 1) / W;
    return launch_pdl(reduce_kernel, dim3(across, static_cast<unsigned>(4 + down)), dim3(32 * W), 0, st, out, ch,
                      dev.status);
}

bool type_ok(f8_dtype t) { return t == F8_BF16 || t == F8_F32; }

f8_status check_call(const f8_residual_norm *n)
{
    if (n == nullptr || (n->kind != F8_LAYER_NORM && n->kind != F8_RMS_NORM) || !type_ok(n->x_type) ||
        !type_ok(n->r_type) || !type_ok(n->w_type) || !type_ok(n->gate_type) || n->rows < 0 ||
        n->cols < 0 || !(n->eps >= 0.0f) || !std::isfinite(n->scale))
        return F8_ERR_INVALID;
    if (n->r_type != n->x_type && n->r_type != F8_F32)
        return F8_ERR_INVALID;
    if ((n->gate != nullptr && n->gate_rows < 1) || (n->b_post != nullptr && n->w_post == nullptr))
        return F8_ERR_INVALID;
    if (n->cols > INT32_MAX / 2 || (n->cols > 0 && n->rows > INT64_MAX / 8 / n->cols))
        return F8_ERR_SHAPE;
    if (n->rows > 0 && n->cols > 0 && n->w_pre == nullptr)
        return F8_ERR_INVALID;
    if (!aligned(n->w_pre, 16) || !aligned(n->b_pre, 16) || !aligned(n->w_post, 16) ||
        !aligned(n->b_post, 16) || !aligned(n->gate, 16))
        return F8_ERR_ALIGN;
    return F8_OK;
}

} // namespace
} // namespace f8

using namespace f8;

extern "C" {

f8_status f8_residual_norm_fwd(const f8_residual_norm *n, const void *a, const void *r, void *r_out,
                               void *y, float *stats, float *amax_out, void *stream)
{
    F8_TRY(check_call(n));
    const bool some = n->rows > 0 && n->cols > 0;
    if (amax_out != nullptr && n->x_type != F8_BF16)
        return F8_ERR_INVALID;
    if (some && (a == nullptr || r == nullptr || r_out == nullptr || y == nullptr || stats == nullptr ||
                 r_out == y || r_out == a || y == r))
        return F8_ERR_INVALID;
    if (!aligned(a, 16) || !aligned(r, 16) || !aligned(r_out, 16) || !aligned(y, 16) ||
        !aligned(stats, 4) || !aligned(amax_out, 4))
        return F8_ERR_ALIGN;
    const DeviceInfo *dev;
    F8_TRY(get_device(&dev));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (amax_out != nullptr)
        F8_TRY_CUDA(cudaMemsetAsync(amax_out, 0, sizeof(float), st));
    if (!some)
        return F8_OK;
    const Call c = call_of(*n, stats);
    unsigned *amax = reinterpret_cast<unsigned *>(amax_out);
    if (n->x_type == F8_F32)
        return from_cuda(fwd<float, float>(c, a, r, r_out, y, amax, *dev, st));
    if (n->r_type == F8_F32)
        return from_cuda(fwd<__nv_bfloat16, float>(c, a, r, r_out, y, amax, *dev, st));
    return from_cuda(fwd<__nv_bfloat16, __nv_bfloat16>(c, a, r, r_out, y, amax, *dev, st));
}

size_t f8_residual_norm_bwd_workspace_bytes(int64_t rows, int64_t cols)
{
    if (rows <= 0 || cols <= 0)
        return 0;
    const DeviceInfo *dev = device_info();
    return workspace_of(rows, cols, dev != nullptr ? dev->sm_count : 152).bytes;
}

f8_status f8_residual_norm_bwd(const f8_residual_norm *n, const void *dy, const void *dr_out,
                               const void *a, const void *r_out, const float *stats,
                               const f8_residual_norm_grads *grads, void *workspace,
                               size_t workspace_bytes, void *stream)
{
    F8_TRY(check_call(n));
    if (grads == nullptr)
        return F8_ERR_INVALID;
    const f8_residual_norm_grads &g = *grads;
    const bool some = n->rows > 0 && n->cols > 0;
    if (((g.dw_post != nullptr || g.db_post != nullptr) && n->w_post == nullptr) ||
        (g.dgate != nullptr && n->gate == nullptr))
        return F8_ERR_INVALID;
    if (some && (dy == nullptr || a == nullptr || r_out == nullptr || stats == nullptr ||
                 workspace == nullptr ||
                 workspace_bytes < f8_residual_norm_bwd_workspace_bytes(n->rows, n->cols)))
        return F8_ERR_INVALID;
    for (const void *in : {dy, dr_out, a, r_out})
        if (some && in != nullptr && (in == g.da || in == g.dr))
            return F8_ERR_INVALID;
    if (!aligned(dy, 16) || !aligned(dr_out, 16) || !aligned(a, 16) || !aligned(r_out, 16) ||
        !aligned(stats, 4) || !aligned(g.da, 16) || !aligned(g.dr, 16) || !aligned(g.dw_pre, 16) ||
        !aligned(g.db_pre, 16) || !aligned(g.dw_post, 16) || !aligned(g.db_post, 16) ||
        !aligned(g.dgate, 16) || !aligned(workspace, 16))
        return F8_ERR_ALIGN;
    // rows are read again for several sums, and partial sums are joined after the rows: an
    // output in the place of an input or of another output would be read or lost
    const void *const outs[] = {g.da, g.dr, g.dw_pre, g.db_pre, g.dw_post, g.db_post, g.dgate};
    const void *const ins[] = {dy, dr_out, a, r_out, stats, n->w_pre, n->b_pre, n->w_post, n->b_post, n->gate};
    for (const void *const *o = outs; some && o != std::end(outs); ++o)
        if (*o != nullptr && (std::find(ins, std::end(ins), *o) != std::end(ins) || std::find(outs, o, *o) != o))
            return F8_ERR_INVALID;
    const DeviceInfo *dev;
    F8_TRY(get_device(&dev));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!some) {  // sums over no rows
        const size_t bytes = static_cast<size_t>(n->cols) * (n->w_type == F8_BF16 ? 2 : 4);
        for (void *p : {g.dw_pre, g.db_pre, g.dw_post, g.db_post})
            if (p != nullptr && bytes > 0)
                F8_TRY_CUDA(cudaMemsetAsync(p, 0, bytes, st));
        return F8_OK;
    }
    const Call c = call_of(*n, const_cast<float *>(stats));
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    if (n->x_type == F8_F32)
        return from_cuda(bwd<float, float>(c, dy, dr_out, a, r_out, g, ws, *dev, st));
    if (n->r_type == F8_F32)
        return from_cuda(bwd<__nv_bfloat16, float>(c, dy, dr_out, a, r_out, g, ws, *dev, st));
    return from_cuda(bwd<__nv_bfloat16, __nv_bfloat16>(c, dy, dr_out, a, r_out, g, ws, *dev, st));
}

} // extern "C"
