// Backward of a linear's activation and bias: dz = dy act'(z) and the column sums
// dbias, in one pass over dy and z.
//
// Bound by HBM: 6 bytes an element (two bf16 read, one written) against some 20
// fp32 operations.  A warp takes rows of a strip of 32 16-byte vectors, one a lane, so
// that a lane's column sums stay in registers over all rows of its block; the block's
// eight warps are joined through shared memory and leave one partial row, and a
// second kernel adds the partial rows in order.  No atomics on the sums: equal
// inputs give equal bits.
//
// Vectors lie on 16-byte boundaries of the tensor, not of its rows: where the width is
// no multiple of eight, a row starts inside a vector, at an element that depends on the
// row's number modulo eight alone.  A warp's rows are eight apart, so its lanes keep
// their columns all the same; only a row's first and last vector go element by element.
//
// Measured, with the bias's gradient: tanh-GELU 8192 x 14336 112 us, 6.3 TB/s of the 6.8
// of a plain copy (at eight rows a warp in flight and two blocks an SM 126 us); GELU 1999
// x 5003 23 us of 8.8 for the bytes, in rows element by element 38.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "f8_act.cuh"
#include "f8_internal.h"
#include "f8_ptx.cuh"

namespace f8 {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kStrip = 256;   // columns of a block
constexpr int kUnroll = 2;    // rows of a warp whose loads are issued together
constexpr int kCarry = 8;     // columns before a strip that its vectors may reach into

__device__ __forceinline__ float2 bf_pair(uint32_t w)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

__device__ __forceinline__ uint32_t bf_pack2(float2 f)
{
    __nv_bfloat162 h = __float22bfloat162_rn(f);
    return *reinterpret_cast<uint32_t *>(&h);
}

// The vector of elements [at, at + 8), of which [at + lo, at + hi) are the row's; the
// others read as 0 and are not stored.
__device__ __forceinline__ uint4 load8(const __nv_bfloat16 *p, int64_t at, int lo, int hi, int64_t total,
                                       unsigned *status)
{
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (lo >= hi || !in_range(at + lo, hi - lo, total, status))
        return v;
    if (lo == 0 && hi == 8)
        return *reinterpret_cast<const uint4 *>(p + at);
    const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e >= lo && e < hi)
            w[e / 2] |= static_cast<uint32_t>(q[at + e]) << (16 * (e & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void store8(__nv_bfloat16 *p, int64_t at, int lo, int hi, const uint32_t (&w)[4],
                                       int64_t total, unsigned *status)
{
    if (lo >= hi || !in_range(at + lo, hi - lo, total, status))
        return;
    if (lo == 0 && hi == 8) {
        *reinterpret_cast<uint4 *>(p + at) = make_uint4(w[0], w[1], w[2], w[3]);
        return;
    }
    uint16_t *q = reinterpret_cast<uint16_t *>(p);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e >= lo && e < hi)
            q[at + e] = static_cast<uint16_t>(w[e / 2] >> (16 * (e & 1)));
}

// Block (x, y): the vectors [32 x, 32 x + 32) of the rows [y chunk, (y + 1) chunk).
// A row's vector q holds its columns 8 q - s .. 8 q - s + 7, s the row's start modulo 8
// (EVEN: the width is a multiple of 8 and s is 0).  parts: [gridDim.y][cols] fp32
// partial sums and carry: [gridDim.y][gridDim.x][kCarry] those of the columns before
// the strip; with out, the sums themselves (one chunk, EVEN).
template <int ACT, bool EVEN>
__global__ void __launch_bounds__(kThreads, 4)
act_bwd_kernel(const __nv_bfloat16 *dy, const __nv_bfloat16 *z, int64_t rows, int64_t cols,
               int64_t chunk, __nv_bfloat16 *dz, float *__restrict__ parts, float *__restrict__ carry,
               void *out, int out_bf16, unsigned *amax, unsigned *status)
{
    __shared__ __align__(16) float sums[kWarps][kStrip];
    __shared__ unsigned blk;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t first = static_cast<int64_t>(blockIdx.y) * chunk;
    const int64_t stop = min(first + chunk, rows);
    const int64_t total = rows * cols;
    const int s = EVEN ? 0 : static_cast<int>(((first + warp) * cols) & 7);
    const int64_t col = static_cast<int64_t>(blockIdx.x) * kStrip + 8 * lane - s;
    const int lo = EVEN ? 0 : (col < 0 ? static_cast<int>(min(-col, int64_t{8})) : 0);
    const int hi = static_cast<int>(max(min(cols - col, int64_t{8}), int64_t{0}));
    if (threadIdx.x == 0)
        blk = 0u;
    griddep_wait();
    griddep_launch_dependents();
    float2 sum[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        sum[i] = make_float2(0.0f, 0.0f);
    uint32_t m2 = 0u;
    const int64_t step = kWarps * cols;
    int64_t at = (first + warp) * cols + col;
    for (int64_t row = first + warp; row < stop; row += kWarps * kUnroll, at += kUnroll * step) {
        uint4 g[kUnroll], v[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int end = row + k * kWarps < stop ? hi : 0;
            g[k] = load8(dy, at + k * step, lo, end, total, status);
            v[k] = ACT != F8_ACT_NONE ? load8(z, at + k * step, lo, end, total, status) : g[k];
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const uint32_t gw[4] = {g[k].x, g[k].y, g[k].z, g[k].w}, vw[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float2 f = bf_pair(gw[i]);
                if (ACT != F8_ACT_NONE)
                    f = __fmul2_rn(f, act::slope<ACT>(bf_pair(vw[i])));
                sum[i] = __fadd2_rn(sum[i], f);
                o[i] = bf_pack2(f);
                m2 = __vmaxu2(m2, o[i] & 0x7FFF7FFFu);
            }
            if (dz != nullptr)
                store8(dz, at + k * step, lo, row + k * kWarps < stop ? hi : 0, o, total, status);
        }
    }
    // columns that are not the row's hold zeros: they add nothing
    if (parts != nullptr || out != nullptr) {
        float4 *to = reinterpret_cast<float4 *>(&sums[warp][8 * lane]);
        to[0] = make_float4(sum[0].x, sum[0].y, sum[1].x, sum[1].y);
        to[1] = make_float4(sum[2].x, sum[2].y, sum[3].x, sum[3].y);
        __syncthreads();
        const int j = threadIdx.x;
        const int64_t c = static_cast<int64_t>(blockIdx.x) * kStrip + j;
        float f = 0.0f, before = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const int sw = EVEN ? 0 : static_cast<int>(((first + w) * cols) & 7);
            if (j + sw < kStrip)
                f += sums[w][j + sw];
            if (!EVEN && j < kCarry && j - kCarry + sw >= 0)
                before += sums[w][j - kCarry + sw];  // column c - kCarry
        }
        if (c < cols) {
            const int64_t part = static_cast<int64_t>(blockIdx.y) * cols + c;
            if (out == nullptr) {
                if (in_range(part, 1, gridDim.y * cols, status))
                    parts[part] = f;
            } else if (out_bf16)
                static_cast<__nv_bfloat16 *>(out)[c] = __float2bfloat16_rn(f);
            else
                static_cast<float *>(out)[c] = f;
        }
        const int64_t unit = static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x;
        if (!EVEN && j < kCarry && in_range(unit, 1, static_cast<int64_t>(gridDim.y) * gridDim.x, status))
            carry[unit * kCarry + j] = before;
    }
    if (amax != nullptr) {
        __syncthreads();
        const unsigned m = __reduce_max_sync(0xFFFFFFFFu, max(m2 & 0xFFFFu, m2 >> 16));
        if (lane == 0)
            atomicMax(&blk, m);
        __syncthreads();
        if (threadIdx.x == 0) {
            if (blk >= 0x7F80u)
                atomicOr(status, kStatusNonfinite);
            atomicMax(amax, blk << 16);  // the maximum does not depend on the order
        }
    }
}

// out[c] = sum of the partial rows in a fixed order: 32 columns a block, 32 threads
// a column, each every 32nd row.  The last columns of a strip have a part in the next
// strip's blocks too (carry, or NULL).
__global__ void __launch_bounds__(1024)
act_reduce_kernel(const float *__restrict__ parts, const float *__restrict__ carry, int nparts, int strips,
                  int64_t cols, int bf16, void *out, unsigned *status)
{
    __shared__ float acc[32][33];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    float s = 0.0f;
    if (c < cols) {
#pragma unroll 4
        for (int i = k; i < nparts; i += 32)
            if (in_range(static_cast<int64_t>(i) * cols + c, 1, nparts * cols, status))
                s += parts[static_cast<int64_t>(i) * cols + c];
        const int64_t strip = c / kStrip + 1;
        const int j = static_cast<int>(c - strip * kStrip) + kCarry;
        if (carry != nullptr && j >= 0 && strip < strips)
            for (int i = k; i < nparts; i += 32)
                if (in_range(i * int64_t{strips} + strip, 1, nparts * int64_t{strips}, status) &&
                    in_range(j, 1, kCarry, status))
                    s += carry[(static_cast<int64_t>(i) * strips + strip) * kCarry + j];
    }
    acc[k][lane] = s;
    __syncthreads();
    s = acc[lane][k];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + k;
    if (lane == 0 && col < cols && in_range(col, 1, cols, status)) {
        if (bf16)
            static_cast<__nv_bfloat16 *>(out)[col] = __float2bfloat16_rn(s);
        else
            static_cast<float *>(out)[col] = s;
    }
}

// Strips of columns, and row chunks: whole rounds of the four blocks an SM runs at
// once, of at least 32 rows (four of each warp).  Even widths: one round for chunks of
// up to 64 rows and up to four for more; 1999 x 5000 in one round 12 us, in two 14.  Odd
// ones, whose rows' first and last vectors keep their warps longer, two: 1999 x 5003 in
// one round 23 us, in two 22, in four 24.
struct Plan {
    int64_t strips, chunks, chunk;
    bool even, direct;  // direct: the one chunk's sums are the result
    size_t parts, bytes;
};

Plan plan_of(int64_t rows, int64_t cols, int sms)
{
    Plan p;
    p.even = cols % 8 == 0;
    p.strips = (cols + (p.even ? 0 : 7) + kStrip - 1) / kStrip;
    const int64_t round = 4ll * sms, least = p.even ? 1 : 2;
    const int64_t rounds = std::max<int64_t>(least, std::min<int64_t>(4, rows * p.strips / (64 * round)));
    const int64_t want = std::max<int64_t>(1, round * rounds / p.strips);
    const int64_t n = std::max<int64_t>(1, std::min<int64_t>({want, (rows + 31) / 32, 65535}));
    p.chunk = (rows + n - 1) / n;
    p.chunks = (rows + p.chunk - 1) / p.chunk;
    p.direct = p.even && p.chunks == 1;
    p.parts = (static_cast<size_t>(p.chunks) * static_cast<size_t>(cols) * sizeof(float) + 255) & ~size_t{255};
    p.bytes = p.direct ? 0 : p.parts + (p.even ? 0 : static_cast<size_t>(p.chunks * p.strips) * kCarry * sizeof(float));
    return p;
}

struct Call {
    const void *dy, *z;
    int64_t rows, cols;
    void *dz, *dbias;
    int bias_bf16;
    unsigned *amax;
    uint8_t *ws;
};

template <int ACT>
cudaError_t launch(const Call &c, const Plan &p, const DeviceInfo &dev, cudaStream_t st)
{
    const dim3 grid(static_cast<unsigned>(p.strips), static_cast<unsigned>(p.chunks));
    const auto *g = static_cast<const __nv_bfloat16 *>(c.dy);
    const auto *v = static_cast<const __nv_bfloat16 *>(c.z);
    auto *o = static_cast<__nv_bfloat16 *>(c.dz);
    const bool sums = c.dbias != nullptr;
    float *parts = sums && !p.direct ? reinterpret_cast<float *>(c.ws) : nullptr;
    float *carry = parts != nullptr && !p.even ? reinterpret_cast<float *>(c.ws + p.parts) : nullptr;
    void *out = sums && p.direct ? c.dbias : nullptr;
    const cudaError_t e =
        p.even ? launch_pdl(act_bwd_kernel<ACT, true>, grid, dim3(kThreads), 0, st, g, v, c.rows, c.cols,
                            p.chunk, o, parts, carry, out, c.bias_bf16, c.amax, dev.status)
               : launch_pdl(act_bwd_kernel<ACT, false>, grid, dim3(kThreads), 0, st, g, v, c.rows, c.cols,
                            p.chunk, o, parts, carry, out, c.bias_bf16, c.amax, dev.status);
    if (e != cudaSuccess || parts == nullptr)
        return e;
    return launch_pdl(act_reduce_kernel, dim3(static_cast<unsigned>((c.cols + 31) / 32)), dim3(1024), 0, st,
                      static_cast<const float *>(parts), static_cast<const float *>(carry),
                      static_cast<int>(p.chunks), static_cast<int>(p.strips), c.cols, c.bias_bf16, c.dbias,
                      dev.status);
}

} // namespace
} // namespace f8

using namespace f8;

extern "C" {

size_t f8_act_bwd_workspace_bytes(int64_t rows, int64_t cols)
{
    if (rows <= 0 || cols <= 0)
        return 0;
    const DeviceInfo *dev = device_info();
    return plan_of(rows, cols, dev != nullptr ? dev->sm_count : 152).bytes;
}

f8_status f8_act_bwd(const void *dy, const void *z, f8_act act, int64_t rows, int64_t cols, void *dz,
                     void *dbias, f8_dtype bias_type, float *amax_out, void *workspace,
                     size_t workspace_bytes, void *stream)
{
    if (act < F8_ACT_NONE || act > F8_ACT_GELU_TANH || (bias_type != F8_BF16 && bias_type != F8_F32) ||
        rows < 0 || cols < 0 || (amax_out != nullptr && dz == nullptr))
        return F8_ERR_INVALID;
    if (cols > INT32_MAX / 2 || (cols > 0 && rows > INT64_MAX / 8 / cols))
        return F8_ERR_SHAPE;
    const bool some = rows > 0 && cols > 0;
    if (some && (dy == nullptr || (act != F8_ACT_NONE && z == nullptr)))
        return F8_ERR_INVALID;
    const size_t need = some && dbias != nullptr ? f8_act_bwd_workspace_bytes(rows, cols) : 0;
    if (need > 0 && (workspace == nullptr || workspace_bytes < need))
        return F8_ERR_INVALID;
    if (!aligned(dy, 16) || !aligned(z, 16) || !aligned(dz, 16) || !aligned(dbias, 16) ||
        !aligned(workspace, 16) || !aligned(amax_out, 4))
        return F8_ERR_ALIGN;
    const DeviceInfo *dev;
    F8_TRY(get_device(&dev));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (amax_out != nullptr)
        F8_TRY_CUDA(cudaMemsetAsync(amax_out, 0, sizeof(float), st));
    if (!some) {  // a sum over no rows
        const size_t bytes = static_cast<size_t>(cols) * (bias_type == F8_BF16 ? 2 : 4);
        if (dbias != nullptr && bytes > 0)
            F8_TRY_CUDA(cudaMemsetAsync(dbias, 0, bytes, st));
        return F8_OK;
    }
    if (dz == nullptr && dbias == nullptr)
        return F8_OK;
    const Plan p = plan_of(rows, cols, dev->sm_count);
    const Call c{dy, z, rows, cols, dz, dbias, bias_type == F8_BF16, reinterpret_cast<unsigned *>(amax_out),
                 static_cast<uint8_t *>(workspace)};
    switch (act) {
    case F8_ACT_RELU: return from_cuda(launch<F8_ACT_RELU>(c, p, *dev, st));
    case F8_ACT_RELU2: return from_cuda(launch<F8_ACT_RELU2>(c, p, *dev, st));
    case F8_ACT_SILU: return from_cuda(launch<F8_ACT_SILU>(c, p, *dev, st));
    case F8_ACT_GELU: return from_cuda(launch<F8_ACT_GELU>(c, p, *dev, st));
    case F8_ACT_GELU_TANH: return from_cuda(launch<F8_ACT_GELU_TANH>(c, p, *dev, st));
    default: return from_cuda(launch<F8_ACT_NONE>(c, p, *dev, st));
    }
}

} // extern "C"
