// Backward of a linear's activation and bias: dz = dy act'(z) and the column sums
// dbias, in one pass over dy and z.
//
// Bound by HBM: 6 bytes an element (two bf16 read, one written) against some 20
// fp32 operations.  A warp takes rows of a strip of 256 columns, 8 a lane, so that
// a lane's column sums stay in registers over all rows of its block; the block's
// eight warps are joined through shared memory and leave one partial row, and a
// second kernel adds the partial rows in order.  No atomics on the sums: equal
// inputs give equal bits.
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
constexpr int kUnroll = 4;    // rows of a warp whose loads are issued together

__device__ __forceinline__ float2 bf_pair(uint32_t w)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

__device__ __forceinline__ uint32_t bf_pack2(float2 f)
{
    __nv_bfloat162 h = __float22bfloat162_rn(f);
    return *reinterpret_cast<uint32_t *>(&h);
}

// Eight columns of one row as four packed pairs.  VEC: columns 8 lane .. 8 lane + 7,
// one 16-byte access; else columns lane + 32 j, element by element.
template <bool VEC>
struct Piece {
    uint32_t w[4];

    __device__ __forceinline__ void load(const __nv_bfloat16 *p, int64_t row, int64_t cols, int64_t col,
                                         int64_t total, unsigned *status)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = 0u;
        const int64_t at = row * cols + col;
        if (VEC) {
            if (col < cols && in_range(at, 8, total, status)) {
                const uint4 v = *reinterpret_cast<const uint4 *>(p + at);
                w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
            }
            return;
        }
        const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (col + 32 * j < cols && in_range(at + 32 * j, 1, total, status))
                w[j / 2] |= static_cast<uint32_t>(q[at + 32 * j]) << (16 * (j & 1));
    }

    __device__ __forceinline__ void store(__nv_bfloat16 *p, int64_t row, int64_t cols, int64_t col,
                                          int64_t total, unsigned *status) const
    {
        const int64_t at = row * cols + col;
        if (VEC) {
            if (col < cols && in_range(at, 8, total, status))
                *reinterpret_cast<uint4 *>(p + at) = make_uint4(w[0], w[1], w[2], w[3]);
            return;
        }
        uint16_t *q = reinterpret_cast<uint16_t *>(p);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (col + 32 * j < cols && in_range(at + 32 * j, 1, total, status))
                q[at + 32 * j] = static_cast<uint16_t>(w[j / 2] >> (16 * (j & 1)));
    }
};

// Block (x, y): columns [256 x, 256 x + 256), rows [y chunk, (y + 1) chunk).
// parts: [gridDim.y][cols] fp32 partial sums, or NULL.
template <int ACT, bool VEC>
__global__ void __launch_bounds__(kThreads)
act_bwd_kernel(const __nv_bfloat16 *dy, const __nv_bfloat16 *z, int64_t rows, int64_t cols,
               int64_t chunk, __nv_bfloat16 *dz, float *__restrict__ parts, unsigned *amax,
               unsigned *status)
{
    __shared__ float4 sums[kWarps - 1][2][32];
    __shared__ unsigned blk;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * kStrip + (VEC ? 8 * lane : lane);
    const int64_t first = static_cast<int64_t>(blockIdx.y) * chunk;
    const int64_t stop = min(first + chunk, rows);
    const int64_t total = rows * cols;
    if (threadIdx.x == 0)
        blk = 0u;
    griddep_wait();
    griddep_launch_dependents();
    float2 s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        s[i] = make_float2(0.0f, 0.0f);
    uint32_t m2 = 0u;
    for (int64_t row = first + warp; row < stop; row += kWarps * kUnroll) {
        Piece<VEC> g[kUnroll], v[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            if (row + k * kWarps < stop) {
                g[k].load(dy, row + k * kWarps, cols, col, total, status);
                if (ACT != F8_ACT_NONE)
                    v[k].load(z, row + k * kWarps, cols, col, total, status);
            }
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            if (row + k * kWarps >= stop)
                break;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float2 f = bf_pair(g[k].w[i]);
                if (ACT != F8_ACT_NONE)
                    f = __fmul2_rn(f, act::slope<ACT>(bf_pair(v[k].w[i])));
                s[i] = __fadd2_rn(s[i], f);
                g[k].w[i] = bf_pack2(f);
                m2 = __vmaxu2(m2, g[k].w[i] & 0x7FFF7FFFu);
            }
            if (dz != nullptr)
                g[k].store(dz, row + k * kWarps, cols, col, total, status);
        }
    }
    // columns past the last hold zeros: they add nothing and are not stored
    if (parts != nullptr) {
        if (warp > 0) {
            sums[warp - 1][0][lane] = make_float4(s[0].x, s[0].y, s[1].x, s[1].y);
            sums[warp - 1][1][lane] = make_float4(s[2].x, s[2].y, s[3].x, s[3].y);
        }
        __syncthreads();
        if (warp == 0) {
            float f[8] = {s[0].x, s[0].y, s[1].x, s[1].y, s[2].x, s[2].y, s[3].x, s[3].y};
            for (int w = 0; w < kWarps - 1; ++w) {
                const float4 a = sums[w][0][lane], b = sums[w][1][lane];
                f[0] += a.x, f[1] += a.y, f[2] += a.z, f[3] += a.w;
                f[4] += b.x, f[5] += b.y, f[6] += b.z, f[7] += b.w;
            }
            float *p = parts + static_cast<int64_t>(blockIdx.y) * cols;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int64_t c = VEC ? col + j : col + 32 * j;
                if (c < cols)
                    p[c] = f[j];
            }
        }
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
// a column, each every 32nd row.
__global__ void __launch_bounds__(1024)
act_reduce_kernel(const float *__restrict__ parts, int nparts, int64_t cols, int bf16, void *out,
                  unsigned *status)
{
    __shared__ float acc[32][33];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    float s = 0.0f;
    if (c < cols)
        for (int i = k; i < nparts; i += 32)
            s += parts[static_cast<int64_t>(i) * cols + c];
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

// Row chunks: about 16 blocks an SM in all, of at least 32 rows (four of each warp).
int64_t chunks(int64_t rows, int64_t cols, int sms)
{
    const int64_t strips = (cols + kStrip - 1) / kStrip;
    const int64_t want = std::max<int64_t>(1, 16ll * sms / strips);
    return std::max<int64_t>(1, std::min<int64_t>({want, (rows + 31) / 32, 65535}));
}

template <int ACT>
cudaError_t launch(const void *dy, const void *z, int64_t rows, int64_t cols, void *dz, float *parts,
                   unsigned *amax, const DeviceInfo &dev, cudaStream_t st, int *nparts)
{
    const int64_t want = chunks(rows, cols, dev.sm_count);
    const int64_t chunk = (rows + want - 1) / want;
    *nparts = static_cast<int>((rows + chunk - 1) / chunk);
    const dim3 grid(static_cast<unsigned>((cols + kStrip - 1) / kStrip), static_cast<unsigned>(*nparts));
    const auto *g = static_cast<const __nv_bfloat16 *>(dy);
    const auto *v = static_cast<const __nv_bfloat16 *>(z);
    auto *o = static_cast<__nv_bfloat16 *>(dz);
    return cols % 8 == 0 ? launch_pdl(act_bwd_kernel<ACT, true>, grid, dim3(kThreads), 0, st, g, v, rows,
                                      cols, chunk, o, parts, amax, dev.status)
                         : launch_pdl(act_bwd_kernel<ACT, false>, grid, dim3(kThreads), 0, st, g, v, rows,
                                      cols, chunk, o, parts, amax, dev.status);
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
    return static_cast<size_t>(chunks(rows, cols, dev != nullptr ? dev->sm_count : 152)) *
           static_cast<size_t>(cols) * sizeof(float);
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
    if (some && dbias != nullptr &&
        (workspace == nullptr || workspace_bytes < f8_act_bwd_workspace_bytes(rows, cols)))
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
    float *parts = dbias != nullptr ? static_cast<float *>(workspace) : nullptr;
    unsigned *amax = reinterpret_cast<unsigned *>(amax_out);
    int n = 0;
    cudaError_t e = cudaErrorInvalidValue;
    switch (act) {
    case F8_ACT_NONE: e = launch<F8_ACT_NONE>(dy, z, rows, cols, dz, parts, amax, *dev, st, &n); break;
    case F8_ACT_RELU: e = launch<F8_ACT_RELU>(dy, z, rows, cols, dz, parts, amax, *dev, st, &n); break;
    case F8_ACT_RELU2: e = launch<F8_ACT_RELU2>(dy, z, rows, cols, dz, parts, amax, *dev, st, &n); break;
    case F8_ACT_SILU: e = launch<F8_ACT_SILU>(dy, z, rows, cols, dz, parts, amax, *dev, st, &n); break;
    case F8_ACT_GELU: e = launch<F8_ACT_GELU>(dy, z, rows, cols, dz, parts, amax, *dev, st, &n); break;
    case F8_ACT_GELU_TANH:
        e = launch<F8_ACT_GELU_TANH>(dy, z, rows, cols, dz, parts, amax, *dev, st, &n);
        break;
    }
    F8_TRY_CUDA(e);
    if (dbias == nullptr)
        return F8_OK;
    return from_cuda(launch_pdl(act_reduce_kernel, dim3(static_cast<unsigned>((cols + 31) / 32)),
                                dim3(1024), 0, st, static_cast<const float *>(parts), n, cols,
                                bias_type == F8_BF16 ? 1 : 0, dbias, dev->status));
}

} // extern "C"
