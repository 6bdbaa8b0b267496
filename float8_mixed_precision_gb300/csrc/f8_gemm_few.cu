// f8_gemm_act for few rows of A (decoding steps, small batches):
//   z = A B^T / (sa sb) + bias,  y = act(z) + residual,  E4M3 / E5M2 operands.
//
// Bound by reading B's codes once, and by latency: with a handful of rows the
// products are nothing.  So B's rows take the tensor core's 128 lanes and A's rows
// its columns (D^T = B A^T; 16 to 256 columns, as many as there are rows), and where
// that leaves SMs over, the CTAs of a cluster share a tile's K blocks: each reads its
// part of B, leaves its fp32 partial sums in its own shared memory, and finishes the
// rows r, r + splits, .. of the tile from all of them, in rank order.  No workspace
// and no atomics on the sums: equal inputs give equal bits.
//
// Measured, B [14336, 4096] and 8 rows: 15.4 us, 3.8 TB/s, of which some 6 are the
// launch, the first loads' and the epilogue's latencies.  A CTA takes 0.26 us a stage
// whatever the other SMs do (128 + 16 rows of 128 bytes by TMA), so its 32 stages take
// 8.3: 112 tiles do not fill 152 SMs, and splits of two, four and eight put three CTAs on
// some SMs and two on others (14.5, 20 and 31 us).  The kernel for many rows took 29.
//
// The tensor core cuts its running sum off rather than round it.  Of the outputs' rms the
// sums are off by 2^-22 at K = 4096 without a split (bit for bit as the kernel for many
// rows), by 2^-23.7 with four, and at 14336 with four by 2^-22.2 against that one's 2^-19.7;
// fp32 sums of the same products by 2^-24 and 2^-23.4.
//
//   warp 0      TMA producer, 128 bytes of K a stage into a ring
//   warp 1      TMEM allocation, tcgen05.mma kind::f8f6f4 (128 x NT x 32)
//   warps 2..5  the accumulators into shared memory, a lane one column of the output;
//               then all warps finish rows from there, eight columns a thread
//
// Every wait is bounded as in f8_gemm.cu; a CTA whose wait gave up still meets its
// cluster's barriers.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>

#include "f8_act.cuh"
#include "f8_internal.h"
#include "f8_ptx.cuh"

namespace f8 {
namespace {

constexpr int kLanes = 128;   // columns of the output a CTA forms
constexpr int kBK = 128;      // bytes of K a stage
constexpr int kThreads = 192;
constexpr int kMaxStages = 8;
constexpr int kBBytes = kLanes * kBK;
constexpr int kRingBytes = 200 * 1024;
constexpr uint64_t kDrainLimitNs = 1000000000ull;

struct Args {
    int M, N, num_kb, per_split;
    int nt;       // rows of a tile (TMEM columns), a multiple of 16
    int tiles_n, splits, stages, tmem_cols;
    uint32_t idesc;
    const float *sa, *sb;
    const void *bias;
    int bias_f32, act;
    const __nv_bfloat16 *residual;
    __nv_bfloat16 *y, *z;
    unsigned *amax;
    unsigned *status;
    uint64_t limit_ns;
};

__device__ __forceinline__ void note_timeout(volatile int *abort_flag, unsigned *status)
{
    *abort_flag = 1;
    atomicOr(status, kStatusTimeout);
}

// 32 lanes x 16 consecutive 32-bit columns: thread i gets lane (base + i).
__device__ __forceinline__ void tc_ld_x16(uint32_t taddr, float (&v)[16])
{
    uint32_t r[16];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                   "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
                   "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr));
    tc_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i)
        v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ float4 ld_cluster4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ uint32_t pack2(float2 f)
{
    __nv_bfloat162 h = __float22bfloat162_rn(f);
    return *reinterpret_cast<uint32_t *>(&h);
}
__device__ __forceinline__ float2 bf2(uint32_t w)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// Eight biases from column n; 0 past the last one.
__device__ __forceinline__ void bias8(const Args &p, int n, float2 (&f)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f[i] = make_float2(0.0f, 0.0f);
    if (p.bias == nullptr || n >= p.N || !in_range(n, min(8, p.N - n), p.N, p.status))
        return;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int c = min(n + e, p.N - 1);
        v[e] = p.bias_f32 ? __ldg(static_cast<const float *>(p.bias) + c)
                          : __bfloat162float(static_cast<const __nv_bfloat16 *>(p.bias)[c]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f[i] = make_float2(v[2 * i], v[2 * i + 1]);
}

// The residual of eight columns from o, one row's; VEC: the rows start on 16-byte
// boundaries.  `some` columns of the eight are the tensor's.
template <bool VEC>
__device__ __forceinline__ uint4 residual8(const Args &p, int64_t o, int some)
{
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    const int64_t total = static_cast<int64_t>(p.M) * p.N;
    if (p.residual != nullptr && some > 0 && in_range(o, some, total, p.status)) {
        if constexpr (VEC) {
            return *reinterpret_cast<const uint4 *>(p.residual + o);
        } else {
            const uint16_t *r = reinterpret_cast<const uint16_t *>(p.residual) + o;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                w[e / 2] |= static_cast<uint32_t>(r[min(e, some - 1)]) << (16 * (e & 1));
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool VEC>
__device__ __forceinline__ void store8(__nv_bfloat16 *to, const uint32_t (&w)[4], int some)
{
    if constexpr (VEC) {
        *reinterpret_cast<uint4 *>(to) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        uint16_t *q = reinterpret_cast<uint16_t *>(to);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < some)
                q[e] = static_cast<uint16_t>(w[e / 2] >> (16 * (e & 1)));
    }
}

// Rows rank, rank + splits, .. of the tile from the partial sums that every CTA of the
// cluster has left at `part` [nt][128]: 16 threads a row, eight columns each, so a
// thread's columns and biases stay the same.  `first` is the residual of its first row.
template <int ACT, bool VEC>
__device__ __forceinline__ void finish(const Args &p, uint32_t part, int rank, int m0, int rows, int n,
                                       float inv, const float2 (&bias)[4], uint4 first, unsigned &top)
{
    constexpr int kStep = kThreads / 16;
    const int some = min(8, p.N - n), col = (threadIdx.x & 15) * 8;
    const int64_t total = static_cast<int64_t>(p.M) * p.N;
    uint4 res = first;
    for (int t = rank + p.splits * (static_cast<int>(threadIdx.x) >> 4); t < rows; t += p.splits * kStep) {
        const int64_t o = static_cast<int64_t>(m0 + t) * p.N + n;
        const uint32_t old[4] = {res.x, res.y, res.z, res.w};
        // the next row's residual is on its way while this one is worked on
        if (t + p.splits * kStep < rows)
            res = residual8<VEC>(p, o + static_cast<int64_t>(p.splits) * kStep * p.N, some);
        float2 a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            a[i] = make_float2(0.0f, 0.0f);
        for (int r = 0; r < p.splits; ++r) {
            const uint32_t from = (p.splits > 1 ? cluster_map(part, r) : part) + (t * kLanes + col) * 4;
            const float4 u = ld_cluster4(from), v = ld_cluster4(from + 16);
            a[0] = __fadd2_rn(a[0], make_float2(u.x, u.y));
            a[1] = __fadd2_rn(a[1], make_float2(u.z, u.w));
            a[2] = __fadd2_rn(a[2], make_float2(v.x, v.y));
            a[3] = __fadd2_rn(a[3], make_float2(v.z, v.w));
        }
        uint32_t yw[4], zw[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 z = __ffma2_rn(a[i], make_float2(inv, inv), bias[i]);
            zw[i] = pack2(z);
            yw[i] = pack2(__fadd2_rn(act::value<ACT>(z), bf2(old[i])));
        }
        if (!in_range(o, some, total, p.status))
            continue;
        store8<VEC>(p.y + o, yw, some);
        if (p.z != nullptr)
            store8<VEC>(p.z + o, zw, some);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (VEC || e < some)
                top = max(top, (yw[e / 2] >> (16 * (e & 1))) & 0x7FFFu);
    }
}

template <bool VEC>
__device__ __forceinline__ void finish_any(const Args &p, uint32_t part, int rank, int m0, int rows, int n,
                                           float inv, const float2 (&bias)[4], uint4 first, unsigned &top)
{
    switch (p.act) {
    case F8_ACT_RELU: finish<F8_ACT_RELU, VEC>(p, part, rank, m0, rows, n, inv, bias, first, top); break;
    case F8_ACT_RELU2: finish<F8_ACT_RELU2, VEC>(p, part, rank, m0, rows, n, inv, bias, first, top); break;
    case F8_ACT_SILU: finish<F8_ACT_SILU, VEC>(p, part, rank, m0, rows, n, inv, bias, first, top); break;
    case F8_ACT_GELU: finish<F8_ACT_GELU, VEC>(p, part, rank, m0, rows, n, inv, bias, first, top); break;
    case F8_ACT_GELU_TANH: finish<F8_ACT_GELU_TANH, VEC>(p, part, rank, m0, rows, n, inv, bias, first, top); break;
    default: finish<F8_ACT_NONE, VEC>(p, part, rank, m0, rows, n, inv, bias, first, top); break;
    }
}

// A thread's scale, biases and first residual of the epilogue.
template <bool VEC>
__device__ __forceinline__ void load_epilogue(const Args &p, int rank, int m0, int n0, float &inv,
                                              float2 (&bias)[4], uint4 &res)
{
    const int n = n0 + (threadIdx.x & 15) * 8, t = rank + p.splits * (static_cast<int>(threadIdx.x) >> 4);
    inv = static_cast<float>(1.0 / (static_cast<double>(*p.sa) * static_cast<double>(*p.sb)));
    bias8(p, n, bias);
    if (t < min(p.nt, p.M - m0))
        res = residual8<VEC>(p, static_cast<int64_t>(m0 + t) * p.N + n, min(8, p.N - n));
}

template <bool VEC>
__global__ void __launch_bounds__(kThreads, 1)
gemm_few_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
                const __grid_constant__ Args p)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], tfull, drain;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_word;
    __shared__ unsigned top_cta;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    volatile int *abort_flag = &abort_word;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = p.splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int tile = static_cast<int>(blockIdx.x) / p.splits;
    const int n0 = tile % p.tiles_n * kLanes, m0 = tile / p.tiles_n * p.nt;
    const int kb0 = rank * p.per_split, kbs = max(0, min(p.per_split, p.num_kb - kb0));
    const int stage_bytes = kBBytes + p.nt * kBK;

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(&tfull, 1);
        mbar_init(&drain, 1);
        abort_word = 0;
        top_cta = 0u;
        fence_mbar_init();
        tma_prefetch_desc(&ma);
        tma_prefetch_desc(&mb);
    }
    if (warp == 1) {
        tmem_alloc(&tmem_slot, p.tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = tmem_slot;
    griddep_wait();
    griddep_launch_dependents();
    // what the epilogue reads besides the sums, while they are formed
    float2 bias[4];
    uint4 res = make_uint4(0u, 0u, 0u, 0u);
    float inv = 0.0f;
    if (warp >= 2 || lane > 0)  // not the two threads that feed the tensor core
        load_epilogue<VEC>(p, rank, m0, n0, inv, bias, res);

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0, issued = 0;
            uint32_t phase = 0;
            for (int kb = 0; kb < kbs; ++kb) {
                if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.limit_ns)) {
                    note_timeout(abort_flag, p.status);
                    break;
                }
                uint8_t *to = smem + stage * stage_bytes;
                mbar_arrive_expect_tx(&full[stage], stage_bytes);
                tma_load_2d(to, &mb, &full[stage], (kb0 + kb) * kBK, n0);
                tma_load_2d(to + kBBytes, &ma, &full[stage], (kb0 + kb) * kBK, m0);
                ++issued;
                if (++stage == p.stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!*abort_flag) {
                // the stages' releases have landed before their barriers go away
                for (int i = 0; i < p.stages; ++i) {
                    if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.limit_ns)) {
                        note_timeout(abort_flag, p.status);
                        break;
                    }
                    if (++stage == p.stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            } else {
                for (int i = 0; i < min(issued, p.stages); ++i) {
                    if (stage == 0) {
                        stage = p.stages - 1;
                        phase ^= 1u;
                    } else {
                        --stage;
                    }
                    mbar_wait(&full[stage], phase, nullptr, kDrainLimitNs);
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            for (int kb = 0; kb < kbs; ++kb) {
                if (!mbar_wait(&full[stage], phase, abort_flag, p.limit_ns)) {
                    note_timeout(abort_flag, p.status);
                    break;
                }
                tc_fence_after_sync();
                const uint32_t at = smem_addr(smem + stage * stage_bytes);
                const uint64_t bd = sdesc_kmajor_sw128(at), ad = sdesc_kmajor_sw128(at + kBBytes);
#pragma unroll
                for (int k = 0; k < kBK / 32; ++k)
                    tc_mma_f8(tmem, bd + 2 * k, ad + 2 * k, p.idesc, (kb | k) != 0);
                tc_commit(&empty[stage]);
                if (++stage == p.stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!*abort_flag) {
                tc_commit(&tfull);
            } else {
                tc_commit(&drain);
                mbar_wait(&drain, 0, nullptr, kDrainLimitNs);
            }
        }
        __syncwarp();
    }

    // ------------------------------------------------------------ epilogue
    if (warp < 2 && lane == 0)
        load_epilogue<VEC>(p, rank, m0, n0, inv, bias, res);
    const int rows = min(p.nt, p.M - m0), n = n0 + (threadIdx.x & 15) * 8;
    if (warp >= 2) {
        const int quad = warp & 3;  // the TMEM lane quarter this warp may read
        const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(&tfull, 0, abort_flag, p.limit_ns));
        if (!ok && lane == 0)
            note_timeout(abort_flag, p.status);
        tc_fence_after_sync();
        const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        float *to = reinterpret_cast<float *>(smem) + quad * 32 + lane;  // [nt][128]
        for (int t = 0; t < rows; t += 16) {
            float v[16];
            if (ok && kbs > 0) {
                tc_ld_x16(taddr + t, v);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    v[i] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i)
                to[(t + i) * kLanes] = v[i];
        }
    }
    __syncwarp();
    if (p.splits > 1)
        cluster_sync();
    else
        __syncthreads();
    unsigned top = 0u;
    if (n < p.N)
        finish_any<VEC>(p, smem_addr(smem), rank, m0, rows, n, inv, bias, res, top);
    __syncwarp();
    if (p.amax != nullptr) {
        top = __reduce_max_sync(0xFFFFFFFFu, top);
        if (lane == 0)
            atomicMax(&top_cta, top);
    }
    tc_fence_before_sync();
    if (p.splits > 1)
        cluster_sync();  // the peers have read this CTA's sums
    else
        __syncthreads();
    if (threadIdx.x == 0 && p.amax != nullptr) {
        if (top_cta >= 0x7F80u)
            atomicOr(p.status, kStatusNonfinite);
        atomicMax(p.amax, top_cta << 16);  // the maximum does not depend on the order
    }
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, p.tmem_cols);
    }
}

} // namespace

FewPlan gemm_few_plan(int64_t M, int64_t N, int64_t K, int sms)
{
    FewPlan p;
    const int64_t tiles_m = (M + 255) / 256;
    p.nt = static_cast<int>(((M + tiles_m - 1) / tiles_m + 15) / 16 * 16);
    p.tiles = tiles_m * ((N + kLanes - 1) / kLanes);
    const int64_t kb = (K + kBK - 1) / kBK;
    p.splits = 1;
    while (p.splits < 8 && p.tiles * p.splits * 2 <= sms && kb >= 4 * p.splits)
        p.splits *= 2;
    return p;
}

cudaError_t launch_gemm_few(const GemmDesc &g, const ActEpilogue &e, const DeviceInfo &dev,
                            cudaStream_t stream)
{
    const FewPlan plan = gemm_few_plan(g.M, g.N, g.K, dev.sm_count);
    if (plan.tiles * plan.splits > INT32_MAX / 2)
        return cudaErrorInvalidValue;
    CUtensorMap ma, mb;
    const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    if (!make_tensor_map_2d(&ma, u8, 1, g.a, g.M, g.K, kBK, plan.nt, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_tensor_map_2d(&mb, u8, 1, g.b, g.N, g.K, kBK, kLanes, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorNotSupported;
    Args p = {};
    p.M = static_cast<int>(g.M);
    p.N = static_cast<int>(g.N);
    p.num_kb = static_cast<int>((g.K + kBK - 1) / kBK);
    p.splits = plan.splits;
    p.per_split = (p.num_kb + p.splits - 1) / p.splits;
    p.nt = plan.nt;
    p.tiles_n = static_cast<int>((g.N + kLanes - 1) / kLanes);
    const int stage = kBBytes + p.nt * kBK;
    p.stages = std::min(kMaxStages, kRingBytes / stage);
    p.tmem_cols = 32;
    while (p.tmem_cols < p.nt)
        p.tmem_cols *= 2;
    p.idesc = idesc_f8_f32(kLanes, static_cast<uint32_t>(p.nt), static_cast<uint32_t>(g.fb),
                           static_cast<uint32_t>(g.fa));
    p.sa = g.sa;
    p.sb = g.sb;
    p.bias = e.bias;
    p.bias_f32 = e.bias_f32;
    p.act = e.act;
    p.residual = static_cast<const __nv_bfloat16 *>(e.residual);
    p.y = static_cast<__nv_bfloat16 *>(g.c);
    p.z = static_cast<__nv_bfloat16 *>(e.z);
    p.amax = e.amax;
    p.status = dev.status;
    p.limit_ns = wait_limit_ns();
    static std::once_flag once[64];
    static cudaError_t err[64];
    const int d = dev.ordinal & 63;
    std::call_once(once[d], [&] {
        for (auto *kernel : {gemm_few_kernel<true>, gemm_few_kernel<false>})
            if (err[d] == cudaSuccess)
                err[d] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                              kRingBytes + 1024);
    });
    if (err[d] != cudaSuccess)
        return err[d];
    // the ring, which the partial sums reuse
    const int ring = std::max(p.stages * stage, p.nt * kLanes * 4);
    return launch_pdl_cluster(g.N % 8 == 0 ? gemm_few_kernel<true> : gemm_few_kernel<false>, dim3(static_cast<unsigned>(plan.tiles * p.splits)),
                              dim3(kThreads), static_cast<size_t>(ring) + 1024, stream,
                              static_cast<unsigned>(p.splits), ma, mb, p);
}

} // namespace f8
