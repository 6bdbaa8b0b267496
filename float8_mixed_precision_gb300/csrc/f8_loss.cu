// What stands behind a head linear: log probabilities of given tokens with
// entropy and top alternatives, and the distillation loss against a teacher's
// top logits, forward and backward.
//
// Every kernel walks rows of the logits [rows, vocab], z = logits / T, and is
// bound by HBM: one value read per element forward, one more written backward.
// A row is walked in 16-byte chunks on 16-byte boundaries.  The loops take the
// whole ones; the first and the last chunk of a row that starts or ends inside
// one (the edges) are read element by element by one thread each.
//
// Softmax statistics, one pass: a thread keeps (m, s, h) with m the largest
// logit so far, s = sum e^((x - m) / T) and, for the entropy, h = sum e^d d (d
// in units of log 2), rescaled when m grows.  Pairs join as
//   M = max(m1, m2), f_i = 2^((m_i - M) c), s = s1 f1 + s2 f2,
//   h = f1 (h1 + s1 (m1 - M) c) + f2 (...),   c = log2(e) / T,
// in a fixed order (lanes, warps, blocks of a cluster): equal inputs give
// equal bits.  Then lse = M / T + ln s and entropy = ln s - ln 2 h / s, sums of
// terms of one sign.
//
// A row goes to one block, or where there are fewer rows than keep the SMs busy
// to a cluster of up to eight, each with a stretch of it, joined in the first
// block's shared memory.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "f8_internal.h"
#include "f8_ptx.cuh"
#include "f8_ring.h"

namespace f8 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr float kLn2 = 0.693147180559945309f;
constexpr double kLog2e = 1.44269504088896340736;
// below any exponent that 2^x tells from 0 in fp32; keeps 0 * d finite
constexpr float kFloor2 = -1.0e4f;
// past this an fp32 log-sum-exp no longer tells a row's tokens apart
constexpr float kMaxLse = 16777216.0f;
// The mass p_r outside a row's slots: below kSmallRest its logarithm stands for
// it (sums of exponentials that far below the row's maximum leave fp32), and
// below 2^kNoRest, where 64 bits hold no normal number, there is none.
constexpr float kSmallRest = 7.888609052210118e-31f;  // 2^-100
constexpr float kNoRest = -1022.0f;
#define F8_NEG_INF __int_as_float(0xff800000)
#define F8_POS_INF __int_as_float(0x7f800000)
#define F8_NAN __int_as_float(0x7fffffff)

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ void prefetch_l2(const void *p)
{
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// ------------------------------------------------------------ rows in chunks
template <typename T>
struct Chunk {
    static constexpr int E = 16 / static_cast<int>(sizeof(T));  // elements
};

// One row as 16-byte chunks: chunk c holds elements c * E - off + [0, E).
template <typename T>
struct Row {
    const T *base;    // chunk 0, on a 16-byte boundary
    int64_t at;       // the row's first element in the whole buffer
    int off, vocab;
    int nch, w0, w1;  // chunks, and the whole ones among them: [w0, w1)

    __device__ __forceinline__ Row(const T *p, int64_t row, int64_t ld, int v)
    {
        const T *r = p + row * ld;
        constexpr int E = Chunk<T>::E;
        off = static_cast<int>((reinterpret_cast<uintptr_t>(r) & 15u) / sizeof(T));
        base = r - off;
        at = row * ld;
        vocab = v;
        nch = (off + v + E - 1) / E;
        w0 = off > 0 ? 1 : 0;
        w1 = max(w0, (off + v) / E);
    }
    __device__ __forceinline__ bool whole(int c) const { return c >= w0 && c < w1; }
    // edge i (0: the first chunk, 1: the last) that lies in chunks [c0, c1), or -1
    __device__ __forceinline__ int edge(int i, int c0, int c1) const
    {
        const int c = i == 0 ? 0 : nch - 1;
        const bool is = i < 2 && !whole(c) && (i == 0 || c > 0);
        return is && c >= c0 && c < c1 ? c : -1;
    }
};

// Threads that take the edges of their block's stretch: lane 0 of two warps.
__device__ __forceinline__ int edge_of_thread()
{
    return (threadIdx.x & 31) == 0 ? static_cast<int>(threadIdx.x >> 5) : 2;
}

__device__ __forceinline__ uint4 neg_inf_chunk(__nv_bfloat16)
{
    return make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
}
__device__ __forceinline__ uint4 neg_inf_chunk(float)
{
    return make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u);
}

// Chunk c if it is a whole one below `end`, else -inf.
template <typename T>
__device__ __forceinline__ uint4 load_chunk(const Row<T> &r, int c, int end, int64_t total,
                                            unsigned *status)
{
    constexpr int E = Chunk<T>::E;
    uint4 v = neg_inf_chunk(T());
    if (c >= r.w0 && c < min(end, r.w1) &&
        in_range(r.at - r.off + static_cast<int64_t>(c) * E, E, total, status))
        v = *reinterpret_cast<const uint4 *>(r.base + static_cast<int64_t>(c) * E);
    return v;
}

template <typename T>
__device__ __forceinline__ float as_float(T x);
template <>
__device__ __forceinline__ float as_float<__nv_bfloat16>(__nv_bfloat16 x)
{
    return __bfloat162float(x);
}
template <>
__device__ __forceinline__ float as_float<float>(float x)
{
    return x;
}

// An edge chunk's elements inside the row, -inf elsewhere.
template <typename T>
__device__ __forceinline__ void load_edge(const Row<T> &r, int c, float (&f)[Chunk<T>::E],
                                          int64_t total, unsigned *status)
{
    constexpr int E = Chunk<T>::E;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int v = c * E + e - r.off;
        f[e] = F8_NEG_INF;
        if (v >= 0 && v < r.vocab && in_range(r.at + v, 1, total, status))
            f[e] = as_float(r.base[r.off + v]);
    }
}

// Walks whole chunks [c0, c1) of a row by N threads, U at a time: body(v, c)
// gets the thread's chunks c + u * N, -inf where that is c1 or past it.
template <typename T, int N, int U, typename F>
__device__ __forceinline__ void walk_chunks(const Row<T> &r, int c0, int c1, int64_t total,
                                            unsigned *status, F body)
{
    constexpr int E = Chunk<T>::E;
    const uint4 *p = reinterpret_cast<const uint4 *>(r.base);
    int c = c0 + static_cast<int>(threadIdx.x) % N;
    for (; c + (U - 1) * N < c1; c += U * N) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            v[u] = neg_inf_chunk(T());
            if (in_range(r.at - r.off + static_cast<int64_t>(c + u * N) * E, E, total, status))
                v[u] = p[c + u * N];
        }
        body(v, c);
    }
    if (c < c1) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            v[u] = load_chunk(r, c + u * N, c1, total, status);
        body(v, c);
    }
}

template <typename T>
__device__ __forceinline__ void unpack(uint4 v, float (&f)[Chunk<T>::E]);
template <>
__device__ __forceinline__ void unpack<__nv_bfloat16>(uint4 v, float (&f)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
template <>
__device__ __forceinline__ void unpack<float>(uint4 v, float (&f)[4])
{
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
}

template <typename T>
__device__ __forceinline__ uint4 pack(const float (&f)[Chunk<T>::E]);
template <>
__device__ __forceinline__ uint4 pack<__nv_bfloat16>(const float (&f)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __nv_bfloat162 h = __float22bfloat162_rn(make_float2(f[2 * i], f[2 * i + 1]));
        w[i] = *reinterpret_cast<uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <>
__device__ __forceinline__ uint4 pack<float>(const float (&f)[4])
{
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
}

// A chunk's elements in pairs, for arithmetic on two at a time.
template <typename T>
__device__ __forceinline__ void unpack2(uint4 v, float2 (&f)[Chunk<T>::E / 2]);
template <>
__device__ __forceinline__ void unpack2<__nv_bfloat16>(uint4 v, float2 (&f)[4])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ void unpack2<float>(uint4 v, float2 (&f)[2])
{
    f[0] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
    f[1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
}
template <typename T>
__device__ __forceinline__ uint4 pack2(const float2 (&f)[Chunk<T>::E / 2]);
template <>
__device__ __forceinline__ uint4 pack2<__nv_bfloat16>(const float2 (&f)[4])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __nv_bfloat162 h = __float22bfloat162_rn(f[i]);
        w[i] = *reinterpret_cast<uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <>
__device__ __forceinline__ uint4 pack2<float>(const float2 (&f)[2])
{
    return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x),
                      __float_as_uint(f[1].y));
}

template <int E>
__device__ __forceinline__ float max_of(const float (&f)[E])
{
    float m = f[0];
#pragma unroll
    for (int e = 1; e < E; ++e)
        m = fmaxf(m, f[e]);
    return m;
}

// Two bf16 at a time: the larger of each pair, without (max2) and with
// (max2_nan) a NaN that either holds.
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Element d of a chunk, and the chunk with it replaced; d is no constant, so the
// word is found by selects.
template <typename T>
__device__ __forceinline__ float get_element(uint4 v, int d)
{
    const int i = sizeof(T) == 2 ? d >> 1 : d;
    const uint32_t w = i < 2 ? (i == 0 ? v.x : v.y) : (i == 2 ? v.z : v.w);
    if (sizeof(T) == 2)
        return __uint_as_float(d & 1 ? w & 0xFFFF0000u : w << 16);
    return __uint_as_float(w);
}
template <typename T>
__device__ __forceinline__ uint4 set_element(uint4 v, int d, float x)
{
    uint32_t keep = 0, w = __float_as_uint(x);
    if (sizeof(T) == 2) {
        w = static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(x))) << (16 * (d & 1));
        keep = d & 1 ? 0x0000FFFFu : 0xFFFF0000u;
    }
    const int i = sizeof(T) == 2 ? d >> 1 : d;
    v.x = i == 0 ? (v.x & keep) | w : v.x;
    v.y = i == 1 ? (v.y & keep) | w : v.y;
    v.z = i == 2 ? (v.z & keep) | w : v.z;
    v.w = i == 3 ? (v.w & keep) | w : v.w;
    return v;
}

// The largest element of a chunk (a NaN only if all are).
template <typename T>
__device__ __forceinline__ float chunk_max(uint4 v);
template <>
__device__ __forceinline__ float chunk_max<__nv_bfloat16>(uint4 v)
{
    const uint32_t m = max2(max2(v.x, v.y), max2(v.z, v.w));
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float chunk_max<float>(uint4 v)
{
    return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)),
                 fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
}

// No element of a chunk below `low` (elements pairwise in one register for
// bf16, whose `low` then is rounded to bf16).
template <typename T>
__device__ __forceinline__ uint4 chunk_floor(uint4 v, float low);
template <>
__device__ __forceinline__ uint4 chunk_floor<__nv_bfloat16>(uint4 v, float low)
{
    const __nv_bfloat162 h = __float22bfloat162_rn(make_float2(low, low));
    const uint32_t l = *reinterpret_cast<const uint32_t *>(&h);
    return make_uint4(max2_nan(v.x, l), max2_nan(v.y, l), max2_nan(v.z, l), max2_nan(v.w, l));
}
template <>
__device__ __forceinline__ uint4 chunk_floor<float>(uint4 v, float low)
{
    return make_uint4(__float_as_uint(max_nan(__uint_as_float(v.x), low)),
                      __float_as_uint(max_nan(__uint_as_float(v.y), low)),
                      __float_as_uint(max_nan(__uint_as_float(v.z), low)),
                      __float_as_uint(max_nan(__uint_as_float(v.w), low)));
}

// ------------------------------------------------------------ softmax sums
struct Stats {
    float m, s, h;  // h only where the entropy is wanted
};

__device__ __forceinline__ Stats stats_empty() { return Stats{F8_NEG_INF, 0.0f, 0.0f}; }

// The sums' reference grows to bm.
template <bool ENT>
__device__ __forceinline__ void raise_max(Stats &t, float bm, float c)
{
    if (bm > t.m) {
        const float d = fmaxf((t.m - bm) * c, kFloor2);
        const float r = ex2(d);
        if (ENT)
            t.h = r * fmaf(t.s, d, t.h);
        t.s *= r;
        t.m = bm;
    }
}

// Adds N values to the running sums, whatever they are.
template <bool ENT, int N>
__device__ __forceinline__ void add_values(Stats &t, const float (&f)[N], float c)
{
    raise_max<ENT>(t, max_of(f), c);
    const float m = t.m == F8_NEG_INF ? 0.0f : t.m;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const float d = (f[e] - m) * c;
        const float x = ex2(d);
        t.s += x;
        if (ENT)
            t.h = fmaf(x, fmaxf(d, kFloor2), t.h);
    }
}

// Past this m c (in units of log 2) the sums take add_values' steps.
constexpr float kFastRange = 4096.0f;

// Adds U chunks.  Where the maximum is of ordinary size the exponent is one
// fused multiply-add, x c - mc with mc = fl(m c), two elements per
// instruction; r = m c - mc, which every term then carries as a factor 2^r, is
// taken out of the sums at the end.  For the entropy the elements are first
// raised to 200 / c below the maximum, which leaves their 2^d at 0 and keeps
// 0 * d finite for masked tokens.
template <typename T, bool ENT, int U>
__device__ __forceinline__ void add_chunks(Stats &t, const uint4 (&v)[U], float c, float inv_c)
{
    constexpr int E = Chunk<T>::E;
    float bm = chunk_max<T>(v[0]);
#pragma unroll
    for (int u = 1; u < U; ++u)
        bm = fmaxf(bm, chunk_max<T>(v[u]));
    raise_max<ENT>(t, bm, c);
    const float mc = t.m * c;
    if (!(fabsf(mc) < kFastRange)) {
#pragma unroll 1
        for (int u = 0; u < U; ++u) {
            uint4 w = v[0];
#pragma unroll
            for (int j = 1; j < U; ++j)
                w = u == j ? v[j] : w;
            float f[E];
            unpack<T>(w, f);
            add_values<ENT>(t, f, c);
        }
        return;
    }
    const float r = fmaf(t.m, c, -mc);
    const float low = t.m - 200.0f * inv_c;
    const float2 c2 = make_float2(c, c), n2 = make_float2(-mc, -mc);
    float2 s[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
    float2 h[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float2 f[E / 2];
        unpack2<T>(ENT ? chunk_floor<T>(v[u], low) : v[u], f);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
            const float2 d = __ffma2_rn(f[e], c2, n2);
            const float2 x = make_float2(ex2(d.x), ex2(d.y));
            s[e & 1] = __fadd2_rn(s[e & 1], x);
            if (ENT)
                h[e & 1] = __ffma2_rn(x, d, h[e & 1]);
        }
    }
    const float bs = (s[0].x + s[0].y) + (s[1].x + s[1].y);
    const float corr = fmaf(-r, kLn2, 1.0f);
    t.s = fmaf(bs, corr, t.s);
    if (ENT) {
        const float bh = (h[0].x + h[0].y) + (h[1].x + h[1].y);
        t.h = fmaf(fmaf(-r, bs, bh), corr, t.h);
    }
}

// The largest value of a warp's lanes (a NaN only if all are).
__device__ __forceinline__ float warp_max_of(float v)
{
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// The joined sums of N lanes (each lane's of its N lanes' group), in every lane:
// the maximum first, so that each lane rescales once; sums in a fixed order.
template <bool ENT, int N>
__device__ __forceinline__ Stats warp_stats(Stats t, float c)
{
    float m = t.m;
    if (N == 32) {
        m = warp_max_of(m);
    } else {
#pragma unroll
        for (int o = N / 2; o > 0; o >>= 1)
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    }
    const float d = fmaxf((t.m - m) * c, kFloor2), f = ex2(d);
    t.m = m;
    if (ENT)
        t.h = f * fmaf(t.s, d, t.h);
    t.s *= f;
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) {
        t.s += __shfl_xor_sync(0xFFFFFFFFu, t.s, o);
        if (ENT)
            t.h += __shfl_xor_sync(0xFFFFFFFFu, t.h, o);
    }
    return t;
}

// The block's sums, in every thread.  `red`: one Stats per warp.
template <bool ENT>
__device__ __forceinline__ Stats block_join(Stats t, float c, Stats *red)
{
    t = warp_stats<ENT, 32>(t, c);
    if ((threadIdx.x & 31) == 0)
        red[threadIdx.x >> 5] = t;
    __syncthreads();
    return warp_stats<ENT, kWarps>(red[threadIdx.x & (kWarps - 1)], c);
}

// The sums of `n` blocks, in every thread.
template <bool ENT>
__device__ __forceinline__ Stats cluster_stats(const Stats *parts, int n, float c)
{
    const int i = threadIdx.x & (kMaxCluster - 1);
    return warp_stats<ENT, kMaxCluster>(i < n ? parts[i] : stats_empty(), c);
}

// ------------------------------------------------------------ clusters
// A block of a cluster may write another's shared memory once that block has
// started (cluster_started, an arrive at the kernel's start and a wait before
// the first write) and until cluster_join, after which the writes can be read.
__device__ __forceinline__ void cluster_start()
{
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_started()
{
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_join()
{
    __syncwarp();
    cluster_sync();
}
// The same shared variable in block `rank` of the cluster.
template <typename P>
__device__ __forceinline__ P *peer(P *p, unsigned rank)
{
    return cooperative_groups::this_cluster().map_shared_rank(p, rank);
}

// ------------------------------------------------------------ top k
// fp32 values as unsigned keys of the same order, never 0; -0 counts as +0,
// any NaN as the largest.
__device__ __forceinline__ uint32_t order_key(float x)
{
    const uint32_t b = __float_as_uint(x + 0.0f);
    const uint32_t k = b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
    return x != x ? 0xFFFFFFFFu : k;
}
__device__ __forceinline__ float key_value(uint32_t k)
{
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// How many of the n keys are >= t; `red`: one word per warp.
__device__ __forceinline__ int count_from(const uint32_t *keys, int n, uint32_t t, int *red)
{
    int c = 0;
    for (int i0 = 0; i0 < n; i0 += kThreads) {
        const int i = i0 + static_cast<int>(threadIdx.x);
        c += __popc(__ballot_sync(0xFFFFFFFFu, i < n && keys[i] >= t));
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        red[threadIdx.x >> 5] = c;
    __syncthreads();
    c = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        c += red[w];
    return c;
}

// The positions of the k largest of n keys in shared memory (equal keys: the
// lower positions), ascending, in out[0 .. min(k, n)), by bisection over the
// key range; n < 2^16.
__device__ __forceinline__ void block_select(const uint32_t *keys, int n, int k, int *out, int *red)
{
    const int tid = threadIdx.x, lane = tid & 31;
    if (n <= k) {
        for (int i = tid; i < n; i += kThreads)
            out[i] = i;
        __syncthreads();
        return;
    }
    uint32_t lo = 0xFFFFFFFFu, hi = 0;
    for (int i = tid; i < n; i += kThreads) {
        lo = min(lo, keys[i]);
        hi = max(hi, keys[i]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        lo = min(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
        hi = max(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
    }
    __syncthreads();
    if (lane == 0) {
        red[tid >> 5] = static_cast<int>(lo);
        red[kWarps + (tid >> 5)] = static_cast<int>(hi);
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        lo = min(lo, static_cast<uint32_t>(red[w]));
        hi = max(hi, static_cast<uint32_t>(red[kWarps + w]));
    }
    // at least k keys are >= lo, fewer than k are > hi
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2 + 1;
        const int c = count_from(keys, n, mid, red);
        if (c >= k)
            lo = mid;
        else
            hi = mid - 1;
        if (c == k)
            break;
    }
    // every key > lo, and the first of those == lo until k are found
    const int per = (n + kThreads - 1) / kThreads;
    const int i0 = min(n, tid * per), i1 = min(n, i0 + per);
    int gt = 0, eq = 0;
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
        gt += keys[i] > lo ? 1 : 0;
        eq += keys[i] == lo ? 1 : 0;
    }
    const int packed = (gt << 16) | eq;  // exclusive sums over the block
    int incl = packed;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        incl += lane >= o ? u : 0;
    }
    __syncthreads();
    if (lane == 31)
        red[tid >> 5] = incl;
    __syncthreads();
    int before = incl - packed, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        before += w < (tid >> 5) ? red[w] : 0;
        all += red[w];
    }
    const int need = k - (all >> 16);
    int a = before >> 16, b = before & 0xFFFF;
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
        if (keys[i] > lo) {
            out[a + min(b, need)] = i;
            ++a;
        } else if (keys[i] == lo) {
            if (b < need)
                out[a + b] = i;
            ++b;
        }
    }
    __syncthreads();
}

// The k-th largest of the block's keys, one per thread (k <= kThreads), by seven
// pivots a round: the largest t with at least k keys >= t, or a lower one with
// few more than k.  `cnt`: three sets of eight counters, zero at the start.
__device__ __forceinline__ uint32_t block_threshold(uint32_t key, int k, int *red, int *cnt)
{
    const int tid = threadIdx.x, lane = tid & 31;
    uint32_t lo = __reduce_min_sync(0xFFFFFFFFu, key), hi = __reduce_max_sync(0xFFFFFFFFu, key);
    if (lane == 0) {
        red[tid >> 5] = static_cast<int>(lo);
        red[kWarps + (tid >> 5)] = static_cast<int>(hi);
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        lo = min(lo, static_cast<uint32_t>(red[w]));
        hi = max(hi, static_cast<uint32_t>(red[kWarps + w]));
    }
    // at least k keys are >= lo, fewer than k are > hi
    int set = 0;
    while (lo < hi) {
        const uint32_t step = (hi - lo) / 8 + 1;
        const int pivots = static_cast<int>((hi - lo) / step);  // those up to hi, 1 .. 7
        int mine = 0;
#pragma unroll
        for (int p = 0; p < 7; ++p) {
            const int c = __popc(__ballot_sync(0xFFFFFFFFu, key >= lo + (p + 1) * step));
            mine = lane == p ? c : mine;
        }
        if (lane < pivots && mine > 0)
            atomicAdd(&cnt[8 * set + lane], mine);
        const int next = set == 2 ? 0 : set + 1;
        if (tid < 8)
            cnt[8 * next + tid] = 0;
        __syncthreads();
        // the last pivot that at least k keys reach
        const int have = lane < pivots ? cnt[8 * set + lane] : 0;
        const int above = __popc(__ballot_sync(0xFFFFFFFFu, have >= k));
        const int at = __shfl_sync(0xFFFFFFFFu, have, above > 0 ? above - 1 : 0);
        if (above < pivots)
            hi = lo + (above + 1) * step - 1;
        lo += above * step;
        set = next;
        if (above > 0 && at <= k + k / 4)
            break;
    }
    return lo;
}

// A value's key and its position as one number: of two items the larger comes
// first, by value, then by position.  0 is no item.
__device__ __forceinline__ uint64_t item_of(uint32_t key, int id)
{
    return static_cast<uint64_t>(key) << 32 | ~static_cast<uint32_t>(id);
}
__device__ __forceinline__ uint32_t item_key(uint64_t v) { return static_cast<uint32_t>(v >> 32); }
__device__ __forceinline__ int item_id(uint64_t v)
{
    return static_cast<int>(~static_cast<uint32_t>(v));
}

// Shared memory of the top-k stage, in 4-byte words; every part starts on a
// 16-byte boundary.
constexpr int kCandidates = 2048;
struct TopLayout {
    int groups, list, keys, pick, cand, best, merge, words;
};
__host__ __device__ inline int words4(int n) { return (n + 3) & ~3; }
__host__ __device__ inline TopLayout top_layout(int ngroups, int k, int cluster)
{
    TopLayout l;
    l.groups = 0;                         // one key per group of 32 chunks
    l.list = l.groups + words4(ngroups);  // k positions
    l.keys = l.list + words4(k);          // 32 k chunk keys
    l.pick = l.keys + 32 * k;             // k chunks
    l.cand = l.pick + words4(k);          // items from here on, two words each
    l.best = l.cand + 2 * kCandidates;    // the block's k best, in order
    l.merge = l.best + words4(2 * k);     // every block's, in the cluster's first
    l.words = l.merge + (cluster > 1 ? words4(2 * cluster * k) : 0);
    return l;
}

// The k largest elements of chunks [32 g0, 32 g1) of a row, in order, in the
// items `best` of `lay`; gkeys holds the groups' largest keys, tkey the
// key of the largest element that this thread has seen.  The k-th largest of
// the threads' is no larger than the k-th largest element, so: that threshold,
// a look at the groups that reach it, and their elements >= it ranked against
// one another.  Where many values are equal to the threshold, fewer than k
// threads have seen any, or some have seen very many large ones, the candidates
// may not fit; then parts are chosen exactly (k parts hold all, by maximum and
// position), groups, chunks, elements in turn.
template <typename T>
__device__ __forceinline__ void block_top(const Row<T> &r, int g0, int g1, int k, int have,
                                          uint32_t tkey, uint32_t *dyn, const TopLayout &lay,
                                          int *red, int *cnt, int *ncand, int64_t total,
                                          unsigned *status)
{
    constexpr int E = Chunk<T>::E;
    const int tid = threadIdx.x, lane = tid & 31;
    uint32_t *gkeys = dyn + lay.groups, *keys = dyn + lay.keys;
    uint64_t *cand = reinterpret_cast<uint64_t *>(dyn + lay.cand);
    uint64_t *best = reinterpret_cast<uint64_t *>(dyn + lay.best);
    int *list = reinterpret_cast<int *>(dyn + lay.list);
    const int ng = g1 - g0;
    auto load = [&](int ch, float (&x)[E]) {
        if (r.whole(ch))
            unpack<T>(load_chunk(r, ch, r.nch, total, status), x);
        else
            load_edge(r, ch, x, total, status);
    };
    auto offer = [&](int ch, const float(&x)[E], uint32_t t) {
        if (order_key(max_of(x)) < t)
            return;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int v = ch * E + e - r.off;
            const uint32_t key = order_key(x[e]);
            if (v >= 0 && v < r.vocab && key >= t) {
                const int at = atomicAdd(ncand, 1);
                if (at < kCandidates)
                    cand[at] = item_of(key, v);
            }
        }
    };
    auto chunk_keys = [&](const int *groups, int n) {
        for (int i = tid; i < n * 32; i += kThreads) {
            const int ch = (g0 + groups[i >> 5]) * 32 + (i & 31);
            uint32_t key = 0;
            if (ch < r.nch) {
                float x[E];
                load(ch, x);
                key = order_key(max_of(x));
            }
            keys[i] = key;
        }
        __syncthreads();
    };
    const uint32_t t = block_threshold(tkey, k, red, cnt);
    // a lane asks for a group, its warp looks at those that reach t, kLook at a
    // time; neighbouring groups go to different warps
    constexpr int kLook = 4;
    for (int i = tid >> 5; i < ng; i += kThreads) {
        unsigned reach = __ballot_sync(0xFFFFFFFFu, i + lane * kWarps < ng && gkeys[i + lane * kWarps] >= t);
        while (reach != 0) {
            int ch[kLook];
            uint4 v[kLook];
#pragma unroll
            for (int u = 0; u < kLook; ++u) {
                ch[u] = reach != 0 ? (g0 + i + (__ffs(reach) - 1) * kWarps) * 32 + lane : r.nch;
                reach &= reach - 1;
                v[u] = load_chunk(r, ch[u], r.nch, total, status);
            }
#pragma unroll
            for (int u = 0; u < kLook; ++u) {
                if (ch[u] < r.nch) {
                    float x[E];
                    if (r.whole(ch[u]))
                        unpack<T>(v[u], x);
                    else
                        load_edge(r, ch[u], x, total, status);
                    offer(ch[u], x, t);
                }
            }
        }
    }
    __syncthreads();
    int n = *ncand;
    if (n > kCandidates) {
        block_select(gkeys, ng, k, list, red);
        const int kg = min(k, ng);
        chunk_keys(list, kg);
        int *pick = reinterpret_cast<int *>(dyn + lay.pick);
        block_select(keys, kg * 32, k, pick, red);
        const int kc = min(k, kg * 32);
        for (int i = tid; i < kc; i += kThreads)
            pick[i] = (g0 + list[pick[i] >> 5]) * 32 + (pick[i] & 31);
        __syncthreads();
        for (int i = tid; i < kc * E; i += kThreads) {
            const int v = pick[i / E] * E + i % E - r.off;
            const bool in = v >= 0 && v < r.vocab;
            cand[i] = in ? item_of(order_key(as_float(r.base[r.off + v])), v) : 0u;
        }
        __syncthreads();
        n = kc * E;
    }
    // each candidate's rank among them
    for (int i = tid; i < n; i += kThreads) {
        const uint64_t v = cand[i];
        int place = 0;
#pragma unroll 8
        for (int j = 0; j < n; ++j)
            place += cand[j] > v ? 1 : 0;
        if (place < have)
            best[place] = v;
    }
    for (int i = have + tid; i < k; i += kThreads)
        best[i] = 0;
    __syncthreads();
}

// ------------------------------------------------------------ log probabilities
struct LogprobArgs {
    const void *logits;
    int64_t rows, ld;
    int vocab, top_k, cluster;
    const int64_t *tokens;
    float inv_t, c, inv_c;  // 1 / T, log2(e) / T, T / log2(e)
    float *logp, *entropy, *lse;
    int32_t *top_ids;
    float *top_logp;
    unsigned *status;
};

constexpr int kUnroll = 4;  // chunks in flight per thread

// TOP: the largest of every 32 consecutive chunks (what one warp loads at once)
// is kept in shared memory, so the row is read once plus the few groups that
// block_top looks at again, from L2.
// bf16 4096 x 131072: 152 us, at the copy rate; with the top 8 175 us, 6.0 TB/s
// (a second look's latency per row, with the other blocks' loads behind it).
// 4 x 131072 with the top 20: 9 us, of which a megabyte's bytes are 0.2: the
// steps after one another bound it.  Loading a step ahead in registers costs
// blocks per SM: 199 against 178 us with the top 8.
template <typename T, bool TOP>
__global__ void __launch_bounds__(kThreads)
logprobs_kernel(const __grid_constant__ LogprobArgs a)
{
    constexpr int E = Chunk<T>::E;
    extern __shared__ __align__(16) uint32_t dyn[];
    __shared__ Stats red[kWarps];
    __shared__ Stats parts[kMaxCluster];
    __shared__ int sred[2 * kWarps];
    __shared__ int cnt[24];
    __shared__ int ncand;
    if (TOP && threadIdx.x < 24)
        cnt[threadIdx.x] = 0;
    if (TOP && threadIdx.x == 0)
        ncand = 0;
    griddep_wait();
    griddep_launch_dependents();
    const int C = a.cluster;
    const int64_t row = blockIdx.x / C;
    const int rank = static_cast<int>(blockIdx.x % C);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t tok = a.tokens != nullptr ? a.tokens[row] : 0;
    if (tok < 0) {  // the whole cluster leaves
        if (rank == 0) {
            if (tid == 0) {
                if (a.logp != nullptr)
                    a.logp[row] = 0.0f;
                if (a.entropy != nullptr)
                    a.entropy[row] = 0.0f;
                if (a.lse != nullptr)
                    a.lse[row] = 0.0f;
            }
            if (TOP && tid < a.top_k) {
                a.top_ids[row * a.top_k + tid] = -1;
                a.top_logp[row * a.top_k + tid] = F8_NEG_INF;
            }
        }
        return;
    }
    if (C > 1)
        cluster_start();
    const Row<T> r(static_cast<const T *>(a.logits), row, a.ld, a.vocab);
    const int64_t total = (a.rows - 1) * a.ld + a.vocab;
    // groups of 32 chunks, dealt to the cluster's blocks in stretches
    const int ngroups = (r.nch + 31) / 32;
    const int per = (ngroups + C - 1) / C;
    const int g0 = min(ngroups, rank * per), g1 = min(ngroups, g0 + per);
    const int per_max = ((r.vocab + E - 1 + E) / E + 31) / 32;  // any row offset
    const TopLayout lay = top_layout((per_max + C - 1) / C, a.top_k, C);
    uint32_t *gkeys = dyn + lay.groups;

    // a warp takes kUnroll groups at a time; their largest elements as floats
    // first, as keys once all are there
    float *gmax = reinterpret_cast<float *>(gkeys);
    Stats t = stats_empty();
    auto add = [&](const uint4(&v)[kUnroll], int g) {
        if (TOP) {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const float m = warp_max_of(chunk_max<T>(v[u]));
                if (lane == u && g + u < g1)
                    gmax[g + u - g0] = m;
            }
        }
        add_chunks<T, true>(t, v, a.c, a.inv_c);
    };
    for (int g = g0 + warp * kUnroll; g < g1; g += kWarps * kUnroll) {
        uint4 v[kUnroll];
        const int c = g * 32 + lane;
        if (g * 32 >= r.w0 && (g + kUnroll) * 32 <= min(g1 * 32, r.w1)) {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                v[u] = neg_inf_chunk(T());
                if (in_range(r.at - r.off + static_cast<int64_t>(c + 32 * u) * E, E, total, a.status))
                    v[u] = reinterpret_cast<const uint4 *>(r.base)[c + 32 * u];
            }
        } else {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                v[u] = load_chunk(r, c + 32 * u, g1 * 32, total, a.status);
        }
        add(v, g);
    }
    const int ec = r.edge(edge_of_thread(), g0 * 32, g1 * 32);
    float edge_max = F8_NEG_INF;
    if (ec >= 0) {
        float x[E];
        load_edge(r, ec, x, total, a.status);
        add_values<true>(t, x, a.c);
        edge_max = max_of(x);
    }
    if (TOP) {
        __syncthreads();
        for (int i = tid; i < g1 - g0; i += kThreads)
            gkeys[i] = order_key(gmax[i]);
        __syncthreads();
        if (ec >= 0)
            atomicMax(&gkeys[ec / 32 - g0], order_key(edge_max));
    }
    const uint32_t tkey = order_key(t.m);
    t = block_join<true>(t, a.c, red);

    if (TOP) {
        const int k = a.top_k;
        const int v0 = g0 * 32 * E - r.off, v1 = min(g1 * 32 * E - r.off, r.vocab);
        const int have = max(0, min(k, v1 - max(v0, 0)));
        block_top<T>(r, g0, g1, k, have, tkey, dyn, lay, sred, cnt, &ncand, total, a.status);
        if (C > 1) {  // into the leader's merge arrays
            cluster_started();
            const uint64_t *best = reinterpret_cast<const uint64_t *>(dyn + lay.best);
            uint64_t *m = peer(reinterpret_cast<uint64_t *>(dyn + lay.merge) + rank * k, 0);
            for (int i = tid; i < k; i += kThreads)
                m[i] = best[i];
        }
    } else if (C > 1) {
        cluster_started();
    }
    if (C > 1) {
        if (tid == 0)
            *peer(&parts[rank], 0) = t;
        cluster_join();
        if (rank != 0)
            return;
        t = cluster_stats<true>(parts, C, a.c);
    } else {
        __syncthreads();
    }

    const bool none = t.m == F8_NEG_INF && t.s == 0.0f;
    const float ls = logf(t.s);
    float lse = fmaf(t.m, a.inv_t, ls);
    if (t.s != t.s || t.m == F8_POS_INF) {
        lse = F8_NAN;
        if (tid == 0)
            atomicOr(a.status, kStatusNonfinite);
    }
    if (none)
        lse = F8_NEG_INF;
    if (tid == 0) {
        if (a.lse != nullptr)
            a.lse[row] = lse;
        if (a.entropy != nullptr)
            // both are of one sign by definition, also where they round to 0
            a.entropy[row] = none ? 0.0f : (lse != lse ? F8_NAN : fmaxf(ls - kLn2 * t.h / t.s, 0.0f));
        if (a.logp != nullptr) {
            // from the difference to the maximum: |logits| does not cancel
            float lp = F8_NAN;
            if (tok >= r.vocab)
                atomicOr(a.status, kStatusIndex);
            else if (none)
                lp = F8_NEG_INF;
            else if (lse == lse)
                lp = fminf((as_float(r.base[r.off + tok]) - t.m) * a.inv_t - ls, 0.0f);
            a.logp[row] = lp;
        }
    }
    if (TOP) {
        const int k = a.top_k;
        auto put = [&](int place, uint64_t v) {
            a.top_ids[row * k + place] = item_id(v);
            a.top_logp[row * k + place] =
                none ? F8_NEG_INF
                     : (lse != lse ? F8_NAN
                                   : fminf((key_value(item_key(v)) - t.m) * a.inv_t - ls, 0.0f));
        };
        if (C == 1) {
            const uint64_t *best = reinterpret_cast<const uint64_t *>(dyn + lay.best);
            for (int i = tid; i < k; i += kThreads)
                put(i, best[i]);
            return;
        }
        // the blocks' lists are in order: an item's place is its own plus how many
        // of each other list come before it; the lists' first items first, so that
        // whole warps are done once their items have dropped out
        constexpr int kLists = 4;
        const uint64_t *m = reinterpret_cast<const uint64_t *>(dyn + lay.merge);
        const int half = 1 << (31 - __clz(k));  // the largest power of two <= k
        for (int i = tid; i < C * k; i += kThreads) {
            const int own = i % C;
            int place = i / C;
            const uint64_t v = m[own * k + place];
            for (int l = 0; l < C && place < k; l += kLists) {
                int at[kLists] = {};
                for (int s = half; s > 0; s >>= 1) {
                    uint64_t o[kLists];  // loads without branches between them
#pragma unroll
                    for (int u = 0; u < kLists; ++u)
                        o[u] = m[min(l + u, C - 1) * k + min(at[u] + s, k) - 1];
#pragma unroll
                    for (int u = 0; u < kLists; ++u)
                        at[u] += at[u] + s <= k && o[u] > v ? s : 0;
                }
#pragma unroll
                for (int u = 0; u < kLists; ++u)
                    place += l + u == own || l + u >= C ? 0 : at[u];
            }
            if (v > 0 && place < k)
                put(place, v);
        }
    }
}

// ------------------------------------------------------------ gradients' output
struct OutArgs {
    void *p;
    int64_t ld;
    unsigned *amax;
};

// Where a row of the gradient goes.
template <typename T>
struct OutRow {
    T *p;
    int64_t at, total;  // the row's first element in the whole buffer, and its size
    bool same;          // starts at the logits row's offset from a 16-byte boundary

    __device__ __forceinline__ OutRow(const OutArgs &o, int64_t rows, int64_t row, const Row<T> &r)
    {
        at = row * o.ld;
        p = static_cast<T *>(o.p) + at;
        total = rows * o.ld;
        same = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T)) == r.off;
    }
};

// Magnitude bits of two bf16 in each word, folded into a running maximum.
__device__ __forceinline__ uint32_t abs_max(uint32_t m, uint4 v)
{
    return __vmaxu2(__vmaxu2(m, __vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu)),
                    __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
}

// Elements of chunk c that lie in the row, one by one; m2: running maximum of
// the stored bf16 values' magnitude bits.
template <typename T>
__device__ __forceinline__ void store_elements(const Row<T> &r, const OutRow<T> &o, int c,
                                               const float (&f)[Chunk<T>::E], uint32_t &m2,
                                               unsigned *status)
{
    constexpr int E = Chunk<T>::E;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int i = c * E + e - r.off;
        const T v = static_cast<T>(f[e]);
        if (i >= 0 && i < r.vocab && in_range(o.at + i, 1, o.total, status)) {
            o.p[i] = v;
            if (sizeof(T) == 2)
                m2 = __vmaxu2(m2, (__float_as_uint(as_float(v)) >> 16) & 0x7FFFu);
        }
    }
}

// Writes U whole chunks c + u * N, those below `end`: vectors where the output
// row has the input row's offset, else element by element.
template <typename T, int N, int U>
__device__ __forceinline__ void store_chunks(const Row<T> &r, const OutRow<T> &o, int c, int end,
                                             const uint4 (&v)[U], bool amax, uint32_t &m2,
                                             unsigned *status)
{
    constexpr int E = Chunk<T>::E;
    if (!o.same) {
#pragma unroll 1
        for (int u = 0; u < U; ++u) {
            uint4 w = v[0];
#pragma unroll
            for (int j = 1; j < U; ++j)
                w = u == j ? v[j] : w;
            float f[E];
            unpack<T>(w, f);
            if (c + u * N < end)
                store_elements(r, o, c + u * N, f, m2, status);
        }
        return;
    }
    uint4 *p = reinterpret_cast<uint4 *>(o.p + (static_cast<int64_t>(c) * E - r.off));
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (c + u * N < end && in_range(o.at + static_cast<int64_t>(c + u * N) * E - r.off, E,
                                        o.total, status))
            p[u * N] = v[u];
    if (amax) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c + u * N < end)
                m2 = abs_max(m2, v[u]);
    }
}

// Zeros in columns [from, to) of an output row, by n threads of which this is
// number t: 16-byte pieces, and single elements at the ends.
template <typename T>
__device__ __forceinline__ void zero_columns(const OutRow<T> &o, int64_t from, int64_t to, int t,
                                             int n, unsigned *status)
{
    constexpr int64_t E = Chunk<T>::E;
    if (from >= to)
        return;
    const int64_t lead = (E - static_cast<int64_t>((reinterpret_cast<uintptr_t>(o.p + from) & 15u) /
                                                   sizeof(T))) % E;
    const int64_t v0 = min(from + lead, to), nv = (to - v0) / E;
    for (int64_t i = from + t; i < v0; i += n)
        if (in_range(o.at + i, 1, o.total, status))
            o.p[i] = T(0.0f);
    for (int64_t i = t; i < nv; i += n)
        if (in_range(o.at + v0 + i * E, E, o.total, status))
            *reinterpret_cast<uint4 *>(o.p + v0 + i * E) = make_uint4(0, 0, 0, 0);
    for (int64_t i = v0 + nv * E + t; i < to; i += n)
        if (in_range(o.at + i, 1, o.total, status))
            o.p[i] = T(0.0f);
}

// One atomicMax per block on the fp32 pattern of a zeroed word (the result
// does not depend on the order).
__device__ __forceinline__ void block_amax(uint32_t m2, unsigned *amax, unsigned *status)
{
    __shared__ unsigned blk;
    if (amax == nullptr)
        return;
    __syncthreads();
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
        atomicMax(amax, blk << 16);
    }
}

// p = norm 2^((x a + b) s): the softmax of an element x from the maximum
// (a 1, b -max, s c, norm 1 / sum) or from lse (a 1 / T, b -lse, s log2 e, norm 1).
struct Softmax {
    float a, b, s, norm;

    __device__ __forceinline__ float exponent(float x) const { return fmaf(x, a, b) * s; }
    __device__ __forceinline__ float2 exponent(float2 x) const
    {
        return __fmul2_rn(__ffma2_rn(x, make_float2(a, a), make_float2(b, b)), make_float2(s, s));
    }
};

// factor p / norm of a chunk's elements.
template <typename T>
__device__ __forceinline__ uint4 scaled_softmax(uint4 v, const Softmax &k, float factor)
{
    constexpr int E = Chunk<T>::E;
    float2 f[E / 2];
    unpack2<T>(v, f);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
        const float2 d = k.exponent(f[e]);
        f[e] = __fmul2_rn(make_float2(ex2(d.x), ex2(d.y)), make_float2(factor, factor));
    }
    return pack2<T>(f);
}

// Blocks of the backward kernels take this many chunks of a row each.
constexpr int kBwdChunks = 16 * kThreads;

// ------------------------------------------------------------ log probabilities, backward
struct LogprobBwdArgs {
    const void *logits;
    int64_t rows, ld;
    int vocab, blocks_per_row;
    const int64_t *tokens;
    const float *lse, *entropy, *dlogp, *dentropy;
    float inv_t, t;  // 1 / T, T
    OutArgs out;
    unsigned *status;
};

// With l = log p, the gradient of a and h is
//   (a 1[v = token] - p (a + h (l + H))) / T,
// for most elements p times a linear function of l.  With an entropy gradient
// the logits are first raised to where p is 0 in fp32 and l still finite.
template <typename T>
__global__ void __launch_bounds__(kThreads)
logprobs_bwd_kernel(const __grid_constant__ LogprobBwdArgs a)
{
    constexpr int E = Chunk<T>::E;
    griddep_wait();
    griddep_launch_dependents();
    const int64_t row = blockIdx.x / a.blocks_per_row;
    const int part = static_cast<int>(blockIdx.x % a.blocks_per_row);
    const int tid = threadIdx.x;
    const Row<T> r(static_cast<const T *>(a.logits), row, a.ld, a.vocab);
    const int64_t total = (a.rows - 1) * a.ld + a.vocab;
    const OutRow<T> o(a.out, a.rows, row, r);
    const int64_t tok = a.tokens != nullptr ? a.tokens[row] : -1;
    const float ga = a.dlogp != nullptr && a.tokens != nullptr ? a.dlogp[row] : 0.0f;
    const float gh = a.dentropy != nullptr ? a.dentropy[row] : 0.0f;
    const float lse = a.lse[row];
    const bool skip = (a.tokens != nullptr && tok < 0) || (ga == 0.0f && gh == 0.0f) ||
                      fabsf(lse) >= kMaxLse;
    const bool amax = a.out.amax != nullptr;
    if (tok >= r.vocab && tid == 0)
        atomicOr(a.status, kStatusIndex);
    uint32_t m2 = 0;
    const int c0 = part * kBwdChunks, c1 = min(r.nch, c0 + kBwdChunks);
    const int wb = max(c0, r.w0), we = min(c1, r.w1);
    if (skip) {
        zero_columns(o, max(static_cast<int64_t>(c0) * E - r.off, static_cast<int64_t>(0)),
                     min(static_cast<int64_t>(c1) * E - r.off, static_cast<int64_t>(r.vocab)), tid,
                     kThreads, a.status);
    } else {
        const float H = gh != 0.0f ? a.entropy[row] : 0.0f;
        const Softmax k{a.inv_t, -lse, static_cast<float>(kLog2e), 1.0f};
        const float fa = ga * a.inv_t, fh = gh * a.inv_t;
        const float f0 = -fmaf(fh, H, fa), f1 = -fh;  // dense part: p (f0 + f1 l)
        const int tok_chunk = tok >= 0 && tok < r.vocab ? (static_cast<int>(tok) + r.off) / E : -1;
        auto elements = [&](int ch, float (&f)[E]) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float l = fmaf(f[e], k.a, k.b);
                const float p = ex2(l * k.s);
                const float g = p * fmaf(f1, fmaxf(l, kFloor2), f0);
                f[e] = ch * E + e - r.off == tok ? fa + g : g;
            }
        };
        // the elements' floor: l = -140, where p is 0.  chunk_floor rounds it to
        // the logits' type, which moves l by up to 2^-9 |lse - 140| for bf16: 8 in
        // the range where it is used.
        const float low = (lse - 140.0f) * a.t;
        const bool dense = gh == 0.0f;
        const bool ordinary = fabsf(low) < kFastRange && fabsf(lse - 140.0f) < kFastRange;
        walk_chunks<T, kThreads, kUnroll>(r, wb, we, total, a.status, [&](uint4(&v)[kUnroll], int c) {
            uint4 g[kUnroll];
            if (dense) {
#pragma unroll
                for (int u = 0; u < kUnroll; ++u)
                    g[u] = scaled_softmax<T>(v[u], k, f0);
            } else {
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    float2 f[E / 2];
                    unpack2<T>(chunk_floor<T>(v[u], low), f);
#pragma unroll
                    for (int e = 0; e < E / 2; ++e) {
                        const float2 l = __ffma2_rn(f[e], make_float2(k.a, k.a), make_float2(k.b, k.b));
                        const float2 d = __fmul2_rn(l, make_float2(k.s, k.s));
                        f[e] = __fmul2_rn(make_float2(ex2(d.x), ex2(d.y)),
                                          __ffma2_rn(l, make_float2(f1, f1), make_float2(f0, f0)));
                    }
                    g[u] = pack2<T>(f);
                }
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (c + u * kThreads == tok_chunk || !(dense || ordinary)) {
                    float f[E];
                    unpack<T>(v[u], f);
                    elements(c + u * kThreads, f);
                    g[u] = pack<T>(f);
                }
            }
            store_chunks<T, kThreads>(r, o, c, we, g, amax, m2, a.status);
        });
        const int ec = r.edge(edge_of_thread(), c0, c1);
        if (ec >= 0) {
            float f[E];
            load_edge(r, ec, f, total, a.status);
            elements(ec, f);
            store_elements(r, o, ec, f, m2, a.status);
        }
    }
    if (part == a.blocks_per_row - 1)
        zero_columns(o, r.vocab, a.out.ld, tid, kThreads, a.status);
    block_amax(m2, a.out.amax, a.status);
}

// ------------------------------------------------------------ distillation
struct DistillArgs {
    const void *logits;
    int64_t rows, ld;
    int vocab, k, cluster, blocks_per_row;
    const int32_t *ids;
    const float *values;
    float inv_t, c;
    float *loss, *lse, *rest;      // written by the forward, read by the backward
    const float *dloss;
    OutArgs out;
    unsigned *status;
};

// The row's slots in shared memory.  Which chunks a slot names an element of is
// one bit each in `named` (exact up to 2^18 bf16 tokens, beyond that one bit
// for several chunks): a warp asks it for every chunk, and a filter with many
// false hits would send nearly every warp through the lists.  head[chunk %
// kHeads] then starts the list of slots.  Slots of equal ids each carry their
// summed q.  The sums over the slots are all that the loss needs of them:
//   loss = sum q log q - sum q (z - zref) / T + sum q ((max - zref) / T + ln S)
// for the row's maximum and S = sum e^((x - max) / T).
constexpr int kHeads = 256;
constexpr int kNamedWords = 1024;
struct alignas(16) Slots {
    uint32_t named[kNamedWords];
    int head[kHeads];
    int next[F8_MAX_TOP];
    int id[F8_MAX_TOP];      // -1: empty
    float q[F8_MAX_TOP];     // the slot's own q
    float qsum[F8_MAX_TOP];  // of all slots with this id
    int any;        // the row has a slot
    int used;       // some slot has q > 0
    int masked;     // such a slot names a masked token
    int skip;       // (backward) no gradient, whatever the logits
    float dloss;
    float lse, rest;  // (backward)
    float total;    // sum q (1 without the tail class); NaN if a value is NaN or +inf
    float qall;     // sum q as it came out
    float left;     // q_r
    float plogp;    // sum q log q
    float zref;     // the largest logit of a slot with q > 0
    float zmean;    // sum q (z - zref)
    float zmax;     // the largest logit of the slots' ids
    float inside;   // sum over these ids of 2^((z - zmax) c)
    float edge[2][8];  // (ring) the row's edge chunks
};

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// What one warp reads of a row's slots: slot lane + 32 i in register i.
struct SlotInput {
    int id[F8_MAX_TOP / 32];
    float t[F8_MAX_TOP / 32];
    float dloss, lse, rest;
};

template <bool TAIL, bool LOSS>
__device__ __forceinline__ SlotInput read_slots(const DistillArgs &a, int64_t row)
{
    SlotInput in;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < F8_MAX_TOP / 32; ++i) {
        const int j = lane + 32 * i;
        in.id[i] = -1;
        in.t[i] = F8_NEG_INF;
        if (32 * i < a.k && j < a.k) {
            in.id[i] = a.ids[row * a.k + j];
            in.t[i] = a.values[row * a.k + j];
        }
    }
    in.dloss = a.dloss != nullptr ? a.dloss[row] : 0.0f;
    in.lse = LOSS ? 0.0f : a.lse[row];
    in.rest = !LOSS && TAIL ? a.rest[row] : 0.0f;
    return in;
}

// One row's slots, by one warp.  Without LOSS only what the gradient needs, and
// no logit is read (in a backward pass in place another block may already have
// written it).
// `announce` is called as soon as s.any and s.skip are known.
template <typename T, bool TAIL, bool LOSS, typename F>
__device__ __forceinline__ void warp_slots(const DistillArgs &a, int64_t row, const SlotInput &in,
                                           Slots &s, F announce)
{
    constexpr int N = F8_MAX_TOP / 32;
    const int lane = threadIdx.x & 31, k = a.k;
    const Row<T> r(static_cast<const T *>(a.logits), row, a.ld, a.vocab);
    int id[N];
    float t[N], z[N];
    bool any = false, outside = false;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        id[i] = in.id[i];
        t[i] = in.t[i];
        z[i] = F8_NEG_INF;
        outside |= id[i] >= r.vocab;
        if (id[i] >= r.vocab || t[i] == F8_NEG_INF)
            id[i] = -1;
        if (id[i] < 0)
            t[i] = F8_NEG_INF;
        any |= id[i] >= 0;
    }
    if (outside)
        atomicOr(a.status, kStatusIndex);
    any = __any_sync(0xFFFFFFFFu, any);
    if (lane == 0) {
        s.any = any;
        s.skip = !LOSS && (in.dloss == 0.0f || fabsf(in.lse) >= kMaxLse);
        announce();
    }
    for (int i = lane; i < kNamedWords / 4; i += 32)
        reinterpret_cast<uint4 *>(s.named)[i] = make_uint4(0, 0, 0, 0);
    for (int i = lane; i < kHeads / 4; i += 32)
        reinterpret_cast<int4 *>(s.head)[i] = make_int4(-1, -1, -1, -1);
    if (any) {
        // slots 32 n and up do not exist; the loops stop there
        const int n = (k + 31) / 32;
        float tm = F8_NEG_INF;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (i >= n)
                break;
            if (LOSS && id[i] >= 0)
                z[i] = as_float(r.base[r.off + id[i]]);
            tm = fmaxf(tm, t[i]);
        }
        float q[N], logq[N], sum = 0.0f;
        if (!TAIL)
            tm = warp_max_of(tm);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            q[i] = logq[i] = 0.0f;
            if (i >= n)
                continue;
            logq[i] = TAIL ? t[i] : (t[i] - tm) * a.inv_t;
            q[i] = id[i] >= 0 ? expf(logq[i]) : 0.0f;
            sum += q[i];
        }
        sum = warp_sum(sum);
        if (!(fabsf(sum) < F8_POS_INF))  // a NaN or +inf among the values
            sum = F8_NAN;
        float qall = sum;
        if (!TAIL) {
            const float ls = logf(sum), inv = 1.0f / sum;
            qall = sum * inv;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                q[i] *= inv;
                logq[i] -= ls;
            }
        }
        // the table
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int j = lane + 32 * i;
            if (i >= n)
                break;
            if (j < k) {
                s.id[j] = id[i];
                s.q[j] = q[i];
            }
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (i >= n)
                break;
            if (id[i] >= 0) {
                const int ch = (id[i] + r.off) / Chunk<T>::E;
                s.next[lane + 32 * i] = atomicExch(&s.head[ch % kHeads], lane + 32 * i);
                atomicOr(&s.named[(ch >> 5) % kNamedWords], 1u << (ch & 31));
            }
        }
        __syncwarp();
        // each id's summed q; the first slot of an id stands for it
        bool first[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int j = lane + 32 * i;
            first[i] = id[i] >= 0;
            if (i >= n)
                continue;
            if (id[i] >= 0) {
                int same = 0;
                for (int p = s.head[((id[i] + r.off) / Chunk<T>::E) % kHeads]; p >= 0; p = s.next[p]) {
                    if (s.id[p] == id[i]) {
                        ++same;
                        first[i] = first[i] && p >= j;
                    }
                }
                float qs = q[i];
                if (same > 1) {  // in slot order
                    qs = 0.0f;
                    for (int p = 0; p < k; ++p)
                        qs += s.id[p] == id[i] ? s.q[p] : 0.0f;
                }
                s.qsum[j] = qs;
            }
        }
        if (LOSS) {
            float zref = F8_NEG_INF, zm = F8_NEG_INF;
            bool used = false, masked = false;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const bool u = q[i] > 0.0f || q[i] != q[i];
                used |= u;
                masked |= u && z[i] == F8_NEG_INF;
                zref = u ? fmaxf(zref, z[i]) : zref;
                zm = fmaxf(zm, z[i]);
            }
            zref = warp_max_of(zref);
            zm = warp_max_of(zm);
            used = __any_sync(0xFFFFFFFFu, used);
            masked = __any_sync(0xFFFFFFFFu, masked);
            float plogp = 0.0f, zmean = 0.0f, inside = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (i >= n)
                    break;
                if (q[i] > 0.0f || q[i] != q[i])
                    plogp = fmaf(q[i], logq[i], plogp);
                if (q[i] > 0.0f && z[i] != F8_NEG_INF)
                    zmean = fmaf(q[i], z[i] - zref, zmean);
                if (TAIL && first[i] && zm != F8_NEG_INF)
                    inside += ex2((z[i] - zm) * a.c);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                plogp += __shfl_xor_sync(0xFFFFFFFFu, plogp, o);
                zmean += __shfl_xor_sync(0xFFFFFFFFu, zmean, o);
                if (TAIL)
                    inside += __shfl_xor_sync(0xFFFFFFFFu, inside, o);
            }
            if (lane == 0) {
                s.used = used;
                s.masked = masked;
                s.plogp = plogp;
                s.zref = zref;
                s.zmean = zmean;
                s.zmax = zm;
                s.inside = inside;
            }
        }
        if (lane == 0) {
            s.total = TAIL || sum != sum ? sum : 1.0f;
            s.qall = qall;
            s.left = TAIL ? fmaxf(1.0f - sum, 0.0f) : 0.0f;
        }
    }
    if (lane == 0) {
        s.dloss = in.dloss;
        s.lse = in.lse;
        s.rest = in.rest;
    }
    __syncwarp();
}

// Which of chunks c + u * N a slot names an element of, as bits u; N a multiple
// of 32.
template <int N, int U>
__device__ __forceinline__ uint32_t named_bits(const Slots &s, int c)
{
    uint32_t bits = 0;
#pragma unroll
    for (int u = 0; u < U; ++u)
        bits |= ((s.named[static_cast<unsigned>((c >> 5) + u * (N / 32)) % kNamedWords] >> (c & 31)) & 1u)
                << u;
    return bits;
}

// -inf in the elements of chunk ch that a slot names.
template <typename T>
__device__ __forceinline__ void drop_slots(const Slots &s, const Row<T> &r, int ch,
                                           float (&f)[Chunk<T>::E])
{
    constexpr int E = Chunk<T>::E;
    for (int j = s.head[static_cast<unsigned>(ch) % kHeads]; j >= 0; j = s.next[j]) {
        const int d = s.id[j] + r.off - ch * E;
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (d == e)
                f[e] = F8_NEG_INF;
    }
}

// The same for U chunks c + u * N.
template <typename T, int N, int U>
__device__ __forceinline__ void drop_slots(const Slots &s, const Row<T> &r, int c, uint4 (&v)[U])
{
#pragma unroll 1
    for (uint32_t named = named_bits<N, U>(s, c); named != 0; named &= named - 1) {
        const int u = __ffs(named) - 1, ch = c + u * N;
        for (int j = s.head[static_cast<unsigned>(ch) % kHeads]; j >= 0; j = s.next[j]) {
            const int d = s.id[j] + r.off - ch * Chunk<T>::E;
            if (d >= 0 && d < Chunk<T>::E) {
#pragma unroll
                for (int i = 0; i < U; ++i)
                    if (i == u)
                        v[i] = set_element<T>(v[i], d, F8_NEG_INF);
            }
        }
    }
}

// What the gradient of a row needs: scale (mass p - q) at the slots' ids.
// Elsewhere it is scale (mass p_r - q_r) times the token's share of p_r, a
// softmax over the tokens outside the slots with a maximum of its own (shift),
// so it does not depend on how small p_r is: factor 2^((x a + shift) s).
// Without the tail class that is scale mass p.
struct RowGrad {
    Softmax p;
    float scale, mass, factor, shift;

    __device__ __forceinline__ Softmax outside() const { return Softmax{p.a, shift, p.s, 1.0f}; }
};

__device__ __forceinline__ float slot_gradient(const Slots &s, const RowGrad &g, int j, float x)
{
    return g.scale * fmaf(g.mass, ex2(g.p.exponent(x)) * g.p.norm, -s.qsum[j]);
}

// The gradient of one chunk's elements, and of U chunks c + u * N.
template <typename T>
__device__ __forceinline__ void row_gradient(const Slots &s, const Row<T> &r, int ch,
                                             const RowGrad &g, float (&x)[Chunk<T>::E])
{
    constexpr int E = Chunk<T>::E;
    float f[E];
#pragma unroll
    for (int e = 0; e < E; ++e)
        f[e] = g.factor * ex2(g.outside().exponent(x[e]));
    for (int j = s.head[static_cast<unsigned>(ch) % kHeads]; j >= 0; j = s.next[j]) {
        const int d = s.id[j] + r.off - ch * E;
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (d == e)
                f[e] = slot_gradient(s, g, j, x[e]);
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
        x[e] = f[e];
}
template <typename T, int N, int U>
__device__ __forceinline__ void row_gradient(const Slots &s, const Row<T> &r, int c,
                                             const RowGrad &g, const uint4 (&v)[U], uint4 (&out)[U])
{
    constexpr int E = Chunk<T>::E;
#pragma unroll
    for (int u = 0; u < U; ++u)
        out[u] = scaled_softmax<T>(v[u], g.outside(), g.factor);
#pragma unroll 1
    for (uint32_t named = named_bits<N, U>(s, c); named != 0; named &= named - 1) {
        const int u = __ffs(named) - 1, ch = c + u * N;
        for (int j = s.head[static_cast<unsigned>(ch) % kHeads]; j >= 0; j = s.next[j]) {
            const int d = s.id[j] + r.off - ch * E;
            if (d >= 0 && d < E) {
                uint4 w = v[0];
#pragma unroll
                for (int i = 1; i < U; ++i)
                    w = i == u ? v[i] : w;
                const float f = slot_gradient(s, g, j, get_element<T>(w, d));
#pragma unroll
                for (int i = 0; i < U; ++i)
                    if (i == u)
                        out[i] = set_element<T>(out[i], d, f);
            }
        }
    }
}

// The constants of the backward pass from the given lse and p_r.
template <bool TAIL>
__device__ __forceinline__ RowGrad row_grad(const DistillArgs &a, const Slots &s)
{
    const float scale = s.dloss * a.inv_t;
    RowGrad g{Softmax{a.inv_t, -s.lse, static_cast<float>(kLog2e), 1.0f}, scale, s.total,
              scale * s.total, -s.lse};
    if (TAIL && s.rest != 0.0f) {
        g.mass = s.total + s.left;
        g.factor = scale * (g.mass * fmaxf(s.rest, 0.0f) - s.left);
        g.shift = -(s.lse + (s.rest > 0.0f ? logf(s.rest) : s.rest));
    }
    return g;
}

// The row's loss and gradient constants from its slots and its sums (TAIL:
// over the tokens outside the slots' ids).
struct RowLoss {
    float loss, lse, rest;
    RowGrad grad;
    bool zero;  // no gradient
};

template <bool TAIL>
__device__ __forceinline__ RowLoss row_loss(const DistillArgs &a, const Slots &s, const Stats &t,
                                            bool loss)
{
    RowLoss o;
    float m = t.m, outside = t.s, sum = t.s;
    if (TAIL) {
        m = fmaxf(t.m, s.zmax);
        outside = t.s * ex2(fmaxf((t.m - m) * a.c, kFloor2));
        sum = outside + s.inside * ex2(fmaxf((s.zmax - m) * a.c, kFloor2));
    }
    const bool bad = sum != sum || m == F8_POS_INF;
    const bool none = !bad && sum == 0.0f;
    const float inv_s = none ? 0.0f : (bad ? F8_NAN : 1.0f / sum);
    const float ls = logf(sum);
    o.rest = TAIL ? outside * inv_s : 0.0f;
    if (TAIL && o.rest < kSmallRest && t.s > 0.0f)
        o.rest = fmaf(t.m - m, a.c, log2f(t.s / sum)) >= kNoRest
                     ? fmaf(t.m - m, a.inv_t, logf(t.s) - ls)
                     : 0.0f;
    const float scale = s.dloss * a.inv_t;
    const float shift = m == F8_NEG_INF ? 0.0f : -m;
    o.grad = RowGrad{Softmax{1.0f, shift, a.c, inv_s}, scale, s.total, scale * s.total * inv_s, shift};
    if (TAIL && o.rest != 0.0f) {
        o.grad.mass = s.total + s.left;
        o.grad.factor = scale * (o.grad.mass * fmaxf(o.rest, 0.0f) - s.left) / t.s;
        o.grad.shift = -t.m;
    }
    o.zero = s.dloss == 0.0f || none;
    if (!loss)
        return o;
    o.lse = bad ? F8_NAN : (none ? F8_NEG_INF : fmaf(m, a.inv_t, ls));
    o.loss = 0.0f;
    if (s.used)
        o.loss = s.masked || none ? F8_POS_INF
                                  : s.plogp - s.zmean * a.inv_t +
                                        s.qall * fmaf(m - s.zref, a.inv_t, ls);
    if (TAIL && o.rest != 0.0f && s.left > 0.0f)
        o.loss += s.left * (logf(s.left) - (o.rest > 0.0f ? logf(o.rest) : o.rest));
    if (bad || s.total != s.total || s.zmean != s.zmean)
        o.loss = F8_NAN;
    return o;
}

template <typename T, bool TAIL>
__global__ void __launch_bounds__(kThreads)
distill_fwd_kernel(const __grid_constant__ DistillArgs a)
{
    constexpr int E = Chunk<T>::E;
    __shared__ __align__(16) Slots slots;
    __shared__ Stats red[kWarps];
    __shared__ Stats parts[kMaxCluster];
    griddep_wait();
    griddep_launch_dependents();
    const int C = a.cluster;
    const int64_t row = blockIdx.x / C;
    const int rank = static_cast<int>(blockIdx.x % C);
    const int tid = threadIdx.x;
    const Row<T> r(static_cast<const T *>(a.logits), row, a.ld, a.vocab);
    const int64_t total = (a.rows - 1) * a.ld + a.vocab;
    if (C > 1)
        cluster_start();
    if (tid < 32)
        warp_slots<T, TAIL, true>(a, row, read_slots<TAIL, true>(a, row), slots, [] {});
    __syncthreads();
    if (!slots.any) {
        if (C > 1)
            cluster_started();
        if (rank == 0 && tid == 0) {
            a.loss[row] = 0.0f;
            a.lse[row] = 0.0f;
            if (TAIL)
                a.rest[row] = 0.0f;
        }
        return;
    }
    const int per = (r.nch + C - 1) / C;
    const int c0 = min(r.nch, rank * per), c1 = min(r.nch, c0 + per);
    Stats t = stats_empty();
    walk_chunks<T, kThreads, kUnroll>(r, max(c0, r.w0), min(c1, r.w1), total, a.status,
                                      [&](uint4(&v)[kUnroll], int c) {
                                          if (TAIL)
                                              drop_slots<T, kThreads>(slots, r, c, v);
                                          add_chunks<T, false>(t, v, a.c, 0.0f);
                                      });
    const int ec = r.edge(edge_of_thread(), c0, c1);
    if (ec >= 0) {
        float x[E];
        load_edge(r, ec, x, total, a.status);
        if (TAIL)
            drop_slots(slots, r, ec, x);
        add_values<false>(t, x, a.c);
    }
    t = block_join<false>(t, a.c, red);
    if (C > 1) {
        cluster_started();
        if (tid == 0)
            *peer(&parts[rank], 0) = t;
        cluster_join();
        if (rank != 0)
            return;
        t = cluster_stats<false>(parts, C, a.c);
    }
    if (tid == 0) {
        const RowLoss o = row_loss<TAIL>(a, slots, t, true);
        a.loss[row] = o.loss;
        a.lse[row] = o.lse;
        if (TAIL)
            a.rest[row] = o.rest;
        if (o.loss != o.loss)
            atomicOr(a.status, kStatusNonfinite);
    }
}

template <typename T, bool TAIL>
__global__ void __launch_bounds__(kThreads)
distill_bwd_kernel(const __grid_constant__ DistillArgs a)
{
    constexpr int E = Chunk<T>::E;
    __shared__ __align__(16) Slots slots;
    griddep_wait();
    griddep_launch_dependents();
    const int64_t row = blockIdx.x / a.blocks_per_row;
    const int part = static_cast<int>(blockIdx.x % a.blocks_per_row);
    const int tid = threadIdx.x;
    const Row<T> r(static_cast<const T *>(a.logits), row, a.ld, a.vocab);
    const int64_t total = (a.rows - 1) * a.ld + a.vocab;
    const OutRow<T> o(a.out, a.rows, row, r);
    if (tid < 32)
        warp_slots<T, TAIL, false>(a, row, read_slots<TAIL, false>(a, row), slots, [] {});
    __syncthreads();
    const RowGrad g = row_grad<TAIL>(a, slots);
    uint32_t m2 = 0;
    const bool amax = a.out.amax != nullptr;
    const int c0 = part * kBwdChunks, c1 = min(r.nch, c0 + kBwdChunks);
    const int wb = max(c0, r.w0), we = min(c1, r.w1);
    if (!slots.any || slots.skip) {
        zero_columns(o, max(static_cast<int64_t>(c0) * E - r.off, static_cast<int64_t>(0)),
                     min(static_cast<int64_t>(c1) * E - r.off, static_cast<int64_t>(r.vocab)), tid,
                     kThreads, a.status);
    } else {
        walk_chunks<T, kThreads, kUnroll>(r, wb, we, total, a.status, [&](uint4(&v)[kUnroll], int c) {
            uint4 f[kUnroll];
            row_gradient<T, kThreads>(slots, r, c, g, v, f);
            store_chunks<T, kThreads>(r, o, c, we, f, amax, m2, a.status);
        });
        const int ec = r.edge(edge_of_thread(), c0, c1);
        if (ec >= 0) {
            float f[E];
            load_edge(r, ec, f, total, a.status);
            row_gradient(slots, r, ec, g, f);
            store_elements(r, o, ec, f, m2, a.status);
        }
    }
    if (part == a.blocks_per_row - 1)
        zero_columns(o, r.vocab, a.out.ld, tid, kThreads, a.status);
    block_amax(m2, a.out.amax, a.status);
}

// Loss and gradient together, for short rows and for few: bf16 4096 x 8000 with
// 32 slots 52 us (2.5 TB/s; the slots' reading and two joins a row bound it), 32
// x 131072 14 us.  A block, or a cluster
// of C blocks, takes a row, each thread holding up to NV of its chunks in
// registers between the two passes, so a row that fits is read once; a longer
// one is walked in stretches and read again (from L2).
template <typename T, bool TAIL, int NV>
__global__ void __launch_bounds__(kThreads, NV > 4 ? 2 : 4)
distill_fused_kernel(const __grid_constant__ DistillArgs a)
{
    constexpr int E = Chunk<T>::E;
    __shared__ __align__(16) Slots slots;
    __shared__ Stats red[kWarps];
    __shared__ Stats parts[kMaxCluster];
    griddep_wait();
    griddep_launch_dependents();
    const int C = a.cluster;
    const int64_t row = blockIdx.x / C;
    const int rank = static_cast<int>(blockIdx.x % C);
    const int tid = threadIdx.x;
    const Row<T> r(static_cast<const T *>(a.logits), row, a.ld, a.vocab);
    const int64_t total = (a.rows - 1) * a.ld + a.vocab;
    const OutRow<T> o(a.out, a.rows, row, r);
    if (C > 1)
        cluster_start();
    if (tid < 32)
        warp_slots<T, TAIL, true>(a, row, read_slots<TAIL, true>(a, row), slots, [] {});
    __syncthreads();
    const int per = (r.nch + C - 1) / C;
    const int c0 = min(r.nch, rank * per), c1 = min(r.nch, c0 + per);
    const int wb = max(c0, r.w0), we = min(c1, r.w1);  // this block's whole chunks
    const int ec = r.edge(edge_of_thread(), c0, c1);
    const bool amax = a.out.amax != nullptr;
    uint32_t m2 = 0;
    bool zero = true;
    if (slots.any) {
        uint4 v[NV / kUnroll][kUnroll];
        const bool fits = we - wb <= NV * kThreads;
        float edge[E];
        Stats t = stats_empty();
        if (ec >= 0) {
            load_edge(r, ec, edge, total, a.status);
            float x[E];
#pragma unroll
            for (int e = 0; e < E; ++e)
                x[e] = edge[e];
            if (TAIL)
                drop_slots(slots, r, ec, x);
            add_values<false>(t, x, a.c);
        }
        if (fits) {
#pragma unroll
            for (int h = 0; h < NV / kUnroll; ++h)
#pragma unroll
                for (int u = 0; u < kUnroll; ++u)
                    v[h][u] = load_chunk(r, wb + (h * kUnroll + u) * kThreads + tid, we, total,
                                         a.status);
#pragma unroll
            for (int h = 0; h < NV / kUnroll; ++h) {
                const int c = wb + h * kUnroll * kThreads + tid;
                if (c < we) {
                    uint4 w[kUnroll];
#pragma unroll
                    for (int u = 0; u < kUnroll; ++u)
                        w[u] = v[h][u];
                    if (TAIL)
                        drop_slots<T, kThreads>(slots, r, c, w);
                    add_chunks<T, false>(t, w, a.c, 0.0f);
                }
            }
        } else {
            walk_chunks<T, kThreads, kUnroll>(r, wb, we, total, a.status,
                                              [&](uint4(&w)[kUnroll], int c) {
                                                  if (TAIL)
                                                      drop_slots<T, kThreads>(slots, r, c, w);
                                                  add_chunks<T, false>(t, w, a.c, 0.0f);
                                              });
        }
        t = block_join<false>(t, a.c, red);
        if (C > 1) {
            cluster_started();
            if (tid < C)
                *peer(&parts[rank], tid) = t;
            cluster_join();
            t = cluster_stats<false>(parts, C, a.c);
        }
        const RowLoss l = row_loss<TAIL>(a, slots, t, rank == 0 && tid == 0);
        zero = l.zero;
        if (rank == 0 && tid == 0) {
            a.loss[row] = l.loss;
            if (l.loss != l.loss)
                atomicOr(a.status, kStatusNonfinite);
        }
        if (!zero) {
            auto gradient = [&](const uint4(&w)[kUnroll], int c) {
                uint4 f[kUnroll];
                row_gradient<T, kThreads>(slots, r, c, l.grad, w, f);
                store_chunks<T, kThreads>(r, o, c, we, f, amax, m2, a.status);
            };
            if (fits) {
#pragma unroll
                for (int h = 0; h < NV / kUnroll; ++h)
                    if (wb + h * kUnroll * kThreads + tid < we)
                        gradient(v[h], wb + h * kUnroll * kThreads + tid);
            } else {
                walk_chunks<T, kThreads, kUnroll>(r, wb, we, total, a.status, gradient);
            }
            if (ec >= 0) {
                row_gradient(slots, r, ec, l.grad, edge);
                store_elements(r, o, ec, edge, m2, a.status);
            }
        }
    } else {
        if (C > 1)
            cluster_started();
        if (rank == 0 && tid == 0)
            a.loss[row] = 0.0f;
    }
    if (zero)
        zero_columns(o, max(static_cast<int64_t>(c0) * E - r.off, static_cast<int64_t>(0)),
                     min(static_cast<int64_t>(c1) * E - r.off, static_cast<int64_t>(r.vocab)), tid,
                     kThreads, a.status);
    if (rank == C - 1)
        zero_columns(o, r.vocab, a.out.ld, tid, kThreads, a.status);
    block_amax(m2, a.out.amax, a.status);
}

// Loss and gradient together, for many long rows.  A row of the logits is
// needed twice, for its sums and for its gradient, and the blocks of all SMs
// together hold more than L2 does, so a block keeps what it can: one persistent
// block per SM takes whole rows through a ring of 32 KB pieces in shared
// memory that bulk copies fill.
//   warps 16..18 each read every third row's slots into a buffer of their own
//                and sum them up, ahead of the others;
//   warp 19      issues the copies: a row's pieces 0 .. n-1, then again those
//                that the ring could not keep, then the next row's;
//   warps 0..15  first pass: running sums over the pieces, releasing all but
//                the last `keep`; the block's join (one barrier); second pass:
//                the gradient of the kept pieces, then of those copied again
//                (from L2, which they have just passed), released one by one.
// The pieces are released in the order of their copies, so the ring is a queue
// and the next row's copies run during the second pass.
// BWD is the backward pass alone, with lse (and p_r) given: the second pass
// only, over every piece once.
// bf16 4096 x 131072 with 64 slots: 356 us, 6.0 TB/s of one read and one write
// (a block per row read twice from L2 took 544); backward alone 1024 x 131072
// 87 us, 6.2 TB/s.  777 rows are six rounds of 152 blocks where 5.1 would do:
// 777 x 50003 50 us, 3.1 TB/s.
constexpr int kRingWarps = 16;
constexpr int kRingConsumers = kRingWarps * 32;
constexpr int kSlotBuffers = 3;
constexpr int kRingThreads = kRingConsumers + 32 * kSlotBuffers + 32;
constexpr int kPieceChunks = kUnroll * kRingConsumers;
constexpr int kPieceBytes = kPieceChunks * 16;
constexpr int kPieces = 6;
constexpr int kKeep = 4;  // the other two are under way

constexpr size_t kRingSmem = static_cast<size_t>(kPieces) * kPieceBytes +
                             kSlotBuffers * sizeof(Slots);

// Piece of position `seq` in the queue: its slot, and the parity of its phase.
__device__ __forceinline__ int ring_slot(uint32_t seq) { return f8::ring_slot(seq, kPieces); }
__device__ __forceinline__ uint32_t ring_parity(uint32_t seq)
{
    return f8::ring_parity(seq, kPieces);
}

template <typename T, bool TAIL, bool BWD>
__global__ void __launch_bounds__(kRingThreads, 1)
distill_ring_kernel(const __grid_constant__ DistillArgs a, uint64_t limit_ns)
{
    constexpr int E = Chunk<T>::E;
    extern __shared__ __align__(128) uint8_t pieces[];
    __shared__ __align__(8) uint64_t full[kPieces];
    __shared__ __align__(8) uint64_t empty[kPieces];
    __shared__ __align__(8) uint64_t sfull[kSlotBuffers];
    __shared__ __align__(8) uint64_t sempty[kSlotBuffers];
    __shared__ __align__(8) uint64_t known[kSlotBuffers];
    __shared__ Stats parts[2][kRingWarps];
    __shared__ int abort_word;
    volatile int *abort_flag = &abort_word;
    Slots *slots = reinterpret_cast<Slots *>(pieces + static_cast<size_t>(kPieces) * kPieceBytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < kPieces; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kRingWarps);
        }
        for (int i = 0; i < kSlotBuffers; ++i) {
            mbar_init(&sfull[i], 1);
            mbar_init(&known[i], 1);
            mbar_init(&sempty[i], kRingWarps + 1);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    griddep_wait();
    griddep_launch_dependents();
    __syncthreads();
    const int64_t total = (a.rows - 1) * a.ld + a.vocab;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (mbar_wait(bar, parity, abort_flag, limit_ns))
            return true;
        *abort_flag = 1;
        atomicOr(a.status, kStatusTimeout);
        return false;
    };
    uint32_t m2 = 0;
    const bool amax = a.out.amax != nullptr;

    if (warp >= kRingWarps && warp < kRingWarps + kSlotBuffers) {
        // ---------------------------------------------------- the rows' slots
        const int b = warp - kRingWarps;
        const int64_t step = static_cast<int64_t>(gridDim.x) * kSlotBuffers;
        int turn = 0;
        for (int64_t row = blockIdx.x + static_cast<int64_t>(b) * gridDim.x; row < a.rows;
             row += step, ++turn) {
            if (row + step < a.rows && lane * 32 < a.k * 4) {  // the next one's, towards L2
                const int64_t at = (row + step) * a.k + lane * 8;
                prefetch_l2(a.ids + at);
                prefetch_l2(a.values + at);
            }
            const bool ok = wait(&sempty[b], (turn & 1) ^ 1u);
            if (!__all_sync(0xFFFFFFFFu, ok))
                break;
            warp_slots<T, TAIL, !BWD>(a, row, read_slots<TAIL, !BWD>(a, row), slots[b],
                                      [&] { mbar_arrive(&known[b]); });
            // the row's edges too, so that no other warp waits for global memory
            const Row<T> r(static_cast<const T *>(a.logits), row, a.ld, a.vocab);
            const int ec = slots[b].any ? r.edge(lane, 0, r.nch) : -1;
            if (ec >= 0) {
                float f[E];
                load_edge(r, ec, f, total, a.status);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    slots[b].edge[lane][e] = f[e];
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sfull[b]);
        }
    } else if (warp == kRingWarps + kSlotBuffers) {
        // ---------------------------------------------------- copies
        if (lane == 0) {
            uint32_t seq = 0;
            int i = 0;
            bool stop = false;
            for (int64_t row = blockIdx.x; row < a.rows && !stop; row += gridDim.x, ++i) {
                const int b = i % kSlotBuffers;
                if (!wait(&known[b], (i / kSlotBuffers) & 1)) {
                    stop = true;
                    break;
                }
                const bool any = slots[b].any != 0 && !(BWD && slots[b].skip);
                mbar_arrive(&sempty[b]);
                if (!any)
                    continue;
                const Row<T> r(static_cast<const T *>(a.logits), row, a.ld, a.vocab);
                const int n = r.w1 - r.w0;
                const int np = (n + kPieceChunks - 1) / kPieceChunks;
                const int again = BWD ? 0 : np - min(np, kKeep);
                for (int j = 0; j < np + again; ++j, ++seq) {
                    const int piece = j < np ? j : j - np;
                    const int slot = ring_slot(seq);
                    if (!wait(&empty[slot], ring_parity(seq) ^ 1u)) {
                        stop = true;
                        break;
                    }
                    const int c0 = piece * kPieceChunks;
                    const uint32_t bytes = 16u * static_cast<uint32_t>(min(kPieceChunks, n - c0));
                    mbar_arrive_expect_tx(&full[slot], bytes);
                    bulk_load(pieces + slot * kPieceBytes,
                              r.base + static_cast<int64_t>(r.w0 + c0) * E, bytes, &full[slot]);
                }
            }
            // the copies land before the block leaves, also where another warp gives up
            // on one after this
            ring_drain(seq, kPieces, [&](int slot, uint32_t parity) {
                mbar_wait(&full[slot], parity, nullptr, kDrainLimitNs);
            });
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------- sums and gradient
        uint32_t seq = 0;
        int i = 0;
        bool alive = true;
        for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, ++i) {
            const int b = i % kSlotBuffers;
            alive = alive && __all_sync(0xFFFFFFFFu, wait(&sfull[b], (i / kSlotBuffers) & 1));
            const Slots &s = slots[b];
            const bool any = alive && s.any != 0 && !(BWD && s.skip);
            const Row<T> r(static_cast<const T *>(a.logits), row, a.ld, a.vocab);
            const int n = r.w1 - r.w0;
            const int np = any ? (n + kPieceChunks - 1) / kPieceChunks : 0;
            const int keep = BWD ? 0 : min(np, kKeep), again = BWD ? 0 : np - keep;
            auto arrived = [&](uint32_t q) {
                alive = alive && __all_sync(0xFFFFFFFFu, wait(&full[ring_slot(q)], ring_parity(q)));
            };
            auto release = [&](uint32_t q) {
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&empty[ring_slot(q)]);
            };
            // this thread's chunk u of a piece; a piece's chunks, and whether it has them all
            auto chunk = [&](uint32_t q, int u) {
                return reinterpret_cast<const uint4 *>(pieces + ring_slot(q) * kPieceBytes)
                    [u * kRingConsumers + tid];
            };
            auto chunks_of = [&](int piece) { return min(n - piece * kPieceChunks, kPieceChunks); };
            const int ec = any ? r.edge(edge_of_thread(), 0, r.nch) : -1;
            Stats t = stats_empty();
            if (!BWD) {
                for (int j = 0; j < np; ++j) {
                    arrived(seq + j);
                    const int c = r.w0 + j * kPieceChunks + tid, have = chunks_of(j);
                    if (have == kPieceChunks) {
                        uint4 v[kUnroll];
#pragma unroll
                        for (int u = 0; u < kUnroll; ++u)
                            v[u] = chunk(seq + j, u);
                        if (j < again)
                            release(seq + j);
                        if (TAIL)
                            drop_slots<T, kRingConsumers>(s, r, c, v);
                        add_chunks<T, false>(t, v, a.c, 0.0f);
                    } else {  // the row's last piece, which is kept: a warp's part of it
#pragma unroll 1
                        for (int u = 0; u * kRingConsumers + warp * 32 < have; ++u) {
                            uint4 v[1] = {neg_inf_chunk(T())};
                            if (u * kRingConsumers + tid < have)
                                v[0] = chunk(seq + j, u);
                            if (TAIL)
                                drop_slots<T, kRingConsumers>(s, r, c + u * kRingConsumers, v);
                            add_chunks<T, false>(t, v, a.c, 0.0f);
                        }
                    }
                }
                if (ec >= 0) {
                    float x[E];
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        x[e] = s.edge[warp][e];
                    if (TAIL)
                        drop_slots(s, r, ec, x);
                    add_values<false>(t, x, a.c);
                }
                // the block's sums: warps' in shared memory, two sets in turn
                t = warp_stats<false, 32>(t, a.c);
                if (lane == 0)
                    parts[i & 1][warp] = t;
                asm volatile("bar.sync 1, %0;" ::"n"(kRingConsumers) : "memory");
                t = warp_stats<false, kRingWarps>(parts[i & 1][lane & (kRingWarps - 1)], a.c);
            }

            const OutRow<T> o(a.out, a.rows, row, r);
            bool zero = true;
            if (any) {
                RowGrad g;
                if (BWD) {
                    g = row_grad<TAIL>(a, s);
                    zero = false;
                } else {
                    const RowLoss l = row_loss<TAIL>(a, s, t, tid == 0);
                    g = l.grad;
                    zero = l.zero;
                    if (tid == 0) {
                        a.loss[row] = l.loss;
                        if (l.loss != l.loss)
                            atomicOr(a.status, kStatusNonfinite);
                    }
                }
                // the kept pieces, then the first ones again
                for (int j = 0; j < np; ++j) {
                    const int piece = j < keep ? again + j : j - keep;
                    const uint32_t q = seq + again + j;
                    if (j >= keep)
                        arrived(q);
                    const int c = r.w0 + piece * kPieceChunks + tid, have = chunks_of(piece);
                    if (zero) {
                        release(q);
                    } else if (have == kPieceChunks) {
                        uint4 v[kUnroll], f[kUnroll];
#pragma unroll
                        for (int u = 0; u < kUnroll; ++u)
                            v[u] = chunk(q, u);
                        release(q);
                        row_gradient<T, kRingConsumers>(s, r, c, g, v, f);
                        store_chunks<T, kRingConsumers>(r, o, c, r.w1, f, amax, m2, a.status);
                    } else {
#pragma unroll 1
                        for (int u = 0; u * kRingConsumers + warp * 32 < have; ++u) {
                            uint4 v[1] = {neg_inf_chunk(T())}, f[1];
                            if (u * kRingConsumers + tid < have)
                                v[0] = chunk(q, u);
                            row_gradient<T, kRingConsumers>(s, r, c + u * kRingConsumers, g, v, f);
                            store_chunks<T, kRingConsumers>(r, o, c + u * kRingConsumers, r.w1, f,
                                                            amax, m2, a.status);
                        }
                        release(q);
                    }
                }
                if (ec >= 0 && !zero) {
                    float x[E];
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        x[e] = s.edge[warp][e];
                    row_gradient(s, r, ec, g, x);
                    store_elements(r, o, ec, x, m2, a.status);
                }
                seq += np + again;
            } else if (!BWD && alive && tid == 0) {
                a.loss[row] = 0.0f;
            }
            if (alive) {
                if (zero)
                    zero_columns(o, 0, r.vocab, tid, kRingConsumers, a.status);
                zero_columns(o, r.vocab, a.out.ld, tid, kRingConsumers, a.status);
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sempty[b]);
        }
    }
    block_amax(m2, a.out.amax, a.status);
}

// ------------------------------------------------------------ launches
// Blocks per row: one where the rows alone keep every SM busy, up to eight
// where they do not, none with less than a group of chunks for each warp.  Two
// blocks an SM are enough: splitting on to four costs more in the joins than it
// gains (fp32 log probabilities of 200 x 32000 with the top 8 14.1 us against
// 17.0, bf16 500 x 50003 with the top 64 30.5 against 36.9; without the top
// alternatives it is 13.8 against 12.7 us at 152 x 131072).
int cluster_for(int64_t rows, int64_t chunks, const DeviceInfo &dev)
{
    int c = 1;
    while (c < kMaxCluster && rows * c < 2 * dev.sm_count && chunks / (2 * c) >= kWarps * 32)
        c *= 2;
    return c;
}

// Lets Kernel be launched with up to `bytes` of dynamic shared memory: once per
// device, at the most that any call needs, since the limit belongs to the kernel
// and calls from other threads launch under it too.
template <auto Kernel>
cudaError_t allow_smem(size_t bytes, const DeviceInfo &dev)
{
    static std::once_flag once[64];
    static cudaError_t err[64];
    const int d = dev.ordinal & 63;
    std::call_once(once[d], [&] {
        err[d] = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      static_cast<int>(bytes));
    });
    return err[d];
}

// Groups of 32 chunks that a row of `vocab` tokens touches at any offset.
template <typename T>
int most_groups(int64_t vocab)
{
    constexpr int E = Chunk<T>::E;
    return static_cast<int>(((vocab + E - 1 + E) / E + 31) / 32);
}

template <typename T>
cudaError_t logprobs(LogprobArgs a, const DeviceInfo &dev, cudaStream_t st)
{
    constexpr int E = Chunk<T>::E;
    const int64_t chunks = (static_cast<int64_t>(a.vocab) + E - 1 + E) / E;
    a.cluster = cluster_for(a.rows, chunks, dev);
    const dim3 grid(static_cast<unsigned>(a.rows * a.cluster));
    if (a.top_k > 0) {
        const int ngroups = most_groups<T>(a.vocab);
        const size_t smem =
            4u * top_layout((ngroups + a.cluster - 1) / a.cluster, a.top_k, a.cluster).words;
        // one block a row of the largest vocabulary: 116 KB for bf16, 180 KB for
        // fp32; a cluster's merge arrays take less than the groups that it shares
        const cudaError_t e = allow_smem<logprobs_kernel<T, true>>(
            4u * top_layout(most_groups<T>(F8_MAX_VOCAB), F8_MAX_TOP, 1).words, dev);
        if (e != cudaSuccess)
            return e;
        return launch_pdl_cluster(logprobs_kernel<T, true>, grid, dim3(kThreads), smem, st,
                                  static_cast<unsigned>(a.cluster), a);
    }
    return launch_pdl_cluster(logprobs_kernel<T, false>, grid, dim3(kThreads), 0, st,
                              static_cast<unsigned>(a.cluster), a);
}

template <typename T>
int bwd_blocks(int64_t vocab)
{
    const int64_t chunks = (vocab + 2 * Chunk<T>::E - 2) / Chunk<T>::E;
    return static_cast<int>((chunks + kBwdChunks - 1) / kBwdChunks);
}

template <typename T>
cudaError_t logprobs_bwd(LogprobBwdArgs a, const DeviceInfo &, cudaStream_t st)
{
    a.blocks_per_row = bwd_blocks<T>(a.vocab);
    return launch_pdl(logprobs_bwd_kernel<T>, dim3(static_cast<unsigned>(a.rows * a.blocks_per_row)),
                      dim3(kThreads), 0, st, a);
}

template <typename T, bool TAIL>
cudaError_t distill_fwd(DistillArgs a, const DeviceInfo &dev, cudaStream_t st)
{
    const int64_t chunks = (static_cast<int64_t>(a.vocab) + 2 * Chunk<T>::E - 2) / Chunk<T>::E;
    a.cluster = cluster_for(a.rows, chunks, dev);
    return launch_pdl_cluster(distill_fwd_kernel<T, TAIL>,
                              dim3(static_cast<unsigned>(a.rows * a.cluster)), dim3(kThreads), 0, st,
                              static_cast<unsigned>(a.cluster), a);
}

// The ring where a row is longer than a block holds in 4 registers a thread and
// there is at least a row for every second SM.  Loss and gradient, bf16, ring
// against blocks and clusters: 4096 x 131072 356 us against 544, 1024 x 131072
// 98 against 158, 4096 x 16000 100 against 112, 152 x 131072 20 against 24, 76 x
// 131072 17 against 25; but 32 x 131072 17 against 14, and 4096 x 8000 83 against
// 52.  The backward pass alone is near even: with the tail class 777 x 50003 31
// against 35 and 2048 x 65536 90 against 95, without it 300 x 131072 28 against
// 29, but 1024 x 131072 88 against 84 and 4096 x 131072 338 against 327: there the
// ring costs 3 to 5 %, and one rule for the calls is kept.
constexpr int kShortChunks = 4 * kThreads;

template <typename T>
int64_t most_chunks(const DistillArgs &a)
{
    return (static_cast<int64_t>(a.vocab) + 2 * Chunk<T>::E - 2) / Chunk<T>::E;
}
template <typename T>
bool ring_takes(const DistillArgs &a, const DeviceInfo &dev)
{
    return most_chunks<T>(a) > kShortChunks && 2 * a.rows >= dev.sm_count;
}

template <typename T, bool TAIL, bool BWD>
cudaError_t distill_ring(const DistillArgs &a, const DeviceInfo &dev, cudaStream_t st)
{
    const cudaError_t e = allow_smem<distill_ring_kernel<T, TAIL, BWD>>(kRingSmem, dev);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(distill_ring_kernel<T, TAIL, BWD>,
                      dim3(static_cast<unsigned>(std::min<int64_t>(a.rows, dev.sm_count))),
                      dim3(kRingThreads), kRingSmem, st, a, wait_limit_ns());
}

template <typename T, bool TAIL>
cudaError_t distill_bwd(DistillArgs a, const DeviceInfo &dev, cudaStream_t st)
{
    if (ring_takes<T>(a, dev))
        return distill_ring<T, TAIL, true>(a, dev, st);
    a.blocks_per_row = bwd_blocks<T>(a.vocab);
    return launch_pdl(distill_bwd_kernel<T, TAIL>,
                      dim3(static_cast<unsigned>(a.rows * a.blocks_per_row)), dim3(kThreads), 0, st,
                      a);
}

template <typename T, bool TAIL>
cudaError_t distill_fused(DistillArgs a, const DeviceInfo &dev, cudaStream_t st)
{
    if (ring_takes<T>(a, dev))
        return distill_ring<T, TAIL, false>(a, dev, st);
    a.cluster = cluster_for(a.rows, most_chunks<T>(a), dev);
    const dim3 grid(static_cast<unsigned>(a.rows * a.cluster));
    const unsigned c = static_cast<unsigned>(a.cluster);
    if (most_chunks<T>(a) <= kShortChunks)
        return launch_pdl_cluster(distill_fused_kernel<T, TAIL, 4>, grid, dim3(kThreads), 0, st, c, a);
    return launch_pdl_cluster(distill_fused_kernel<T, TAIL, 8>, grid, dim3(kThreads), 0, st, c, a);
}

// log2(e) / T.
float exponent_scale(float temperature)
{
    return static_cast<float>(kLog2e / static_cast<double>(temperature));
}

// What every call of this file asks of its logits.
f8_status check_logits(const void *logits, f8_dtype type, int64_t rows, int64_t vocab, int64_t ld,
                       float temperature)
{
    if ((type != F8_BF16 && type != F8_F32) || rows < 0 || vocab < 0 || ld < vocab)
        return F8_ERR_INVALID;
    // the kernels work with log2(e) / T, which leaves fp32's range before 1 / T does
    if (!(temperature > 0.0f) || !std::isfinite(temperature) || !std::isfinite(exponent_scale(temperature)))
        return F8_ERR_INVALID;
    if (rows > 0 && (vocab == 0 || logits == nullptr))
        return F8_ERR_INVALID;
    // blocks are numbered in 32 bits: at most kMaxCluster, or the backward's share, per row
    if (vocab > F8_MAX_VOCAB || ld > INT32_MAX || rows > INT32_MAX / 1024)
        return F8_ERR_SHAPE;
    if (!aligned(logits, 16))
        return F8_ERR_ALIGN;
    return F8_OK;
}

f8_status check_out(const void *dlogits, f8_dtype type, int64_t rows, int64_t vocab, int64_t ld,
                    const void *logits, int64_t ldd, const float *amax_out)
{
    if (ldd < vocab || (rows > 0 && dlogits == nullptr))
        return F8_ERR_INVALID;
    // in place the rows have to lie alike; a single one has no stride
    if (dlogits != nullptr && dlogits == logits && ldd != ld && rows > 1)
        return F8_ERR_INVALID;
    if (amax_out != nullptr && type != F8_BF16)
        return F8_ERR_INVALID;
    if (ldd > INT32_MAX)
        return F8_ERR_SHAPE;
    if (!aligned(dlogits, 16) || !aligned(amax_out, 4))
        return F8_ERR_ALIGN;
    return F8_OK;
}

f8_status check_slots(const int32_t *ids, const float *values, int k, int tail, int64_t rows)
{
    if (k < 1 || (tail != 0 && tail != 1) || (rows > 0 && (ids == nullptr || values == nullptr)))
        return F8_ERR_INVALID;
    if (k > F8_MAX_TOP)
        return F8_ERR_SHAPE;
    if (!aligned(ids, 4) || !aligned(values, 4))
        return F8_ERR_ALIGN;
    return F8_OK;
}

DistillArgs distill_args(const void *logits, int64_t rows, int64_t vocab, int64_t ld,
                         const int32_t *ids, const float *values, int k, float temperature,
                         float *loss, float *lse, float *rest, const float *dloss, void *dlogits,
                         int64_t ldd, float *amax_out, const DeviceInfo &dev)
{
    DistillArgs a = {};
    a.logits = logits;
    a.rows = rows;
    a.ld = ld;
    a.vocab = static_cast<int>(vocab);
    a.k = k;
    a.ids = ids;
    a.values = values;
    a.inv_t = 1.0f / temperature;
    a.c = exponent_scale(temperature);
    a.loss = loss;
    a.lse = lse;
    a.rest = rest;
    a.dloss = dloss;
    a.out = OutArgs{dlogits, ldd, reinterpret_cast<unsigned *>(amax_out)};
    a.status = dev.status;
    return a;
}

} // namespace
} // namespace f8

using namespace f8;

#define F8_BY_TYPE(fn, type, tail, ...)                                                            \
    ((type) == F8_BF16 ? ((tail) ? fn<__nv_bfloat16, true>(__VA_ARGS__)                            \
                                 : fn<__nv_bfloat16, false>(__VA_ARGS__))                          \
                       : ((tail) ? fn<float, true>(__VA_ARGS__) : fn<float, false>(__VA_ARGS__)))

extern "C" {

f8_status f8_token_logprobs(const void *logits, f8_dtype type, int64_t rows, int64_t vocab,
                            int64_t ld, const int64_t *tokens, float temperature, int top_k,
                            float *logp, float *entropy, float *lse, int32_t *top_ids,
                            float *top_logp, void *stream)
{
    F8_TRY(check_logits(logits, type, rows, vocab, ld, temperature));
    if (top_k < 0 || (top_k > 0 && rows > 0 && (top_ids == nullptr || top_logp == nullptr)) ||
        (tokens == nullptr && logp != nullptr))
        return F8_ERR_INVALID;
    if (top_k > F8_MAX_TOP || (rows > 0 && top_k > vocab))
        return F8_ERR_SHAPE;
    if (!aligned(tokens, 8) || !aligned(logp, 4) || !aligned(entropy, 4) || !aligned(lse, 4) ||
        !aligned(top_ids, 4) || !aligned(top_logp, 4))
        return F8_ERR_ALIGN;
    const DeviceInfo *dev;
    F8_TRY(get_device(&dev));
    if (rows == 0)
        return F8_OK;
    LogprobArgs a = {};
    a.logits = logits;
    a.rows = rows;
    a.ld = ld;
    a.vocab = static_cast<int>(vocab);
    a.top_k = top_k;
    a.tokens = tokens;
    a.inv_t = 1.0f / temperature;
    a.c = exponent_scale(temperature);
    a.inv_c = static_cast<float>(static_cast<double>(temperature) / kLog2e);
    a.logp = logp;
    a.entropy = entropy;
    a.lse = lse;
    a.top_ids = top_ids;
    a.top_logp = top_logp;
    a.status = dev->status;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return from_cuda(type == F8_BF16 ? logprobs<__nv_bfloat16>(a, *dev, st)
                                     : logprobs<float>(a, *dev, st));
}

f8_status f8_token_logprobs_bwd(const void *logits, f8_dtype type, int64_t rows, int64_t vocab,
                                int64_t ld, const int64_t *tokens, const float *lse,
                                const float *entropy, const float *dlogp, const float *dentropy,
                                float temperature, void *dlogits, int64_t ldd, float *amax_out,
                                void *stream)
{
    F8_TRY(check_logits(logits, type, rows, vocab, ld, temperature));
    F8_TRY(check_out(dlogits, type, rows, vocab, ld, logits, ldd, amax_out));
    if (rows > 0 && (lse == nullptr || (dentropy != nullptr && entropy == nullptr) ||
                     (dlogp != nullptr && tokens == nullptr)))
        return F8_ERR_INVALID;
    if (!aligned(tokens, 8) || !aligned(lse, 4) || !aligned(entropy, 4) || !aligned(dlogp, 4) ||
        !aligned(dentropy, 4))
        return F8_ERR_ALIGN;
    const DeviceInfo *dev;
    F8_TRY(get_device(&dev));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (amax_out != nullptr)
        F8_TRY_CUDA(cudaMemsetAsync(amax_out, 0, sizeof(float), st));
    if (rows == 0)
        return F8_OK;
    LogprobBwdArgs a = {};
    a.logits = logits;
    a.rows = rows;
    a.ld = ld;
    a.vocab = static_cast<int>(vocab);
    a.tokens = tokens;
    a.lse = lse;
    a.entropy = entropy;
    a.dlogp = dlogp;
    a.dentropy = dentropy;
    a.inv_t = 1.0f / temperature;
    a.t = temperature;
    a.out = OutArgs{dlogits, ldd, reinterpret_cast<unsigned *>(amax_out)};
    a.status = dev->status;
    return from_cuda(type == F8_BF16 ? logprobs_bwd<__nv_bfloat16>(a, *dev, st)
                                     : logprobs_bwd<float>(a, *dev, st));
}

f8_status f8_distill_fwd(const void *logits, f8_dtype type, int64_t rows, int64_t vocab, int64_t ld,
                         const int32_t *ids, const float *values, int k, float temperature,
                         int tail, float *loss, float *lse, float *rest, void *stream)
{
    F8_TRY(check_logits(logits, type, rows, vocab, ld, temperature));
    F8_TRY(check_slots(ids, values, k, tail, rows));
    if (rows > 0 && (loss == nullptr || lse == nullptr || (tail && rest == nullptr)))
        return F8_ERR_INVALID;
    if (!aligned(loss, 4) || !aligned(lse, 4) || !aligned(rest, 4))
        return F8_ERR_ALIGN;
    const DeviceInfo *dev;
    F8_TRY(get_device(&dev));
    if (rows == 0)
        return F8_OK;
    const DistillArgs a = distill_args(logits, rows, vocab, ld, ids, values, k, temperature, loss,
                                       lse, rest, nullptr, nullptr, 0, nullptr, *dev);
    return from_cuda(F8_BY_TYPE(f8::distill_fwd, type, tail, a, *dev,
                                static_cast<cudaStream_t>(stream)));
}

f8_status f8_distill_bwd(const void *logits, f8_dtype type, int64_t rows, int64_t vocab, int64_t ld,
                         const int32_t *ids, const float *values, int k, float temperature,
                         int tail, const float *lse, const float *rest, const float *dloss,
                         void *dlogits, int64_t ldd, float *amax_out, void *stream)
{
    F8_TRY(check_logits(logits, type, rows, vocab, ld, temperature));
    F8_TRY(check_slots(ids, values, k, tail, rows));
    F8_TRY(check_out(dlogits, type, rows, vocab, ld, logits, ldd, amax_out));
    if (rows > 0 && (lse == nullptr || dloss == nullptr || (tail && rest == nullptr)))
        return F8_ERR_INVALID;
    if (!aligned(lse, 4) || !aligned(rest, 4) || !aligned(dloss, 4))
        return F8_ERR_ALIGN;
    const DeviceInfo *dev;
    F8_TRY(get_device(&dev));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (amax_out != nullptr)
        F8_TRY_CUDA(cudaMemsetAsync(amax_out, 0, sizeof(float), st));
    if (rows == 0)
        return F8_OK;
    const DistillArgs a =
        distill_args(logits, rows, vocab, ld, ids, values, k, temperature, nullptr,
                     const_cast<float *>(lse), const_cast<float *>(rest), dloss, dlogits, ldd,
                     amax_out, *dev);
    return from_cuda(F8_BY_TYPE(f8::distill_bwd, type, tail, a, *dev, st));
}

f8_status f8_distill_fwd_bwd(const void *logits, f8_dtype type, int64_t rows, int64_t vocab,
                             int64_t ld, const int32_t *ids, const float *values, int k,
                             float temperature, int tail, const float *dloss, float *loss,
                             void *dlogits, int64_t ldd, float *amax_out, void *stream)
{
    F8_TRY(check_logits(logits, type, rows, vocab, ld, temperature));
    F8_TRY(check_slots(ids, values, k, tail, rows));
    F8_TRY(check_out(dlogits, type, rows, vocab, ld, logits, ldd, amax_out));
    if (rows > 0 && (loss == nullptr || dloss == nullptr))
        return F8_ERR_INVALID;
    if (!aligned(loss, 4) || !aligned(dloss, 4))
        return F8_ERR_ALIGN;
    const DeviceInfo *dev;
    F8_TRY(get_device(&dev));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (amax_out != nullptr)
        F8_TRY_CUDA(cudaMemsetAsync(amax_out, 0, sizeof(float), st));
    if (rows == 0)
        return F8_OK;
    const DistillArgs a = distill_args(logits, rows, vocab, ld, ids, values, k, temperature, loss,
                                       nullptr, nullptr, dloss, dlogits, ldd, amax_out, *dev);
    return from_cuda(F8_BY_TYPE(f8::distill_fused, type, tail, a, *dev, st));
}

} // extern "C"
