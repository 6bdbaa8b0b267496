// Rotary positions: pairs of columns of each head turned by position * frequency.
//
// Bound by HBM: each element is read and written once, with three operations on it.
// A block takes a few rows (tokens) and forms their cosines and sines once in shared
// memory, for all heads of queries and keys; then a thread keeps its place in the head
// and walks the rows' heads, moving two vectors of VEC elements that hold VEC whole
// pairs.  Addresses are the larger part of its instructions: with a place and a head
// worked out per unit, and the rows' starts by division, 8192 rows of 32 + 8 heads of 128
// (96 turned, out of a packed projection) took 34.6 us; so 30.3, 5.5 TB/s.  Dense, halves
// of whole heads 38 us against 31 interleaved.  Units are as wide as rot / 2 lets them be: 8
// bytes for heads of 96 with 24 turned (31 us halves, 27 interleaved, of 18.5 for the
// bytes), 4 for heads of 80 with 20 turned (41 of 15.5).
//
// The angle: a frequency becomes a fraction of a turn in 64-bit fixed point, so
// position * fraction mod 2^64 is the angle's fraction of a turn, exactly; its upper
// 32 bits as a signed number lie in half a turn either way, and sincospi takes them
// without any further reduction.  A far position thus costs no precision, and one
// 64-bit floating point multiplication is all there is of those.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdlib>

#include "f8_internal.h"
#include "f8_ptx.cuh"

namespace f8 {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxDim = 1024;
constexpr int kMaxRows = 8;  // of a block

// x / d for 0 <= x < 2^16 and 1 <= d < 2^16, by the rounded-up reciprocal.
struct Div {
    uint32_t mul, d;
    explicit Div(uint32_t v) : mul(v > 1 ? (0xFFFFFFFFu / v + 1u) : 0u), d(v) {}
    Div() = default;
    __device__ __forceinline__ uint32_t operator()(uint32_t x) const
    {
        return d > 1 ? __umulhi(x, mul) : x;
    }
};

// The elements that a call may touch, around its pointer: for the checked build.
struct Span {
    int64_t lo, n;
    __device__ __forceinline__ bool holds(int64_t i, int len, unsigned *status) const
    {
        return in_range(i - lo, len, n, status);
    }
};

// Of up to three dimensions, `last` dense elements in each place.
Span span_of(const int64_t (&sizes)[3], const int64_t (&strides)[3], int64_t last)
{
    Span s{0, last};
    for (int i = 0; i < 3; ++i) {
        const int64_t far = (sizes[i] - 1) * strides[i];
        s.lo += std::min<int64_t>(far, 0);
        s.n += std::abs(far);
    }
    return s;
}

struct Tensor {
    const void *x;
    void *out;
    int64_t x_batch, x_seq, x_head, out_batch, out_seq, out_head;
    Span x_span, out_span;
};

struct Args {
    Tensor t[2];
    int heads0;          // heads of the first tensor
    int heads;           // of both
    int half;            // pairs of a head
    int turned;          // units of a head that turn
    int units;           // units of a head
    int dim;
    int rows_per_block;
    int64_t rows, seq;
    const int64_t *pos;
    int64_t pos_batch, pos_seq;
    const double *freqs;
    float scale;
    int inverse;
    Span pos_span;
    unsigned *status;
    Div by_units, by_heads, by_half;  // by_units of min(units, threads)
};

template <typename T, int VEC>
struct Vec;
template <>
struct Vec<__nv_bfloat16, 8> {
    using type = uint4;
};
template <>
struct Vec<__nv_bfloat16, 4> {
    using type = uint2;
};
template <>
struct Vec<__nv_bfloat16, 2> {
    using type = uint32_t;
};
template <>
struct Vec<__nv_bfloat16, 1> {
    using type = uint16_t;
};
template <>
struct Vec<float, 4> {
    using type = uint4;
};
template <>
struct Vec<float, 2> {
    using type = uint2;
};
template <>
struct Vec<float, 1> {
    using type = uint32_t;
};

__device__ __forceinline__ float2 to_pair(uint32_t w)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t from_pair(float2 f)
{
    __nv_bfloat162 h = __float22bfloat162_rn(f);
    return *reinterpret_cast<uint32_t *>(&h);
}

// A vector's elements as floats, and back.
template <typename T, int VEC>
__device__ __forceinline__ void unpack(const typename Vec<T, VEC>::type &v, float (&f)[VEC])
{
    if constexpr (sizeof(T) == 4) {
        const float *p = reinterpret_cast<const float *>(&v);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            f[e] = p[e];
    } else if constexpr (VEC == 1) {
        f[0] = __uint_as_float(static_cast<uint32_t>(v) << 16);
    } else {
        const uint32_t *p = reinterpret_cast<const uint32_t *>(&v);
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            const float2 g = to_pair(p[i]);
            f[2 * i] = g.x, f[2 * i + 1] = g.y;
        }
    }
}

template <typename T, int VEC>
__device__ __forceinline__ void pack(const float (&f)[VEC], typename Vec<T, VEC>::type &v)
{
    if constexpr (sizeof(T) == 4) {
        float *p = reinterpret_cast<float *>(&v);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            p[e] = f[e];
    } else if constexpr (VEC == 1) {
        v = __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
    } else {
        uint32_t *p = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i)
            p[i] = from_pair(make_float2(f[2 * i], f[2 * i + 1]));
    }
}

// One pair; the same roundings whatever the vector's width.
__device__ __forceinline__ void turn_pair(float &x1, float &x2, float c, float s)
{
    const float y = fmaf(x1, c, -__fmul_rn(x2, s));
    x2 = fmaf(x2, c, __fmul_rn(x1, s));
    x1 = y;
}

// VEC cosines or sines from shared memory.
template <int VEC>
__device__ __forceinline__ void angles(const float *p, float (&f)[VEC])
{
    if constexpr (VEC >= 4) {
#pragma unroll
        for (int e = 0; e < VEC; e += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(p + e);
            f[e] = v.x, f[e + 1] = v.y, f[e + 2] = v.z, f[e + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            f[e] = p[e];
    }
}

// A frequency (radians a position) as a fraction of a turn in 64 bits; whole turns do
// not count.  The double's 53 bits are moved to their place by shifts.
__device__ __forceinline__ uint64_t turn_fraction(double f)
{
    const int64_t bits = __double_as_longlong(f * 0.15915494309189535);
    const int e = static_cast<int>((bits >> 52) & 0x7FF) - 1023;  // 2^e times [1, 2)
    const uint64_t m = (static_cast<uint64_t>(bits) & 0xFFFFFFFFFFFFFull) | 0x10000000000000ull;
    const int left = e + 12;  // of the 52 bits behind the point
    const uint64_t v = left >= 64 || left <= -64 ? 0ull : (left >= 0 ? m << left : m >> -left);
    return bits < 0 ? 0ull - v : v;
}

// A unit is VEC pairs: columns [VEC u, VEC u + VEC) and the same rot / 2 further on
// (half), or [2 VEC u, 2 VEC u + 2 VEC) (interleaved).  Units from `turned` on are
// two vectors of the columns that are copied, the last unit's second one perhaps
// past the head's end.  A thread keeps its unit and walks the rows' heads.
template <typename T, int VEC, bool HALF>
__global__ void __launch_bounds__(kThreads)
rope_kernel(const __grid_constant__ Args a)
{
    using V = typename Vec<T, VEC>::type;
    extern __shared__ __align__(16) float turn[];  // [2][rows_per_block][half] cosines, then sines, scaled
    __shared__ int64_t at[kMaxRows], base[kMaxRows][4];  // the rows' positions, and where they start
    griddep_wait();
    griddep_launch_dependents();
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * a.rows_per_block;
    const int nrows = static_cast<int>(min(static_cast<int64_t>(a.rows_per_block), a.rows - row0));
    if (threadIdx.x < nrows) {
        const int64_t row = row0 + threadIdx.x, b = row / a.seq, s = row - b * a.seq;
        const int64_t p = b * a.pos_batch + s * a.pos_seq;
        at[threadIdx.x] = a.pos_span.holds(p, 1, a.status) ? a.pos[p] : -1;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            base[threadIdx.x][2 * k] = b * a.t[k].x_batch + s * a.t[k].x_seq;
            base[threadIdx.x][2 * k + 1] = b * a.t[k].out_batch + s * a.t[k].out_seq;
        }
    }
    __syncthreads();
    float *const cosines = turn, *const sines = turn + a.rows_per_block * a.half;
    for (int p = threadIdx.x; p < a.half * nrows; p += kThreads) {
        const int j = static_cast<int>(a.by_half(p));
        if (!in_range(p - j * a.half, 1, a.half, a.status) || !in_range(j, 1, nrows, a.status))
            continue;
        const double f = a.freqs[p - j * a.half];
        const uint64_t angle = turn_fraction(f) * static_cast<uint64_t>(at[j]);
        float t = static_cast<float>(static_cast<int32_t>(angle >> 32)) * 0x1p-31f;  // half turns
        if (((__double_as_longlong(f) >> 52) & 0x7FF) == 0x7FF)
            t = __int_as_float(0x7FC00000);  // infinite or NaN: no angle, and NaN for the pair
        float sn, cs;
        sincospif(t, &sn, &cs);
        cosines[p] = cs * a.scale;
        sines[p] = (a.inverse ? -sn : sn) * a.scale;
    }
    __syncthreads();
    // thread = (slot of heads, unit)
    const int wide = min(a.units, kThreads), slots = kThreads / wide;
    const int slot = static_cast<int>(a.by_units(threadIdx.x)), heads = nrows * a.heads;
    if (slot >= slots)
        return;
    for (int u = threadIdx.x - slot * wide; u < a.units; u += wide) {
        const bool turned = u < a.turned;
        const int c0 = turned ? (HALF ? VEC * u : 2 * VEC * u) : 2 * a.half + 2 * VEC * (u - a.turned);
        const int c1 = turned && HALF ? c0 + a.half : c0 + VEC;
        const bool second = c1 < a.dim;
        for (int i = slot; i < heads; i += slots) {
            const int j = static_cast<int>(a.by_heads(i));
            int h = i - j * a.heads;
            const int k = h >= a.heads0 ? 1 : 0;
            h -= k ? a.heads0 : 0;
            const Tensor &t = a.t[k];
            const int64_t xo = base[j][2 * k] + h * t.x_head, oo = base[j][2 * k + 1] + h * t.out_head;
            const T *x = static_cast<const T *>(t.x) + xo;
            T *o = static_cast<T *>(t.out) + oo;
            if (!in_range(c0, VEC, a.dim, a.status) || !t.x_span.holds(xo + c0, VEC, a.status) ||
                !t.out_span.holds(oo + c0, VEC, a.status))
                continue;
            if (second && (!in_range(c1, VEC, a.dim, a.status) || !t.x_span.holds(xo + c1, VEC, a.status) ||
                           !t.out_span.holds(oo + c1, VEC, a.status)))
                continue;
            V v0 = *reinterpret_cast<const V *>(x + c0), v1 = v0;
            if (second)
                v1 = *reinterpret_cast<const V *>(x + c1);
            if (turned && at[j] >= 0) {
                float p[VEC], q[VEC], cs[VEC], sn[VEC];
                unpack<T, VEC>(v0, p);
                unpack<T, VEC>(v1, q);
                const int from = j * a.half + VEC * u;
                angles<VEC>(cosines + from, cs);
                angles<VEC>(sines + from, sn);
                if constexpr (HALF || VEC == 1) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        turn_pair(p[e], q[e], cs[e], sn[e]);
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; e += 2) {
                        turn_pair(p[e], p[e + 1], cs[e / 2], sn[e / 2]);
                        turn_pair(q[e], q[e + 1], cs[VEC / 2 + e / 2], sn[VEC / 2 + e / 2]);
                    }
                }
                pack<T, VEC>(p, v0);
                pack<T, VEC>(q, v1);
            }
            *reinterpret_cast<V *>(o + c0) = v0;
            if (second)
                *reinterpret_cast<V *>(o + c1) = v1;
        }
    }
}

template <typename T, int VEC, bool HALF>
cudaError_t run(Args &a, const DeviceInfo &dev, cudaStream_t st)
{
    a.turned = a.half / VEC;
    a.units = a.turned + (a.dim - 2 * a.half + 2 * VEC - 1) / (2 * VEC);
    const int per_row = a.heads * a.units;
    // rows of a block: some 1024 units, while all SMs have blocks, within 32 KB of
    // cosines and sines
    int64_t r = std::min<int64_t>(kMaxRows, std::max(1, 1024 / per_row));
    r = std::min<int64_t>(r, std::max<int64_t>(1, a.rows / (4 * dev.sm_count)));
    r = std::min<int64_t>(r, std::max(1, 4096 / a.half));
    a.rows_per_block = static_cast<int>(r);
    a.by_units = Div(static_cast<uint32_t>(std::min(a.units, kThreads)));
    a.by_heads = Div(static_cast<uint32_t>(a.heads));
    a.by_half = Div(static_cast<uint32_t>(a.half));
    const int64_t blocks = (a.rows + r - 1) / r;
    return launch_pdl(rope_kernel<T, VEC, HALF>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads),
                      2 * static_cast<size_t>(r) * a.half * sizeof(float), st, a);
}

template <typename T, bool HALF>
cudaError_t pick(Args &a, int vec, const DeviceInfo &dev, cudaStream_t st)
{
    if constexpr (sizeof(T) == 2)
        if (vec == 8)
            return run<T, 8, HALF>(a, dev, st);
    switch (vec) {
    case 4: return run<T, 4, HALF>(a, dev, st);
    case 2: return run<T, 2, HALF>(a, dev, st);
    default: return run<T, 1, HALF>(a, dev, st);
    }
}

// The widest vector (elements) whose units the columns, strides and addresses allow.
int vector_of(const f8_rope_tensor *t, int count, int esize, int64_t batch, int64_t seq, int64_t dim,
              int64_t rot)
{
    for (int v = 16 / esize; v > 1; v /= 2) {
        bool ok = (rot / 2) % v == 0 && dim % v == 0;
        for (int i = 0; i < count && ok; ++i) {
            const int64_t strides[6] = {batch > 1 ? t[i].x_batch : 0,   seq > 1 ? t[i].x_seq : 0,
                                        t[i].heads > 1 ? t[i].x_head : 0, batch > 1 ? t[i].out_batch : 0,
                                        seq > 1 ? t[i].out_seq : 0,     t[i].heads > 1 ? t[i].out_head : 0};
            for (int64_t s : strides)
                ok = ok && s % v == 0;
            ok = ok && aligned(t[i].x, static_cast<uintptr_t>(v) * esize) &&
                 aligned(t[i].out, static_cast<uintptr_t>(v) * esize);
        }
        if (ok)
            return v;
    }
    return 1;
}

} // namespace
} // namespace f8

using namespace f8;

extern "C" {

f8_status f8_rope(const f8_rope_tensor *tensors, int count, f8_dtype type, int64_t batch,
                  int64_t seq, int64_t dim, int64_t rot, f8_rope_layout layout,
                  const int64_t *positions, int64_t pos_batch, int64_t pos_seq, const double *freqs,
                  float scale, int inverse, void *stream)
{
    if (tensors == nullptr || count < 1 || count > 2 || (type != F8_BF16 && type != F8_F32) ||
        (layout != F8_ROPE_HALF && layout != F8_ROPE_INTERLEAVED) || batch < 0 || seq < 0 || dim < 0 ||
        !std::isfinite(scale))
        return F8_ERR_INVALID;
    if (rot < 2 || rot % 2 != 0 || rot > dim || dim > kMaxDim)
        return F8_ERR_SHAPE;
    const int esize = type == F8_BF16 ? 2 : 4;
    int64_t heads = 0;
    const bool some = batch > 0 && seq > 0;
    for (int i = 0; i < count; ++i) {
        const f8_rope_tensor &t = tensors[i];
        if (t.heads < 0)
            return F8_ERR_INVALID;
        if (t.heads > 1 << 12)
            return F8_ERR_SHAPE;
        heads += t.heads;
        if (some && t.heads > 0 && (t.x == nullptr || t.out == nullptr))
            return F8_ERR_INVALID;
        if (some && t.heads > 0) {
            // strides count where more than one element goes by them
            const bool b = batch > 1, q = seq > 1, h = t.heads > 1;
            // in place means in place: another order of the rows would read what it wrote
            if (t.x == t.out && ((b && t.x_batch != t.out_batch) || (q && t.x_seq != t.out_seq) ||
                                 (h && t.x_head != t.out_head)))
                return F8_ERR_INVALID;
            // rows of the output lie apart
            if ((b && t.out_batch == 0) || (q && t.out_seq == 0) || (h && t.out_head == 0))
                return F8_ERR_INVALID;
        }
        if (!aligned(t.x, esize) || !aligned(t.out, esize))
            return F8_ERR_ALIGN;
    }
    if (some && heads > 0 && (positions == nullptr || freqs == nullptr))
        return F8_ERR_INVALID;
    if (!aligned(positions, 8) || !aligned(freqs, 8))
        return F8_ERR_ALIGN;
    if (batch > 0 && seq > INT32_MAX / batch)
        return F8_ERR_SHAPE;
    const DeviceInfo *dev;
    F8_TRY(get_device(&dev));
    if (!some || heads == 0)
        return F8_OK;
    const int vec = vector_of(tensors, count, esize, batch, seq, dim, rot);
    Args a = {};
    for (int i = 0; i < count; ++i) {
        const f8_rope_tensor &t = tensors[i];
        const int64_t sizes[3] = {batch, seq, std::max<int64_t>(t.heads, 1)};
        a.t[i] = Tensor{t.x, t.out, t.x_batch, t.x_seq, t.x_head, t.out_batch, t.out_seq, t.out_head,
                        span_of(sizes, {t.x_batch, t.x_seq, t.x_head}, dim),
                        span_of(sizes, {t.out_batch, t.out_seq, t.out_head}, dim)};
    }
    a.heads0 = static_cast<int>(tensors[0].heads);
    a.heads = static_cast<int>(heads);
    a.half = static_cast<int>(rot / 2);
    a.dim = static_cast<int>(dim);
    a.rows = batch * seq;
    a.seq = seq;
    a.pos = positions;
    a.pos_batch = pos_batch;
    a.pos_seq = pos_seq;
    a.freqs = freqs;
    a.scale = scale;
    a.inverse = inverse != 0;
    a.pos_span = span_of({batch, seq, 1}, {pos_batch, pos_seq, 0}, 1);
    a.status = dev->status;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool half = layout == F8_ROPE_HALF;
    if (type == F8_BF16)
        return from_cuda(half ? pick<__nv_bfloat16, true>(a, vec, *dev, st)
                              : pick<__nv_bfloat16, false>(a, vec, *dev, st));
    return from_cuda(half ? pick<float, true>(a, vec, *dev, st) : pick<float, false>(a, vec, *dev, st));
}

f8_status f8_rope_frequencies(int64_t rot, double base, f8_rope_scaling scaling, double factor,
                              double original, double slow, double fast, double *freqs)
{
    if (freqs == nullptr || !(base > 0.0) || !std::isfinite(base) || scaling < F8_ROPE_PLAIN ||
        scaling > F8_ROPE_BY_PARTS)
        return F8_ERR_INVALID;
    if (rot < 2 || rot % 2 != 0 || rot > kMaxDim || (scaling == F8_ROPE_BASE && rot == 2))
        return F8_ERR_SHAPE;
    if (scaling != F8_ROPE_PLAIN && !(factor > 0.0 && std::isfinite(factor)))
        return F8_ERR_INVALID;
    if (scaling == F8_ROPE_BY_PARTS && !(original > 0.0 && std::isfinite(original) && slow >= 0.0 && slow < fast &&
                                         std::isfinite(fast)))
        return F8_ERR_INVALID;
    const double n = static_cast<double>(rot);
    if (scaling == F8_ROPE_BASE)
        base *= std::pow(factor, n / (n - 2.0));
    for (int64_t i = 0; i < rot / 2; ++i) {
        double f = std::pow(base, -2.0 * static_cast<double>(i) / n);
        if (scaling == F8_ROPE_LINEAR) {
            f /= factor;
        } else if (scaling == F8_ROPE_BY_PARTS) {
            const double turns = original * f / 6.283185307179586;
            const double keep = std::min(1.0, std::max(0.0, (turns - slow) / (fast - slow)));
            f = f * keep + f / factor * (1.0 - keep);
        }
        freqs[i] = f;
    }
    return F8_OK;
}

} // extern "C"
