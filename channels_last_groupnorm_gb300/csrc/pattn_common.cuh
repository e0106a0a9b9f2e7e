// pattn_common.cuh -- what the packed-attention kernels share: which keys a
// query sees (and which queries see a key), the score of a pair, and half
// precision packing.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "block_internal.h"
#include "block_math.cuh"
#include "gn_ptx.cuh"

namespace gn {
namespace pattn {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// A run [lo, hi) of tokens on the other side.  pos: for a query, the key
// coordinate it stands at (the last query of a document stands at its last key).
struct Span {
    int lo, hi, pos;
};

// The document whose run holds `token`, or -1.  ends: [docs + 1] non-decreasing
// (whatever it holds, the search ends and reads only the array).
__device__ __forceinline__ int doc_of(const int32_t *ends, int docs, int token)
{
    int low = 0, high = docs;   // ends[low] <= token is only known once low moved
    while (high - low > 1) {
        const int mid = (low + high) >> 1;
        if (__ldg(ends + mid) <= token)
            low = mid;
        else
            high = mid;
    }
    return token >= __ldg(ends + low) && token < __ldg(ends + low + 1) ? low : -1;
}

// A document's queries [qb, qe) and keys [kb, ke), clamped into the tensors,
// and its prefix length in [0, ke - kb].
struct Doc {
    int qb, qe, kb, ke, prefix;
};

__device__ __forceinline__ Doc doc_bounds(const gn_attn_packed_args &a, int d)
{
    Doc r;
    const int tq = static_cast<int>(a.tokens_q), tk = static_cast<int>(a.tokens_k);
    r.qb = a.cu_q ? min(max(__ldg(a.cu_q + d), 0), tq) : 0;
    r.qe = a.cu_q ? min(max(__ldg(a.cu_q + d + 1), r.qb), tq) : tq;
    r.kb = a.cu_k ? min(max(__ldg(a.cu_k + d), 0), tk) : 0;
    r.ke = a.cu_k ? min(max(__ldg(a.cu_k + d + 1), r.kb), tk) : tk;
    r.prefix = a.prefix ? min(max(__ldg(a.prefix + d), 0), r.ke - r.kb) : 0;
    return r;
}

// The keys that query i sees.
__device__ __forceinline__ Span query_span_in(const gn_attn_packed_args &a, const Doc &d, int i)
{
    Span s;
    s.lo = d.kb;
    s.hi = d.ke;
    s.pos = d.ke - (d.qe - i);
    if (a.causal) s.hi = max(d.kb, min(d.ke, max(s.pos + 1, d.kb + d.prefix)));
    return s;
}

__device__ __forceinline__ Span query_span(const gn_attn_packed_args &a, int i)
{
    const int d = a.cu_q ? doc_of(a.cu_q, a.docs, i) : 0;
    if (d < 0) return Span{0, 0, 0};
    return query_span_in(a, doc_bounds(a, d), i);
}

// The queries that see key j (pos unused).
__device__ __forceinline__ Span key_span(const gn_attn_packed_args &a, int j)
{
    const int n = a.cu_k ? doc_of(a.cu_k, a.docs, j) : 0;
    if (n < 0) return Span{0, 0, 0};
    const Doc d = doc_bounds(a, n);
    Span s = {d.qb, d.qe, 0};
    // position of query i: ke - (qe - i) >= j
    if (a.causal && j - d.kb >= d.prefix) s.lo = min(d.qe, max(d.qb, j - d.ke + d.qe));
    return s;
}

// tanh to full fp32 accuracy near and far from zero (the one-instruction
// approximation is good to 2^-11 only, which a cap of 50 would turn into a
// score error of 0.02): 1 - 2 / (1 + e^2|x|), whose absolute error is a few 2^-24.
__device__ __forceinline__ float tanh_full(float x)
{
    const float e = ex2_approx(2.0f * kLog2e * fabsf(x));
    return copysignf(1.0f - 2.0f * __frcp_rn(1.0f + e), x);
}

// The same in four instructions (rcp.approx: 2^-23 of a quotient of at most
// 1), for the kernels that do it for every score.
__device__ __forceinline__ float tanh_fast(float x)
{
    const float e = ex2_approx(2.0f * kLog2e * fabsf(x));
    return copysignf(fmaf(-2.0f, rcp_approx(1.0f + e), 1.0f), x);
}

// The score of a pair in units of log2 (dot: q . k unscaled), and in `slack`
// the derivative of the capped score by the uncapped one.
__device__ __forceinline__ float score_log2(const gn_attn_packed_args &a, float slope, float dot, int pos, int j,
                                            float &slack)
{
    float t = dot * a.scale;
    slack = 1.0f;
    if (a.cap > 0.f) {
        const float th = tanh_full(t / a.cap);
        t = a.cap * th;
        slack = fmaf(-th, th, 1.0f);
    }
    return (t - slope * fabsf(static_cast<float>(pos - j))) * kLog2e;
}

template <typename T>
__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = Half2<T>::unpack(w[i]);
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
    }
}

// Four channels of one token's head, lane l of a warp taking channels 4 l..4 l + 3
// (zeros past the head's width).
template <typename T>
__device__ __forceinline__ float4 load4(const void *base, int64_t offset, int lane, int dim)
{
    if (4 * lane >= dim) return make_float4(0.f, 0.f, 0.f, 0.f);
    const uint2 v = *reinterpret_cast<const uint2 *>(static_cast<const T *>(base) + offset + 4 * lane);
    const float2 a = Half2<T>::unpack(v.x), b = Half2<T>::unpack(v.y);
    return make_float4(a.x, a.y, b.x, b.y);
}

template <typename T>
__device__ __forceinline__ void store4(void *base, int64_t offset, int lane, int dim, float4 f)
{
    if (4 * lane >= dim) return;
    *reinterpret_cast<uint2 *>(static_cast<T *>(base) + offset + 4 * lane) =
        make_uint2(Half2<T>::pack(f.x, f.y), Half2<T>::pack(f.z, f.w));
}

__device__ __forceinline__ float dot4(float4 a, float4 b) { return a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w; }

__device__ __forceinline__ void axpy4(float4 &acc, float s, float4 x)
{
    acc.x = fmaf(s, x.x, acc.x);
    acc.y = fmaf(s, x.y, acc.y);
    acc.z = fmaf(s, x.z, acc.z);
    acc.w = fmaf(s, x.w, acc.w);
}

// Whether a warp's sums (four channels a lane, dim in all) are NaN throughout:
// nothing that is added changes them any more.
__device__ __forceinline__ bool all_nan(float4 f, int lane, int dim)
{
    return __all_sync(0xffffffffu, 4 * lane >= dim || (isnan(f.x) && isnan(f.y) && isnan(f.z) && isnan(f.w)));
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

}  // namespace pattn
}  // namespace gn
