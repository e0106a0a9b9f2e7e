// norm_common.cuh -- what layer norm and RMS norm share: parameter vectors in
// any format, where rows lie, and sums over the threads of a row.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "block_internal.h"
#include "block_math.cuh"
#include "gn_ptx.cuh"

namespace gn {
namespace norm {

template <typename T, int N>
__device__ __forceinline__ void load_as(const T *p, float (&f)[N])
{
    // (a parameter vector has only its element's alignment)
#pragma unroll
    for (int e = 0; e < N; ++e) f[e] = to_float(p[e]);
}

// N consecutive elements of the weight or the bias, in its own format.
template <int N>
__device__ __forceinline__ void load_params(const void *p, int format, int c, float (&f)[N])
{
    if (format == GN_FORMAT_FP32) {
        const float *q = static_cast<const float *>(p) + c;
        if (N % 4 == 0 && reinterpret_cast<uintptr_t>(q) % 16 == 0) {
#pragma unroll
            for (int e = 0; e < N / 4; ++e) {
                const float4 v = reinterpret_cast<const float4 *>(q)[e];
                f[4 * e] = v.x;
                f[(4 * e + 1) % N] = v.y;
                f[(4 * e + 2) % N] = v.z;
                f[(4 * e + 3) % N] = v.w;
            }
        } else {
            load_as(q, f);
        }
    } else if (format == GN_FORMAT_BF16) {
        load_as(static_cast<const __nv_bfloat16 *>(p) + c, f);
    } else {
        load_as(static_cast<const __half *>(p) + c, f);
    }
}

__device__ __forceinline__ void store_param(void *p, int format, int c, float v)
{
    if (format == GN_FORMAT_FP32)
        static_cast<float *>(p)[c] = v;
    else if (format == GN_FORMAT_BF16)
        static_cast<__nv_bfloat16 *>(p)[c] = __float2bfloat16_rn(v);
    else
        static_cast<__half *>(p)[c] = __float2half_rn(v);
}

// Element offset of row n (rows are counted in 32 bits where they are in two levels).
__device__ __forceinline__ int64_t row_offset(const RowsAt &at, int64_t inner, int64_t rows, int64_t n)
{
    if (inner >= rows) return n * at.stride;
    const uint32_t a = static_cast<uint32_t>(n) / static_cast<uint32_t>(inner);
    return a * at.outer + (n - a * inner) * at.stride;
}

// The same in two steps, for several tensors of a row: the division is most of it.
struct Place {
    int64_t a, b;
};

__device__ __forceinline__ Place row_place(int64_t inner, int64_t rows, int64_t n)
{
    if (inner >= rows) return {0, n};
    const uint32_t a = static_cast<uint32_t>(n) / static_cast<uint32_t>(inner);
    return {a, static_cast<int64_t>(static_cast<uint32_t>(n) - a * static_cast<uint32_t>(inner))};
}

__device__ __forceinline__ int64_t offset_at(const RowsAt &at, const Place &p) { return p.a * at.outer + p.b * at.stride; }

// The threads of one row: tpr of them (a power of two up to 32, or whole
// warps), group g of the CTA's.
struct Group {
    int tpr, g, lane;                // lane: this thread's place in its group
    float (*scratch)[32][2];         // two buffers of the group, taken in turn
    int turn;
};

// Sums of N values over a group.  Within a warp by shuffles; over several
// warps through the group's scratch, whose two buffers make one barrier per
// reduction enough.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], Group &gr)
{
    if (gr.tpr < 32) {
        for (int o = gr.tpr >> 1; o > 0; o >>= 1)
#pragma unroll
            for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
        return;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
    if (gr.tpr == 32) return;
    const int warp = gr.lane >> 5, lane = threadIdx.x & 31, warps = gr.tpr >> 5;
    float(*s)[2] = gr.scratch[gr.turn];
    gr.turn ^= 1;
    if (lane == 0)
#pragma unroll
        for (int n = 0; n < N; ++n) s[warp][n] = v[n];
    named_sync(1 + gr.g, gr.tpr);
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = lane < warps ? s[lane][n] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
}

}  // namespace norm
}  // namespace gn
