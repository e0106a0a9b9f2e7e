// rms_kernels.cu -- sm_103a kernels of RMS norm over the last axis, with the
// residual's addition and an output in 8 bits, and of its backward pass.
//
//   forward   t = x + residual (rounded to the type of x), rstd = 1 / sqrt(sum(t^2) / C + eps),
//             y = t rstd w, in the type of x or as e4m3 of y / scale, scale = max |y| / 448
//   backward  with g = dy w and h = t rstd,
//             dx = rstd g - t rstd^3 sum(g t) / C + dtotal,  dw = sum over rows of dy h
//
// Both are bound by memory.  A row is held in the registers of `tpr` threads (NV
// slots each of EPV consecutive elements), so that everything is read once: the
// sum of squares, the largest magnitude and the output are passes over registers.
// A thread keeps its columns for every row that it meets: in the backward pass it
// adds up its part of dw in registers.  Sums are fp32; each output is rounded once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <initializer_list>
#include <utility>

#include "block_internal.h"
#include "block_math.cuh"
#include "gn_ptx.cuh"
#include "norm_common.cuh"
#include "tc_common.cuh"

namespace gn {
namespace {

using namespace norm;

// A row in 8 bits: its scale and what is made of t w, from the largest |t w|.  The quotient
// q = 448 t w / max |t w| gets one step of Newton's method, q0 + (448 t w - q0 max) / max with
// q0 = t w (448 / max): with half formats t w is exact, and what lies halfway between two e4m3
// numbers then still does.  (448 = 7 x 64, so 7 t w is exact too.  4608 x 6144: 48 us replayed, 45
// without the step, when one value in 6144 or so came out a step off.)
struct RowScale {
    float scale, by, seventh, part;
    __device__ __forceinline__ RowScale(float most, float rstd)
    {
        const float top = most * rstd;
        const bool none = top < 1e-30f || most < 0x1p-110f;
        scale = none ? 0.f : top / 448.0f;
        by = none ? 0.f : top == top ? 448.0f / most : top;      // (an infinity's row is no number)
        seventh = by * (1.0f / 7.0f);
        part = most * (1.0f / 64.0f);
    }
    __device__ __forceinline__ float of(float v) const
    {
        const float q = v * by;
        return fmaf(fmaf(-q, part, 7.0f * v), seventh, q);
    }
};

template <typename T, int EPV>
struct Slot {
    uint4 raw;          // EPV == 1: raw.x is the value in fp32

    __device__ __forceinline__ void load(const T *p)
    {
        if (EPV == 1)
            raw.x = __float_as_uint(to_float(*p));
        else
            raw = *reinterpret_cast<const uint4 *>(p);
    }
    __device__ __forceinline__ void clear() { raw = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(float (&f)[EPV]) const
    {
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
        if constexpr (EPV == 1) {
            f[0] = __uint_as_float(w[0]);
        } else if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = __uint_as_float(w[e]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 v = Half2<T>::unpack(w[e]);
                f[2 * e] = v.x;
                f[2 * e + 1] = v.y;
            }
        }
    }
    // (rounded to T)
    __device__ __forceinline__ void set(const float (&f)[EPV])
    {
        if constexpr (EPV == 1) {
            raw.x = __float_as_uint(to_float(from_float<T>(f[0])));
        } else if constexpr (sizeof(T) == 4) {
            raw = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
        } else {
            raw = make_uint4(Half2<T>::pack(f[0], f[1]), Half2<T>::pack(f[2], f[3]), Half2<T>::pack(f[4], f[5]),
                             Half2<T>::pack(f[6], f[7]));
        }
    }
    __device__ __forceinline__ void store(T *p) const
    {
        if (EPV == 1)
            *p = from_float<T>(__uint_as_float(raw.x));
        else
            *reinterpret_cast<uint4 *>(p) = raw;
    }
};

template <int EPV>
__device__ __forceinline__ void store_e4m3(uint8_t *p, const float (&f)[EPV])
{
    if constexpr (EPV == 8)
        *reinterpret_cast<uint2 *>(p) = make_uint2(e4m3_four(f[0], f[1], f[2], f[3]), e4m3_four(f[4], f[5], f[6], f[7]));
    else if constexpr (EPV == 4)
        *reinterpret_cast<uint32_t *>(p) = e4m3_four(f[0], f[1], f[2], f[3]);
    else
        *p = static_cast<uint8_t>(e4m3_pair(f[0], 0.f));
}

// A sum and a maximum (NaN if any value is) over a group, in one go.
__device__ __forceinline__ void row_sum_max(float &sum, float &most, Group &gr)
{
    for (int o = min(gr.tpr, 32) >> 1; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, o));
    }
    if (gr.tpr <= 32) return;
    const int warp = gr.lane >> 5, lane = threadIdx.x & 31, warps = gr.tpr >> 5;
    float(*s)[2] = gr.scratch[gr.turn];
    gr.turn ^= 1;
    if (lane == 0) {
        s[warp][0] = sum;
        s[warp][1] = most;
    }
    named_sync(1 + gr.g, gr.tpr);
    sum = lane < warps ? s[lane][0] : 0.f;
    most = lane < warps ? s[lane][1] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, o));
    }
}

__device__ __forceinline__ Group group_of(int tpr, float (*scratch)[2][32][2])
{
    Group gr;
    gr.tpr = tpr;
    gr.g = static_cast<int>(threadIdx.x) / tpr;
    gr.lane = static_cast<int>(threadIdx.x) - gr.g * tpr;
    gr.scratch = scratch[tpr > 32 ? gr.g : 0];
    gr.turn = 0;
    return gr;
}

constexpr int kMaxGroups = 8;      // of more than a warp in a CTA

// The weight in fp32 in shared memory: as vectors whatever its format is, and no registers
// held for it (two CTAs on an SM instead of one; 4608 x 6144 with residual, e4m3 out).
__device__ __forceinline__ void stage_weight(float *to, const void *weight, int format, int cols)
{
    if (!weight) return;
    const int bytes = format == GN_FORMAT_FP32 ? 4 : 2, wide = 16 / bytes;
    if (cols % wide || reinterpret_cast<uintptr_t>(weight) % 16) {
        for (int c = threadIdx.x; c < cols; c += blockDim.x) {
            float w[1];
            load_params<1>(weight, format, c, w);
            to[c] = w[0];
        }
        return;
    }
    for (int i = threadIdx.x; i < cols / wide; i += blockDim.x) {
        const uint4 v = __ldg(static_cast<const uint4 *>(weight) + i);
        if (format == GN_FORMAT_FP32) {
            reinterpret_cast<uint4 *>(to)[i] = v;
            continue;
        }
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
            const float2 p = format == GN_FORMAT_BF16 ? Half2<__nv_bfloat16>::unpack(w[e]) : Half2<__half>::unpack(w[e]);
            const float2 q = format == GN_FORMAT_BF16 ? Half2<__nv_bfloat16>::unpack(w[e + 1]) : Half2<__half>::unpack(w[e + 1]);
            reinterpret_cast<float4 *>(to)[2 * i + e / 2] = make_float4(p.x, p.y, q.x, q.y);
        }
    }
}

// EPV of them, ones without a weight.
template <int EPV>
__device__ __forceinline__ void weight_at(const float *staged, bool there, int c, float (&w)[EPV])
{
    if (!there) {
#pragma unroll
        for (int e = 0; e < EPV; ++e) w[e] = 1.0f;
    } else if constexpr (EPV == 1) {
        w[0] = staged[c];
    } else {
#pragma unroll
        for (int e = 0; e < EPV; e += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(staged + c + e);
            w[e] = v.x, w[e + 1] = v.y, w[e + 2] = v.z, w[e + 3] = v.w;
        }
    }
}

// A thread's slots of a row (zeros where there is none).
template <typename T, int EPV, int NV>
__device__ __forceinline__ void load_row(Slot<T, EPV> (&s)[NV], const void *p, const RowsAt &at, int64_t inner, int64_t rows,
                                         int64_t n, const Group &gr, int cols)
{
    const T *row = p && n < rows ? static_cast<const T *>(p) + row_offset(at, inner, rows, n) : nullptr;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = (gr.lane + k * gr.tpr) * EPV;
        if (row && c < cols)
            s[k].load(row + c);
        else
            s[k].clear();
    }
}

// Rows of up to 32 vectors (the heads of a projection): a group of lanes takes some of them
// at a time, so that enough is on its way, and looks up once where a row lies in all tensors
// (4608 x 24 rows of 128, a training step replayed: 42 us with two rows, 49 with four, 58 with
// eight, whose registers leave too few CTAs).
constexpr int kShortRows = 2;

template <typename T, int EPV>
__global__ void __launch_bounds__(256) rms_short_kernel(const __grid_constant__ RmsArgs a, int tpr)
{
    extern __shared__ __align__(16) float staged[];
    tc::griddep_wait();
    if (threadIdx.x == 0) tc::griddep_launch_dependents();
    const int per = blockDim.x / tpr, group = threadIdx.x / tpr, lane = threadIdx.x - group * tpr, c = lane * EPV;
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    const bool in = c < a.cols;
    stage_weight(staged, a.weight, a.weight_format, a.cols);
    __syncthreads();
    float w[EPV];
    if (in) weight_at<EPV>(staged, a.weight != nullptr, c, w);
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * per * kShortRows; first < a.rows;
         first += static_cast<int64_t>(gridDim.x) * per * kShortRows) {
        Slot<T, EPV> t[kShortRows], r[kShortRows];
        float sum[kShortRows], most[kShortRows];
        Place at[kShortRows];
#pragma unroll
        for (int q = 0; q < kShortRows; ++q) {
            const int64_t n = first + group + q * per;
            t[q].clear();
            r[q].clear();
            at[q] = row_place(a.inner, a.rows, n);
            if (in && n < a.rows) {
                t[q].load(static_cast<const T *>(a.x) + offset_at(a.x_at, at[q]) + c);
                if (a.residual) r[q].load(static_cast<const T *>(a.residual) + offset_at(a.residual_at, at[q]) + c);
            }
        }
#pragma unroll
        for (int q = 0; q < kShortRows; ++q) {
            const int64_t n = first + group + q * per;
            float f[EPV], g[EPV];
            t[q].get(f);
            if (a.residual) {
                r[q].get(g);
#pragma unroll
                for (int e = 0; e < EPV; ++e) f[e] += g[e];
                t[q].set(f);
                if (in && n < a.rows) t[q].store(static_cast<T *>(a.total) + offset_at(a.total_at, at[q]) + c);
                t[q].get(f);
            }
            sum[q] = most[q] = 0.f;
#pragma unroll
            for (int e = 0; e < EPV; ++e) sum[q] = fmaf(f[e], f[e], sum[q]);
            if (a.scales && in)
#pragma unroll
                for (int e = 0; e < EPV; ++e) most[q] = max_nan(most[q], fabsf(f[e] * w[e]));
        }
        for (int o = tpr >> 1; o > 0; o >>= 1)
#pragma unroll
            for (int q = 0; q < kShortRows; ++q) {
                sum[q] += __shfl_xor_sync(0xffffffffu, sum[q], o);
                if (a.scales) most[q] = max_nan(most[q], __shfl_xor_sync(0xffffffffu, most[q], o));
            }
#pragma unroll
        for (int q = 0; q < kShortRows; ++q) {
            const int64_t n = first + group + q * per;
            if (!in || n >= a.rows) continue;
            const float rstd = 1.0f / sqrtf(fmaf(sum[q], inv_cols, a.eps));
            if (lane == 0 && a.rstd) a.rstd[n] = rstd;
            float f[EPV];
            t[q].get(f);
            const int64_t to = offset_at(a.y_at, at[q]) + c;
            if (!a.scales) {
#pragma unroll
                for (int e = 0; e < EPV; ++e) f[e] = f[e] * rstd * w[e];
                Slot<T, EPV> o;
                o.set(f);
                o.store(static_cast<T *>(a.y) + to);
                continue;
            }
            const RowScale o(most[q], rstd);
            if (lane == 0) a.scales[n] = o.scale;
#pragma unroll
            for (int e = 0; e < EPV; ++e) f[e] = o.of(f[e] * w[e]);
            store_e4m3<EPV>(static_cast<uint8_t *>(a.y) + to, f);
        }
    }
}

template <typename T, int EPV>
__global__ void __launch_bounds__(256) rms_short_grad_kernel(const __grid_constant__ RmsGradArgs a, int tpr)
{
    extern __shared__ __align__(16) float staged[];       // the weight, then [groups][cols] sums
    tc::griddep_wait();
    if (threadIdx.x == 0) tc::griddep_launch_dependents();
    const int per = blockDim.x / tpr, group = threadIdx.x / tpr, lane = threadIdx.x - group * tpr, c = lane * EPV;
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    const bool in = c < a.cols;
    stage_weight(staged, a.weight, a.weight_format, a.cols);
    __syncthreads();
    float w[EPV], dw[EPV] = {};
    if (in) weight_at<EPV>(staged, a.weight != nullptr, c, w);
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * per * kShortRows; first < a.rows;
         first += static_cast<int64_t>(gridDim.x) * per * kShortRows) {
        Slot<T, EPV> t[kShortRows], dy[kShortRows], dt[kShortRows];
        float sum[kShortRows], rstd[kShortRows];
        Place at[kShortRows];
#pragma unroll
        for (int q = 0; q < kShortRows; ++q) {
            const int64_t n = first + group + q * per;
            t[q].clear();
            dy[q].clear();
            dt[q].clear();
            rstd[q] = 0.f;
            at[q] = row_place(a.inner, a.rows, n);
            if (in && n < a.rows) {
                t[q].load(static_cast<const T *>(a.total) + offset_at(a.total_at, at[q]) + c);
                dy[q].load(static_cast<const T *>(a.dy) + offset_at(a.dy_at, at[q]) + c);
                if (a.dtotal) dt[q].load(static_cast<const T *>(a.dtotal) + offset_at(a.dtotal_at, at[q]) + c);
                rstd[q] = __ldg(a.rstd + n);
            }
        }
#pragma unroll
        for (int q = 0; q < kShortRows; ++q) {
            float f[EPV], g[EPV];
            t[q].get(f);
            dy[q].get(g);
            sum[q] = 0.f;
            if (in)
#pragma unroll
                for (int e = 0; e < EPV; ++e) {
                    dw[e] = fmaf(g[e], f[e] * rstd[q], dw[e]);
                    sum[q] = fmaf(g[e] * w[e], f[e], sum[q]);
                }
        }
        for (int o = tpr >> 1; o > 0; o >>= 1)
#pragma unroll
            for (int q = 0; q < kShortRows; ++q) sum[q] += __shfl_xor_sync(0xffffffffu, sum[q], o);
#pragma unroll
        for (int q = 0; q < kShortRows; ++q) {
            const int64_t n = first + group + q * per;
            if (!in || n >= a.rows) continue;
            const float along = sum[q] * inv_cols * rstd[q] * rstd[q];
            float f[EPV], g[EPV], r[EPV];
            t[q].get(f);
            dy[q].get(g);
            dt[q].get(r);
#pragma unroll
            for (int e = 0; e < EPV; ++e) f[e] = fmaf(rstd[q], fmaf(-f[e], along, g[e] * w[e]), r[e]);
            Slot<T, EPV> o;
            o.set(f);
            o.store(static_cast<T *>(a.dx) + offset_at(a.dx_at, at[q]) + c);
        }
    }
    if (!a.weight) return;
    float *columns = staged + (a.cols + 3) / 4 * 4;
    if (in)
#pragma unroll
        for (int e = 0; e < EPV; ++e) columns[group * a.cols + c + e] = dw[e];
    __syncthreads();
    float *out = a.partial + static_cast<int64_t>(blockIdx.x) * a.cols;
    for (int i = threadIdx.x; i < a.cols; i += blockDim.x) {
        float v = 0.f;
        for (int g = 0; g < per; ++g) v += columns[g * a.cols + i];
        out[i] = v;
    }
}

template <typename T, int EPV, int NV, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) rms_kernel(const __grid_constant__ RmsArgs a, int tpr)
{
    __shared__ float scratch[kMaxGroups][2][32][2];
    extern __shared__ __align__(16) float staged[];
    tc::griddep_wait();
    if (threadIdx.x == 0) tc::griddep_launch_dependents();
    Group gr = group_of(tpr, scratch);
    const int per = blockDim.x / tpr;
    const int64_t step = static_cast<int64_t>(gridDim.x) * per;
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    const bool weighed = a.weight != nullptr;
    int64_t first = static_cast<int64_t>(blockIdx.x) * per;
    Slot<T, EPV> x[NV], r[NV];
    load_row(x, a.x, a.x_at, a.inner, a.rows, first + gr.g, gr, a.cols);
    if (a.residual) load_row(r, a.residual, a.residual_at, a.inner, a.rows, first + gr.g, gr, a.cols);
    stage_weight(staged, a.weight, a.weight_format, a.cols);
    __syncthreads();
    // (the rows of a CTA's groups end together: a warp's lanes shuffle as one)
    for (; first < a.rows; first += step) {
        const int64_t n = first + gr.g;
        const bool live = n < a.rows;
        Slot<T, EPV> t[NV];
        float sum = 0.f, most = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) t[k] = x[k];
        if (a.residual) {
            T *to = live ? static_cast<T *>(a.total) + row_offset(a.total_at, a.inner, a.rows, n) : nullptr;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (gr.lane + k * tpr) * EPV;
                float f[EPV], g[EPV];
                x[k].get(f);
                r[k].get(g);
#pragma unroll
                for (int e = 0; e < EPV; ++e) f[e] += g[e];
                t[k].set(f);
                if (live && c < a.cols) t[k].store(to + c);
            }
        }
        // the next row is on its way while this one is worked on (in place, another
        // row's elements are another's: nothing written here is read there)
        load_row(x, a.x, a.x_at, a.inner, a.rows, n + step, gr, a.cols);
        if (a.residual) load_row(r, a.residual, a.residual_at, a.inner, a.rows, n + step, gr, a.cols);
        // the squares' sum, and the largest |t w| with it: |y| is that times rstd
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (gr.lane + k * tpr) * EPV;
            float f[EPV], w[EPV];
            t[k].get(f);
#pragma unroll
            for (int e = 0; e < EPV; ++e) sum = fmaf(f[e], f[e], sum);
            if (!a.scales || c >= a.cols) continue;
            weight_at<EPV>(staged, weighed, c, w);
#pragma unroll
            for (int e = 0; e < EPV; ++e) most = max_nan(most, fabsf(f[e] * w[e]));
        }
        row_sum_max(sum, most, gr);
        const float rstd = 1.0f / sqrtf(fmaf(sum, inv_cols, a.eps));
        if (live && gr.lane == 0 && a.rstd) a.rstd[n] = rstd;
        if (!a.scales) {
            T *y = live ? static_cast<T *>(a.y) + row_offset(a.y_at, a.inner, a.rows, n) : nullptr;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (gr.lane + k * tpr) * EPV;
                if (!live || c >= a.cols) continue;
                float f[EPV], w[EPV];
                t[k].get(f);
                weight_at<EPV>(staged, weighed, c, w);
#pragma unroll
                for (int e = 0; e < EPV; ++e) f[e] = f[e] * rstd * w[e];
                Slot<T, EPV> o;
                o.set(f);
                o.store(y + c);
            }
            continue;
        }
        const RowScale o(most, rstd);
        if (live && gr.lane == 0) a.scales[n] = o.scale;
        uint8_t *y = live ? static_cast<uint8_t *>(a.y) + row_offset(a.y_at, a.inner, a.rows, n) : nullptr;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (gr.lane + k * tpr) * EPV;
            if (!live || c >= a.cols) continue;
            float f[EPV], w[EPV];
            t[k].get(f);
            weight_at<EPV>(staged, weighed, c, w);
#pragma unroll
            for (int e = 0; e < EPV; ++e) f[e] = o.of(f[e] * w[e]);
            store_e4m3<EPV>(y + c, f);
        }
    }
}

// Rows on their way to a thread's own places in shared memory (whole vectors only):
// nobody else reads them, so no barrier is needed, and no registers are held.
__device__ __forceinline__ void copy_async(uint32_t to, const void *from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// AHEAD rows of each thread's groups are on their way while one is worked on (vectors only;
// 4608 x 6144 with dtotal, a step replayed: 104 us with the next row's loads behind this one's
// stores, 98 with one row ahead, 99 with two).
template <typename T, int EPV, int NV, int THREADS, int CTAS, int AHEAD>
__global__ void __launch_bounds__(THREADS, CTAS) rms_grad_kernel(const __grid_constant__ RmsGradArgs a, int tpr)
{
    __shared__ float scratch[kMaxGroups][2][32][2];
    // the weight, [AHEAD][3][NV][threads] vectors, then [groups][cols] sums where a CTA has several
    extern __shared__ __align__(16) float staged[];
    tc::griddep_wait();
    if (threadIdx.x == 0) tc::griddep_launch_dependents();
    Group gr = group_of(tpr, scratch);
    const int per = blockDim.x / tpr, weight_floats = a.weight ? (a.cols + 3) / 4 * 4 : 0;
    const int64_t step = static_cast<int64_t>(gridDim.x) * per;
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    const bool weighed = a.weight != nullptr;
    float dw[NV][EPV] = {};
    int64_t first = static_cast<int64_t>(blockIdx.x) * per;
    Slot<T, EPV> t[NV], dy[NV], dt[NV];
    const uint32_t room = smem_addr(staged + weight_floats) + 16u * threadIdx.x;
    const auto place = [&](int stage, int which, int k) {
        return room + 16u * blockDim.x * static_cast<uint32_t>((stage * 3 + which) * NV + k);
    };
    const auto load = [&](int64_t n, int stage) {
        if constexpr (AHEAD == 0) {
            load_row(t, a.total, a.total_at, a.inner, a.rows, n, gr, a.cols);
            load_row(dy, a.dy, a.dy_at, a.inner, a.rows, n, gr, a.cols);
            if (a.dtotal) load_row(dt, a.dtotal, a.dtotal_at, a.inner, a.rows, n, gr, a.cols);
        } else {
            if (n < a.rows) {
                const Place at = row_place(a.inner, a.rows, n);
                const T *rows[3] = {static_cast<const T *>(a.total) + offset_at(a.total_at, at),
                                    static_cast<const T *>(a.dy) + offset_at(a.dy_at, at),
                                    a.dtotal ? static_cast<const T *>(a.dtotal) + offset_at(a.dtotal_at, at) : nullptr};
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int c = (gr.lane + k * gr.tpr) * EPV;
#pragma unroll
                    for (int w = 0; w < 3; ++w)
                        if (rows[w] && c < a.cols) copy_async(place(stage, w, k), rows[w] + c);
                }
            }
            copy_commit();
        }
    };
    const auto rstd_of = [&](int64_t n) { return n < a.rows ? __ldg(a.rstd + n) : 0.f; };
    constexpr int kDeep = AHEAD ? AHEAD : 1;
#pragma unroll
    for (int i = 0; i < kDeep; ++i) load(first + gr.g + i * step, i);
    float rstd_next = rstd_of(first + gr.g);
    stage_weight(staged, a.weight, a.weight_format, a.cols);
    __syncthreads();
    int stage = 0;
    for (; first < a.rows; first += step) {
        const int64_t n = first + gr.g;
        const bool live = n < a.rows;
        const float rstd = rstd_next;
        if constexpr (AHEAD > 0) {
            copy_wait<kDeep - 1>();
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                t[k].raw = lds128(place(stage, 0, k));
                dy[k].raw = lds128(place(stage, 1, k));
                if (a.dtotal) dt[k].raw = lds128(place(stage, 2, k));
            }
        }
        rstd_next = rstd_of(n + step);
        float sum[1] = {0.f};
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (gr.lane + k * tpr) * EPV;
            if (c >= a.cols) continue;
            float f[EPV], g[EPV], w[EPV];
            t[k].get(f);
            dy[k].get(g);
            weight_at<EPV>(staged, weighed, c, w);
#pragma unroll
            for (int e = 0; e < EPV; ++e) {
                if (weighed && live) dw[k][e] = fmaf(g[e], f[e] * rstd, dw[k][e]);
                sum[0] = fmaf(g[e] * w[e], f[e], sum[0]);
            }
        }
        if constexpr (AHEAD > 0) {
            load(n + kDeep * step, stage);         // (what was in its place is in registers)
            stage = stage + 1 == kDeep ? 0 : stage + 1;
        }
        row_sum(sum, gr);
        const float along = sum[0] * inv_cols * rstd * rstd;
        Slot<T, EPV> o[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (gr.lane + k * tpr) * EPV;
            if (c >= a.cols) continue;
            float f[EPV], g[EPV], r[EPV], w[EPV];
            t[k].get(f);
            dy[k].get(g);
            weight_at<EPV>(staged, weighed, c, w);
#pragma unroll
            for (int e = 0; e < EPV; ++e) r[e] = 0.f;
            if (a.dtotal) dt[k].get(r);
#pragma unroll
            for (int e = 0; e < EPV; ++e) f[e] = fmaf(rstd, fmaf(-f[e], along, g[e] * w[e]), r[e]);
            o[k].set(f);
        }
        if constexpr (AHEAD == 0) load(n + step, 0);
        T *dx = live ? static_cast<T *>(a.dx) + row_offset(a.dx_at, a.inner, a.rows, n) : nullptr;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (gr.lane + k * tpr) * EPV;
            if (live && c < a.cols) o[k].store(dx + c);
        }
    }
    if constexpr (AHEAD > 0) copy_wait<0>();
    if (!weighed) return;
    float *out = a.partial + static_cast<int64_t>(blockIdx.x) * a.cols;
    if (per == 1) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (gr.lane + k * tpr) * EPV;
            if (c >= a.cols) continue;
#pragma unroll
            for (int e = 0; e < EPV; ++e) out[c + e] = dw[k][e];
        }
        return;
    }
    float *columns = staged + weight_floats + AHEAD * 3 * NV * 4 * blockDim.x;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = (gr.lane + k * tpr) * EPV;
        if (c >= a.cols) continue;
#pragma unroll
        for (int e = 0; e < EPV; ++e) columns[gr.g * a.cols + c + e] = dw[k][e];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
        float v = 0.f;
        for (int g = 0; g < per; ++g) v += columns[g * a.cols + c];
        out[c] = v;
    }
}

// ---- half-type rows that begin at any element, alike in all tensors ------------------
// (Odd widths of contiguous tensors.)  A row is peeled: up to 7 elements to the first 16-byte
// boundary, whole vectors, up to 7 elements behind them; the first ones and the last ones are
// single elements of the row's first lanes.  Which column a thread has changes from row to row,
// so the weight and, backward, its gradient's sums are in shared memory, a place left free behind
// every eight: eight neighbours a lane then lie in different banks.
constexpr int kEdge = 14;

__device__ __forceinline__ int padded(int c) { return c + (c >> 3); }

struct Peel {
    int head, vectors, edge;          // edge: this lane's single element, or -1
    __device__ __forceinline__ Peel(uintptr_t row, int cols, int lane)
    {
        head = static_cast<int>((8 - (row >> 1 & 7)) & 7);
        vectors = (cols - head) >> 3;
        const int tail = head + 8 * vectors;
        const int c = lane < head ? lane : tail + lane - head;
        edge = lane < kEdge && c < cols ? c : -1;
    }
};

__device__ __forceinline__ void stage_padded(float *to, const void *weight, int format, int cols)
{
    for (int c = threadIdx.x; c < cols; c += blockDim.x) {
        float w[1] = {1.0f};
        if (weight) load_params<1>(weight, format, c, w);
        to[padded(c)] = w[0];
    }
}

template <typename T, int NV>
__global__ void __launch_bounds__(512, 2) rms_peeled_kernel(const __grid_constant__ RmsArgs a, int tpr)
{
    __shared__ float scratch[kMaxGroups][2][32][2];
    extern __shared__ __align__(16) float staged[];
    tc::griddep_wait();
    if (threadIdx.x == 0) tc::griddep_launch_dependents();
    Group gr = group_of(tpr, scratch);
    const int per = blockDim.x / tpr;
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    stage_padded(staged, a.weight, a.weight_format, a.cols);
    __syncthreads();
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * per; first < a.rows; first += static_cast<int64_t>(gridDim.x) * per) {
        const int64_t n = first + gr.g;
        const bool live = n < a.rows;
        const Place at = row_place(a.inner, a.rows, live ? n : 0);
        const T *x = static_cast<const T *>(a.x) + offset_at(a.x_at, at);
        const T *r = a.residual ? static_cast<const T *>(a.residual) + offset_at(a.residual_at, at) : nullptr;
        T *total = a.residual ? static_cast<T *>(a.total) + offset_at(a.total_at, at) : nullptr;
        const Peel p(reinterpret_cast<uintptr_t>(x), a.cols, gr.lane);
        const int edge = live ? p.edge : -1;
        Slot<T, 8> t[NV], s[NV];
        float one = 0.f, sum = 0.f, most = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int j = gr.lane + k * tpr;
            t[k].clear();
            s[k].clear();
            if (live && j < p.vectors) {
                t[k].load(x + p.head + 8 * j);
                if (r) s[k].load(r + p.head + 8 * j);
            }
        }
        if (edge >= 0) {
            one = to_float(x[edge]);
            if (r) {
                const T v = from_float<T>(one + to_float(r[edge]));
                total[edge] = v;
                one = to_float(v);
            }
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int j = gr.lane + k * tpr, c = p.head + 8 * j;
            float f[8], g[8];
            t[k].get(f);
            if (r) {
                s[k].get(g);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] += g[e];
                t[k].set(f);
                if (live && j < p.vectors) t[k].store(total + c);
                t[k].get(f);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fmaf(f[e], f[e], sum);
            if (a.scales && live && j < p.vectors)
#pragma unroll
                for (int e = 0; e < 8; ++e) most = max_nan(most, fabsf(f[e] * staged[padded(c + e)]));
        }
        sum = fmaf(one, one, sum);
        if (a.scales && edge >= 0) most = max_nan(most, fabsf(one * staged[padded(edge)]));
        row_sum_max(sum, most, gr);
        const float rstd = 1.0f / sqrtf(fmaf(sum, inv_cols, a.eps));
        const RowScale o(most, rstd);
        if (live && gr.lane == 0) {
            if (a.rstd) a.rstd[n] = rstd;
            if (a.scales) a.scales[n] = o.scale;
        }
        const int64_t to = offset_at(a.y_at, at);
        const auto put = [&](int c, float v) {
            const float w = staged[padded(c)];
            if (a.scales)
                static_cast<uint8_t *>(a.y)[to + c] = static_cast<uint8_t>(e4m3_pair(o.of(v * w), 0.f));
            else
                static_cast<T *>(a.y)[to + c] = from_float<T>(v * rstd * w);
        };
        if (edge >= 0) put(edge, one);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int j = gr.lane + k * tpr, c = p.head + 8 * j;
            if (!live || j >= p.vectors) continue;
            float f[8];
            t[k].get(f);
            if (a.scales) {
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = o.of(f[e] * staged[padded(c + e)]);
                store_e4m3<8>(static_cast<uint8_t *>(a.y) + to + c, f);
            } else {
                Slot<T, 8> v;
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = f[e] * rstd * staged[padded(c + e)];
                v.set(f);
                v.store(static_cast<T *>(a.y) + to + c);
            }
        }
    }
}

// (NV = 4, 2300 rows of 12001: 111 us in the 64 registers that two CTAs leave, 94 with one)
template <typename T, int NV>
__global__ void __launch_bounds__(512, NV == 2 ? 2 : 1) rms_peeled_grad_kernel(const __grid_constant__ RmsGradArgs a, int tpr)
{
    __shared__ float scratch[kMaxGroups][2][32][2];
    extern __shared__ __align__(16) float staged[];       // the weight, then [groups] sums of its gradient
    tc::griddep_wait();
    if (threadIdx.x == 0) tc::griddep_launch_dependents();
    Group gr = group_of(tpr, scratch);
    const int per = blockDim.x / tpr, width = padded(a.cols) + 1;
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    float *dw = staged + width * (1 + gr.g);
    stage_padded(staged, a.weight, a.weight_format, a.cols);
    if (a.weight)
        for (int c = threadIdx.x; c < width * per; c += blockDim.x) staged[width + c] = 0.f;
    __syncthreads();
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * per; first < a.rows; first += static_cast<int64_t>(gridDim.x) * per) {
        const int64_t n = first + gr.g;
        const bool live = n < a.rows;
        const Place at = row_place(a.inner, a.rows, live ? n : 0);
        const T *pt = static_cast<const T *>(a.total) + offset_at(a.total_at, at);
        const T *pd = static_cast<const T *>(a.dy) + offset_at(a.dy_at, at);
        const T *pr = a.dtotal ? static_cast<const T *>(a.dtotal) + offset_at(a.dtotal_at, at) : nullptr;
        const Peel p(reinterpret_cast<uintptr_t>(pt), a.cols, gr.lane);
        const int edge = live ? p.edge : -1;
        const float rstd = live ? __ldg(a.rstd + n) : 0.f;
        Slot<T, 8> t[NV], dy[NV], dt[NV];
        float one = 0.f, grad = 0.f, back = 0.f, sum[1] = {0.f};
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int j = gr.lane + k * tpr, c = p.head + 8 * j;
            t[k].clear();
            dy[k].clear();
            dt[k].clear();
            if (live && j < p.vectors) {
                t[k].load(pt + c);
                dy[k].load(pd + c);
                if (pr) dt[k].load(pr + c);
            }
        }
        if (edge >= 0) {
            one = to_float(pt[edge]);
            grad = to_float(pd[edge]);
            if (pr) back = to_float(pr[edge]);
        }
        // (Sums of a column are added to by one thread a row; the row's threads meet in its
        // reduction before the next row, whose columns are dealt out anew.)
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int j = gr.lane + k * tpr, c = p.head + 8 * j;
            if (!live || j >= p.vectors) continue;
            float f[8], g[8];
            t[k].get(f);
            dy[k].get(g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (a.weight) dw[padded(c + e)] += g[e] * (f[e] * rstd);
                sum[0] = fmaf(g[e] * staged[padded(c + e)], f[e], sum[0]);
            }
        }
        if (edge >= 0) {
            if (a.weight) dw[padded(edge)] += grad * (one * rstd);
            grad *= staged[padded(edge)];
            sum[0] = fmaf(grad, one, sum[0]);
        }
        row_sum(sum, gr);
        if (gr.tpr <= 32) __syncwarp();
        const float along = sum[0] * inv_cols * rstd * rstd;
        T *dx = static_cast<T *>(a.dx) + offset_at(a.dx_at, at);
        if (edge >= 0) dx[edge] = from_float<T>(fmaf(rstd, fmaf(-one, along, grad), back));
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int j = gr.lane + k * tpr, c = p.head + 8 * j;
            if (!live || j >= p.vectors) continue;
            float f[8], g[8], r[8];
            t[k].get(f);
            dy[k].get(g);
            dt[k].get(r);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = fmaf(rstd, fmaf(-f[e], along, g[e] * staged[padded(c + e)]), r[e]);
            Slot<T, 8> o;
            o.set(f);
            o.store(dx + c);
        }
    }
    if (!a.weight) return;
    __syncthreads();
    float *out = a.partial + static_cast<int64_t>(blockIdx.x) * a.cols;
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
        float v = 0.f;
        for (int g = 0; g < per; ++g) v += staged[width * (1 + g) + padded(c)];
        out[c] = v;
    }
}

// dweight: the CTAs' rows of partial sums, 32 columns a CTA, 32 warps taking every 32nd
// row, and those sums in order.  (8 warps took 10 us for 608 rows.)
__global__ void __launch_bounds__(1024) rms_columns_kernel(const __grid_constant__ RmsGradArgs a, int blocks)
{
    __shared__ float part[32][33];
    tc::griddep_wait();
    if (threadIdx.x == 0) tc::griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float v = 0.f;
    if (c < a.cols)
#pragma unroll 10
        for (int b = warp; b < blocks; b += 32) v += a.partial[static_cast<int64_t>(b) * a.cols + c];
    part[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && c < a.cols) {
        v = 0.f;
#pragma unroll
        for (int w = 0; w < 32; ++w) v += part[w][lane];
        store_param(a.dweight, a.weight_format, c, v);
    }
}

// Slots of a thread, threads of a row and of a CTA.
struct Shape {
    int nv, tpr, threads;
    int rows = 1;                 // of a group at a time
};

int row_threads(int slots, int nv)
{
    const int need = (slots + nv - 1) / nv;
    if (need <= 32) {
        int t = 1;
        while (t < need) t *= 2;
        return t;
    }
    return (need + 31) / 32 * 32;
}

// (one slot a thread where the rows are few: 1 x 6144 11.4 us replayed, 15.5 with two;
// where they are many two keep more rows on an SM: 4608 x 6144 58 us, 73 with one)
Shape shape_of(int slots, bool vec, int64_t rows, int sm_count)
{
    Shape s;
    const int one = rows <= sm_count ? 1024 : 512;
    if (vec)
        s.nv = slots <= one ? 1 : slots <= 1024 ? 2 : 4;
    else
        s.nv = slots <= 4096 ? 4 : 16;
    s.tpr = row_threads(slots, s.nv);
    if (vec && s.tpr <= 32 && s.nv == 1 && rows > 256 / s.tpr * sm_count) s.rows = kShortRows;
    s.threads = s.tpr >= 256 ? s.tpr : s.tpr * std::max(1, 256 / s.tpr);
    return s;
}

bool vectors(int cols, int epv, std::initializer_list<std::pair<const void *, const RowsAt *>> rows)
{
    if (cols % epv) return false;
    for (const auto &r : rows)
        if (r.first && (reinterpret_cast<uintptr_t>(r.first) % 16 || r.second->outer % epv || r.second->stride % epv)) return false;
    return true;
}

// Whether all tensors' rows lie alike to 16 bytes (`y`: a row of bytes, eight of which go
// with 16 of the others').
bool alike(std::initializer_list<std::pair<const void *, const RowsAt *>> rows, const void *y, const RowsAt *y_at)
{
    const void *first = nullptr;
    const RowsAt *at = nullptr;
    for (const auto &r : rows) {
        if (!r.first) continue;
        if (!first) first = r.first, at = r.second;
        if ((reinterpret_cast<uintptr_t>(r.first) - reinterpret_cast<uintptr_t>(first)) % 16 ||
            (r.second->outer - at->outer) % 8 || (r.second->stride - at->stride) % 8)
            return false;
    }
    return !y || ((reinterpret_cast<uintptr_t>(y) - reinterpret_cast<uintptr_t>(first) / 2) % 8 == 0 &&
                  (y_at->outer - at->outer) % 8 == 0 && (y_at->stride - at->stride) % 8 == 0);
}

// Peeled rows: two vectors a thread (4608 x 6143 backward 73 us, 100 with four), four where two
// would take more than 512 threads a row.
Shape peeled_shape(int cols)
{
    Shape s;
    const int slots = cols / 8;
    s.nv = slots <= 1024 ? 2 : 4;
    s.tpr = std::max(16, row_threads(slots, s.nv));
    s.threads = s.tpr >= 256 ? s.tpr : s.tpr * std::max(1, 256 / s.tpr);
    return s;
}

// Fewer columns than this take single elements (forward, 300000 x 65: 88 us, 138 so;
// 500000 x 33: 140 us peeled, 115 so).
constexpr int kPeeledCols = 64;

template <auto KERNEL, typename Args>
cudaError_t run(const Args &a, const Shape &d, int64_t most, size_t smem, int sm_count, cudaStream_t s, int *blocks)
{
    // (weights of up to 16384 columns and the sums of a few groups, or two rows on their way)
    static std::atomic<uint64_t> done{0};
    cudaError_t e = smem > 40 * 1024 ? allow_shared(reinterpret_cast<const void *>(KERNEL), 160 * 1024, done) : cudaSuccess;
    if (e != cudaSuccess) return e;
    // as many CTAs as are on the SMs at once: each goes through several rows
    const int64_t per = d.threads / d.tpr * d.rows, all = std::min((a.rows + per - 1) / per, most);
    int fit = 1;
    if (all > sm_count) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, KERNEL, d.threads, smem);
    if (e != cudaSuccess) return e;
    *blocks = static_cast<int>(std::min<int64_t>(all, static_cast<int64_t>(std::max(1, fit)) * sm_count));
    return tc::launch_pdl(KERNEL, dim3(static_cast<unsigned>(*blocks)), dim3(d.threads), smem, s, a, d.tpr);
}

template <typename T>
cudaError_t forward(const RmsArgs &a, int sm_count, cudaStream_t s)
{
    constexpr int EPV = 16 / sizeof(T);
    // (a row of bytes takes stores of EPV bytes)
    const bool y_ok = !a.scales || reinterpret_cast<uintptr_t>(a.y) % EPV == 0;
    const bool vec = y_ok && vectors(a.cols, EPV, {{a.x, &a.x_at}, {a.residual, &a.residual_at}, {a.total, &a.total_at},
                                                   {a.scales ? nullptr : a.y, &a.y_at}}) &&
                     a.y_at.outer % EPV == 0 && a.y_at.stride % EPV == 0;
    if constexpr (sizeof(T) == 2) {
        if (!vec && a.cols >= kPeeledCols &&
            alike({{a.x, &a.x_at}, {a.residual, &a.residual_at}, {a.total, &a.total_at}, {a.scales ? nullptr : a.y, &a.y_at}},
                  a.scales ? a.y : nullptr, &a.y_at)) {
            const Shape d = peeled_shape(a.cols);
            const size_t smem = 4u * (static_cast<size_t>(a.cols) + static_cast<size_t>(a.cols) / 8 + 1);
            int blocks;
            if (d.nv == 2) return run<rms_peeled_kernel<T, 2>>(a, d, INT32_MAX, smem, sm_count, s, &blocks);
            return run<rms_peeled_kernel<T, 4>>(a, d, INT32_MAX, smem, sm_count, s, &blocks);
        }
    }
    const Shape d = shape_of(vec ? a.cols / EPV : a.cols, vec, a.rows, sm_count);
    const size_t smem = a.weight ? 4u * static_cast<size_t>(a.cols) : 0;
    int blocks;
    if (d.rows > 1) return run<rms_short_kernel<T, EPV>>(a, d, INT32_MAX, smem, sm_count, s, &blocks);
    if (vec && d.nv == 1) return run<rms_kernel<T, EPV, 1, 1024, 1>>(a, d, INT32_MAX, smem, sm_count, s, &blocks);
    if (vec && d.nv == 2 && d.threads <= 384) return run<rms_kernel<T, EPV, 2, 384, 3>>(a, d, INT32_MAX, smem, sm_count, s, &blocks);
    if (vec && d.nv == 2) return run<rms_kernel<T, EPV, 2, 512, 1>>(a, d, INT32_MAX, smem, sm_count, s, &blocks);
    if (vec) return run<rms_kernel<T, EPV, 4, (EPV == 8 ? 512 : 1024), 1>>(a, d, INT32_MAX, smem, sm_count, s, &blocks);
    if (d.nv == 4) return run<rms_kernel<T, 1, 4, 1024, 1>>(a, d, INT32_MAX, smem, sm_count, s, &blocks);
    return run<rms_kernel<T, 1, 16, 1024, 1>>(a, d, INT32_MAX, smem, sm_count, s, &blocks);
}

template <typename T>
cudaError_t backward(const RmsGradArgs &a, int sm_count, cudaStream_t s, int *blocks)
{
    constexpr int EPV = 16 / sizeof(T);
    const bool vec = vectors(a.cols, EPV, {{a.total, &a.total_at}, {a.dy, &a.dy_at}, {a.dtotal, &a.dtotal_at}, {a.dx, &a.dx_at}});
    if constexpr (sizeof(T) == 2) {
        if (!vec && a.cols >= kPeeledCols &&
            alike({{a.total, &a.total_at}, {a.dy, &a.dy_at}, {a.dtotal, &a.dtotal_at}, {a.dx, &a.dx_at}}, nullptr, nullptr)) {
            const Shape d = peeled_shape(a.cols);
            const size_t width = static_cast<size_t>(a.cols) + static_cast<size_t>(a.cols) / 8 + 1;
            const size_t smem = 4u * width * (a.weight ? 1 + static_cast<size_t>(d.threads / d.tpr) : 1);
            const int64_t most = rms_norm_blocks(a.rows, sm_count);
            if (d.nv == 2) return run<rms_peeled_grad_kernel<T, 2>>(a, d, most, smem, sm_count, s, blocks);
            return run<rms_peeled_grad_kernel<T, 4>>(a, d, most, smem, sm_count, s, blocks);
        }
    }
    const Shape d = shape_of(vec ? a.cols / EPV : a.cols, vec, a.rows, sm_count);
    const size_t per = static_cast<size_t>(d.threads / d.tpr), cols = static_cast<size_t>(a.cols);
    const auto smem = [&](int ahead) {
        return (a.weight ? 4u * ((cols + 3) / 4 * 4 + (per > 1 ? per * cols : 0)) : 0) +
               16u * static_cast<size_t>(3 * ahead * d.nv * d.threads);
    };
    const int64_t most = rms_norm_blocks(a.rows, sm_count);
    if (d.rows > 1) return run<rms_short_grad_kernel<T, EPV>>(a, d, most, smem(0), sm_count, s, blocks);
    if (vec && d.nv == 1) return run<rms_grad_kernel<T, EPV, 1, 1024, 1, 1>>(a, d, most, smem(1), sm_count, s, blocks);
    if (vec && d.nv == 2 && d.threads <= 384)
        return run<rms_grad_kernel<T, EPV, 2, 384, 2, 1>>(a, d, most, smem(1), sm_count, s, blocks);
    if (vec && d.nv == 2) return run<rms_grad_kernel<T, EPV, 2, 512, 1, 2>>(a, d, most, smem(2), sm_count, s, blocks);
    if (vec) return run<rms_grad_kernel<T, EPV, 4, (EPV == 8 ? 512 : 1024), 1, 0>>(a, d, most, smem(0), sm_count, s, blocks);
    if (d.nv == 4) return run<rms_grad_kernel<T, 1, 4, 1024, 1, 0>>(a, d, most, smem(0), sm_count, s, blocks);
    return run<rms_grad_kernel<T, 1, 16, 1024, 1, 0>>(a, d, most, smem(0), sm_count, s, blocks);
}

}  // namespace

int rms_norm_blocks(int64_t rows, int sm_count) { return static_cast<int>(std::min<int64_t>(rows, 4 * sm_count)); }

cudaError_t launch_rms_norm(const RmsArgs &a, int sm_count, cudaStream_t s)
{
    if (a.format == GN_FORMAT_BF16) return forward<__nv_bfloat16>(a, sm_count, s);
    if (a.format == GN_FORMAT_FP16) return forward<__half>(a, sm_count, s);
    return forward<float>(a, sm_count, s);
}

cudaError_t launch_rms_norm_backward(const RmsGradArgs &a, int sm_count, cudaStream_t s, int *launches)
{
    cudaError_t e;
    int blocks = 0;
    if (a.format == GN_FORMAT_BF16)
        e = backward<__nv_bfloat16>(a, sm_count, s, &blocks);
    else if (a.format == GN_FORMAT_FP16)
        e = backward<__half>(a, sm_count, s, &blocks);
    else
        e = backward<float>(a, sm_count, s, &blocks);
    if (e != cudaSuccess) return e;
    *launches = 1;
    if (!a.weight) return e;
    e = tc::launch_pdl(rms_columns_kernel, dim3((a.cols + 31) / 32), dim3(1024), 0, s, a, blocks);
    if (e == cudaSuccess) *launches = 2;
    return e;
}

}  // namespace gn
