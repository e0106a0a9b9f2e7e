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
#include <cstdint>

#include "block_internal.h"
#include "block_math.cuh"
#include "gn_ptx.cuh"
#include "norm_common.cuh"
#include "tc_common.cuh"

namespace gn {
namespace {

using namespace norm;

constexpr float kLeastMagnitude = 1e-30f;    // of a row in 8 bits: below it the scale is 0

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

// The largest of a group's values (NaN if any is).
__device__ __forceinline__ float row_max(float v, Group &gr)
{
    const int within = min(gr.tpr, 32) >> 1;
    for (int o = within; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (gr.tpr <= 32) return v;
    const int warp = gr.lane >> 5, lane = threadIdx.x & 31, warps = gr.tpr >> 5;
    float(*s)[2] = gr.scratch[gr.turn];
    gr.turn ^= 1;
    if (lane == 0) s[warp][0] = v;
    named_sync(1 + gr.g, gr.tpr);
    v = lane < warps ? s[lane][0] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
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

template <typename T, int EPV, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) rms_kernel(const __grid_constant__ RmsArgs a, int tpr)
{
    __shared__ float scratch[kMaxGroups][2][32][2];
    tc::griddep_wait();
    if (threadIdx.x == 0) tc::griddep_launch_dependents();
    Group gr = group_of(tpr, scratch);
    const int per = blockDim.x / tpr;
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    // (the rows of a CTA's groups end together: a warp's lanes shuffle as one)
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * per; first < a.rows; first += static_cast<int64_t>(gridDim.x) * per) {
        const int64_t n = first + gr.g;
        const bool live = n < a.rows;
        Slot<T, EPV> t[NV];
        float sum[1] = {0.f};
        const T *x = live ? static_cast<const T *>(a.x) + row_offset(a.x_at, a.inner, a.rows, n) : nullptr;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (gr.lane + k * tpr) * EPV;
            if (live && c < a.cols)
                t[k].load(x + c);
            else
                t[k].clear();
        }
        if (a.residual) {
            Slot<T, EPV> r[NV];
            const T *p = live ? static_cast<const T *>(a.residual) + row_offset(a.residual_at, a.inner, a.rows, n) : nullptr;
            T *to = live ? static_cast<T *>(a.total) + row_offset(a.total_at, a.inner, a.rows, n) : nullptr;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (gr.lane + k * tpr) * EPV;
                if (live && c < a.cols)
                    r[k].load(p + c);
                else
                    r[k].clear();
            }
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (gr.lane + k * tpr) * EPV;
                float f[EPV], g[EPV];
                t[k].get(f);
                r[k].get(g);
#pragma unroll
                for (int e = 0; e < EPV; ++e) f[e] += g[e];
                t[k].set(f);
                if (live && c < a.cols) t[k].store(to + c);
            }
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float f[EPV];
            t[k].get(f);
#pragma unroll
            for (int e = 0; e < EPV; ++e) sum[0] = fmaf(f[e], f[e], sum[0]);
        }
        row_sum(sum, gr);
        const float rstd = 1.0f / sqrtf(fmaf(sum[0], inv_cols, a.eps));
        if (live && gr.lane == 0 && a.rstd) a.rstd[n] = rstd;
        const auto value = [&](int k, int c, float (&f)[EPV]) {
            t[k].get(f);
            float w[EPV];
            if (a.weight) load_params<EPV>(a.weight, a.weight_format, c, w);
#pragma unroll
            for (int e = 0; e < EPV; ++e) f[e] = f[e] * rstd * (a.weight ? w[e] : 1.0f);
        };
        if (!a.scales) {
            T *y = live ? static_cast<T *>(a.y) + row_offset(a.y_at, a.inner, a.rows, n) : nullptr;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (gr.lane + k * tpr) * EPV;
                if (!live || c >= a.cols) continue;
                float f[EPV];
                value(k, c, f);
                Slot<T, EPV> o;
                o.set(f);
                o.store(y + c);
            }
            continue;
        }
        float most = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (gr.lane + k * tpr) * EPV;
            if (!live || c >= a.cols) continue;
            float f[EPV];
            value(k, c, f);
#pragma unroll
            for (int e = 0; e < EPV; ++e) most = max_nan(most, fabsf(f[e]));
        }
        most = row_max(most, gr);
        const bool none = most < kLeastMagnitude;
        const float by = none ? 0.f : 448.0f / most;
        if (live && gr.lane == 0) a.scales[n] = none ? 0.f : most / 448.0f;
        uint8_t *y = live ? static_cast<uint8_t *>(a.y) + row_offset(a.y_at, a.inner, a.rows, n) : nullptr;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (gr.lane + k * tpr) * EPV;
            if (!live || c >= a.cols) continue;
            float f[EPV];
            value(k, c, f);
#pragma unroll
            for (int e = 0; e < EPV; ++e) f[e] *= by;
            store_e4m3<EPV>(y + c, f);
        }
    }
}

template <typename T, int EPV, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) rms_grad_kernel(const __grid_constant__ RmsGradArgs a, int tpr)
{
    __shared__ float scratch[kMaxGroups][2][32][2];
    extern __shared__ float columns[];       // [groups][cols] where a CTA has several
    tc::griddep_wait();
    if (threadIdx.x == 0) tc::griddep_launch_dependents();
    Group gr = group_of(tpr, scratch);
    const int per = blockDim.x / tpr;
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    float dw[NV][EPV] = {};
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * per; first < a.rows; first += static_cast<int64_t>(gridDim.x) * per) {
        const int64_t n = first + gr.g;
        const bool live = n < a.rows;
        Slot<T, EPV> t[NV], dy[NV], dt[NV];
        const T *pt = live ? static_cast<const T *>(a.total) + row_offset(a.total_at, a.inner, a.rows, n) : nullptr;
        const T *pd = live ? static_cast<const T *>(a.dy) + row_offset(a.dy_at, a.inner, a.rows, n) : nullptr;
        const T *pr = live && a.dtotal ? static_cast<const T *>(a.dtotal) + row_offset(a.dtotal_at, a.inner, a.rows, n) : nullptr;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (gr.lane + k * tpr) * EPV;
            t[k].clear();
            dy[k].clear();
            dt[k].clear();
            if (live && c < a.cols) {
                t[k].load(pt + c);
                dy[k].load(pd + c);
                if (pr) dt[k].load(pr + c);
            }
        }
        const float rstd = live ? __ldg(a.rstd + n) : 0.f;
        float sum[1] = {0.f};
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (gr.lane + k * tpr) * EPV;
            float f[EPV], g[EPV], w[EPV];
            t[k].get(f);
            dy[k].get(g);
            if (a.weight && c < a.cols) {
                load_params<EPV>(a.weight, a.weight_format, c, w);
#pragma unroll
                for (int e = 0; e < EPV; ++e) {
                    if (live) dw[k][e] = fmaf(g[e], f[e] * rstd, dw[k][e]);
                    g[e] *= w[e];
                }
            }
#pragma unroll
            for (int e = 0; e < EPV; ++e) sum[0] = fmaf(g[e], f[e], sum[0]);
        }
        row_sum(sum, gr);
        // (the factors of t in this order: rstd^2 may leave fp32's range where the product does not)
        const float along = sum[0] * inv_cols * rstd * rstd;
        T *dx = live ? static_cast<T *>(a.dx) + row_offset(a.dx_at, a.inner, a.rows, n) : nullptr;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (gr.lane + k * tpr) * EPV;
            if (!live || c >= a.cols) continue;
            float f[EPV], g[EPV], r[EPV], w[EPV];
            t[k].get(f);
            dy[k].get(g);
            dt[k].get(r);
            if (a.weight) load_params<EPV>(a.weight, a.weight_format, c, w);
#pragma unroll
            for (int e = 0; e < EPV; ++e)
                f[e] = fmaf(rstd, fmaf(-f[e], along, a.weight ? g[e] * w[e] : g[e]), r[e]);
            Slot<T, EPV> o;
            o.set(f);
            o.store(dx + c);
        }
    }
    if (!a.weight) return;
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

// dweight: the CTAs' rows of partial sums, 32 columns a CTA, 8 warps taking every
// eighth row, and those eight sums in order.
__global__ void __launch_bounds__(256) rms_columns_kernel(const __grid_constant__ RmsGradArgs a, int blocks)
{
    __shared__ float part[8][33];
    tc::griddep_wait();
    if (threadIdx.x == 0) tc::griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float v = 0.f;
    if (c < a.cols)
#pragma unroll 8
        for (int b = warp; b < blocks; b += 8) v += a.partial[static_cast<int64_t>(b) * a.cols + c];
    part[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && c < a.cols) {
        v = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) v += part[w][lane];
        store_param(a.dweight, a.weight_format, c, v);
    }
}

// Slots of a thread, threads of a row and of a CTA.
struct Shape {
    int nv, tpr, threads;
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

Shape shape_of(int slots, bool vec)
{
    Shape s;
    if (vec)
        s.nv = slots <= 512 ? 1 : slots <= 1024 ? 2 : 4;
    else
        s.nv = slots <= 4096 ? 4 : 16;
    s.tpr = row_threads(slots, s.nv);
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

template <typename T>
cudaError_t forward(const RmsArgs &a, int sm_count, cudaStream_t s)
{
    constexpr int EPV = 16 / sizeof(T);
    // (a row of bytes takes stores of EPV bytes)
    const bool y_ok = !a.scales || reinterpret_cast<uintptr_t>(a.y) % EPV == 0;
    const bool vec = y_ok && vectors(a.cols, EPV, {{a.x, &a.x_at}, {a.residual, &a.residual_at}, {a.total, &a.total_at},
                                                   {a.scales ? nullptr : a.y, &a.y_at}}) &&
                     a.y_at.outer % EPV == 0 && a.y_at.stride % EPV == 0;
    const Shape d = shape_of(vec ? a.cols / EPV : a.cols, vec);
    const int64_t per = d.threads / d.tpr, fit = 2048 / d.threads;
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>((a.rows + per - 1) / per, fit * sm_count))), block(d.threads);
    if (vec && d.nv == 1) return tc::launch_pdl(rms_kernel<T, EPV, 1, 512>, grid, block, 0, s, a, d.tpr);
    if (vec && d.nv == 2) return tc::launch_pdl(rms_kernel<T, EPV, 2, 512>, grid, block, 0, s, a, d.tpr);
    if (vec) return tc::launch_pdl(rms_kernel<T, EPV, 4, EPV == 8 ? 512 : 1024>, grid, block, 0, s, a, d.tpr);
    if (d.nv == 4) return tc::launch_pdl(rms_kernel<T, 1, 4, 1024>, grid, block, 0, s, a, d.tpr);
    return tc::launch_pdl(rms_kernel<T, 1, 16, 1024>, grid, block, 0, s, a, d.tpr);
}

template <typename T>
cudaError_t backward(const RmsGradArgs &a, int sm_count, cudaStream_t s, int *blocks)
{
    constexpr int EPV = 16 / sizeof(T);
    const bool vec = vectors(a.cols, EPV, {{a.total, &a.total_at}, {a.dy, &a.dy_at}, {a.dtotal, &a.dtotal_at}, {a.dx, &a.dx_at}});
    const Shape d = shape_of(vec ? a.cols / EPV : a.cols, vec);
    const int64_t per = d.threads / d.tpr;
    *blocks = static_cast<int>(std::min<int64_t>((a.rows + per - 1) / per, rms_norm_blocks(a.rows, sm_count)));
    const dim3 grid(static_cast<unsigned>(*blocks)), block(d.threads);
    const size_t smem = a.weight && per > 1 ? 4u * static_cast<size_t>(per) * static_cast<size_t>(a.cols) : 0;
    if (vec && d.nv == 1) return tc::launch_pdl(rms_grad_kernel<T, EPV, 1, 512>, grid, block, smem, s, a, d.tpr);
    if (vec && d.nv == 2) return tc::launch_pdl(rms_grad_kernel<T, EPV, 2, 512>, grid, block, smem, s, a, d.tpr);
    if (vec) return tc::launch_pdl(rms_grad_kernel<T, EPV, 4, EPV == 8 ? 512 : 1024>, grid, block, smem, s, a, d.tpr);
    if (d.nv == 4) return tc::launch_pdl(rms_grad_kernel<T, 1, 4, 1024>, grid, block, smem, s, a, d.tpr);
    return tc::launch_pdl(rms_grad_kernel<T, 1, 16, 1024>, grid, block, smem, s, a, d.tpr);
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
    e = tc::launch_pdl(rms_columns_kernel, dim3((a.cols + 31) / 32), dim3(256), 0, s, a, blocks);
    if (e == cudaSuccess) *launches = 2;
    return e;
}

}  // namespace gn
