// norm_kernels.cu -- sm_103a kernels of layer norm over the last axis and its
// backward pass.
//
//   forward   mean = sum(x) / C, rstd = 1 / sqrt(sum((x - mean)^2) / C + eps),
//             y = (x - mean) rstd w + b
//   backward  with h = (x - mean) rstd and g = dy w,
//             dx = rstd (g - sum(g) / C - h sum(g h) / C),
//             dw = sum over rows of dy h,  db = sum over rows of dy
//
// A row is held in the registers of `tpr` threads (NV slots each of EPV
// consecutive elements), so that x (and dy) are read once, the variance is
// the second pass over registers about the exact mean, and nothing is
// recomputed.  All sums are fp32; y and dx are rounded once to the type of x,
// dw and db once to the type of the weight.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cstdint>

#include "block_internal.h"
#include "tc_common.cuh"

namespace gn {
namespace {

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }

template <typename T> __device__ __forceinline__ T from_float(float v);
template <> __device__ __forceinline__ float from_float<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }

template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
    T v[N];
};

// One element of the weight or the bias, in its own format.
__device__ __forceinline__ float load_param(const void *p, int format, int c)
{
    if (format == GN_FORMAT_FP32) return __ldg(static_cast<const float *>(p) + c);
    if (format == GN_FORMAT_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[c]);
    return __half2float(static_cast<const __half *>(p)[c]);
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

// Sum of one or two values over the tpr threads that share a row: within a
// warp (tpr <= 32, a power of two), or over the whole CTA (tpr == blockDim.x).
// The CTA's sums go through `scratch`, two buffers taken in turn so that one
// barrier per reduction is enough.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int tpr, float (*scratch)[32][2], int &turn)
{
    const int width = tpr < 32 ? tpr : 32;
    for (int o = width >> 1; o > 0; o >>= 1)
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
    if (tpr <= 32) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = tpr >> 5;
    float(*s)[2] = scratch[turn];
    turn ^= 1;
    if (lane == 0)
#pragma unroll
        for (int n = 0; n < N; ++n) s[warp][n] = v[n];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = lane < warps ? s[lane][n] : 0.f;
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
}

template <typename T, int EPV, int NV>
__device__ __forceinline__ void load_row(const T *row, int lane, int tpr, int cols, float (&f)[NV][EPV])
{
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = (lane + k * tpr) * EPV;
        Pack<T, EPV> p;
        if (c < cols) p = *reinterpret_cast<const Pack<T, EPV> *>(row + c);
#pragma unroll
        for (int e = 0; e < EPV; ++e) f[k][e] = c < cols ? to_float(p.v[e]) : 0.f;
    }
}

template <typename T, int EPV, int NV>
__global__ void __launch_bounds__(1024) norm_forward_kernel(const NormArgs a, int tpr)
{
    __shared__ float scratch[2][32][2];
    tc::griddep_wait();
    if (threadIdx.x == 0) tc::griddep_launch_dependents();
    const int per = blockDim.x / tpr, lane = threadIdx.x % tpr;
    const float inv = 1.0f / static_cast<float>(a.cols);
    int turn = 0;
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * per; r0 < a.rows; r0 += static_cast<int64_t>(gridDim.x) * per) {
        const int64_t row = r0 + threadIdx.x / tpr;
        const bool live = row < a.rows;   // whole warps stay for the shuffles
        float f[NV][EPV];
        const T *x = static_cast<const T *>(a.x) + (live ? row : r0) * a.x_stride;
        load_row<T, EPV, NV>(x, lane, tpr, a.cols, f);
        float s[1] = {0.f};
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int e = 0; e < EPV; ++e) s[0] += f[k][e];
        row_sum(s, tpr, scratch, turn);
        const float mean = s[0] * inv;
        float q[1] = {0.f};
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int e = 0; e < EPV; ++e) {
                f[k][e] -= mean;
                if ((lane + k * tpr) * EPV < a.cols) q[0] = fmaf(f[k][e], f[k][e], q[0]);
            }
        row_sum(q, tpr, scratch, turn);
        const float rstd = 1.0f / sqrtf(fmaf(q[0], inv, a.eps));
        if (!live) continue;
        if (lane == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
        T *y = static_cast<T *>(a.y) + row * a.y_stride;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (lane + k * tpr) * EPV;
            if (c >= a.cols) break;
            Pack<T, EPV> p;
#pragma unroll
            for (int e = 0; e < EPV; ++e) {
                float v = f[k][e] * rstd;
                if (a.weight) v *= load_param(a.weight, a.weight_format, c + e);
                if (a.bias) v += load_param(a.bias, a.weight_format, c + e);
                p.v[e] = from_float<T>(v);
            }
            *reinterpret_cast<Pack<T, EPV> *>(y + c) = p;
        }
    }
}

template <typename T, int EPV, int NV>
__global__ void __launch_bounds__(1024) norm_backward_kernel(const NormGradArgs a, int tpr)
{
    extern __shared__ float columns[];    // [2][cols], tpr < blockDim.x with a weight
    __shared__ float scratch[2][32][2];
    tc::griddep_wait();
    if (threadIdx.x == 0) tc::griddep_launch_dependents();
    const int per = blockDim.x / tpr, lane = threadIdx.x % tpr;
    const float inv = 1.0f / static_cast<float>(a.cols);
    float sw[NV][EPV] = {}, sb[NV][EPV] = {};
    int turn = 0;
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * per; r0 < a.rows; r0 += static_cast<int64_t>(gridDim.x) * per) {
        const int64_t row = r0 + threadIdx.x / tpr;
        const bool live = row < a.rows;
        const int64_t at = live ? row : r0;
        float x[NV][EPV], g[NV][EPV];
        load_row<T, EPV, NV>(static_cast<const T *>(a.x) + at * a.x_stride, lane, tpr, a.cols, x);
        load_row<T, EPV, NV>(static_cast<const T *>(a.dy) + at * a.dy_stride, lane, tpr, a.cols, g);
        const float mean = a.mean[at], rstd = a.rstd[at];
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (lane + k * tpr) * EPV;
            if (c >= a.cols) break;
#pragma unroll
            for (int e = 0; e < EPV; ++e) {
                x[k][e] = (x[k][e] - mean) * rstd;
                if (a.weight) {
                    if (live) {
                        sw[k][e] = fmaf(g[k][e], x[k][e], sw[k][e]);
                        sb[k][e] += g[k][e];
                    }
                    g[k][e] *= load_param(a.weight, a.weight_format, c + e);
                }
                s[0] += g[k][e];
                s[1] = fmaf(g[k][e], x[k][e], s[1]);
            }
        }
        row_sum(s, tpr, scratch, turn);
        if (!live) continue;
        T *dx = static_cast<T *>(a.dx) + row * a.dx_stride;
        const float m0 = s[0] * inv, m1 = s[1] * inv;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (lane + k * tpr) * EPV;
            if (c >= a.cols) break;
            Pack<T, EPV> p;
#pragma unroll
            for (int e = 0; e < EPV; ++e) p.v[e] = from_float<T>(rstd * (g[k][e] - m0 - x[k][e] * m1));
            *reinterpret_cast<Pack<T, EPV> *>(dx + c) = p;
        }
    }
    if (!a.weight) return;
    // the CTA's sums: the row groups one after the other (a fixed order), then out
    float *out = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
    if (per > 1) {
        for (int g = 0; g < per; ++g) {
            if (static_cast<int>(threadIdx.x) / tpr == g)
#pragma unroll
                for (int k = 0; k < NV; ++k)
#pragma unroll
                    for (int e = 0; e < EPV; ++e) {
                        const int c = (lane + k * tpr) * EPV + e;
                        if (c >= a.cols) continue;
                        columns[c] = (g ? columns[c] : 0.f) + sw[k][e];
                        columns[a.cols + c] = (g ? columns[a.cols + c] : 0.f) + sb[k][e];
                    }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < 2 * a.cols; c += blockDim.x) out[c] = columns[c];
    } else {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int e = 0; e < EPV; ++e) {
                const int c = (lane + k * tpr) * EPV + e;
                if (c >= a.cols) continue;
                out[c] = sw[k][e];
                out[a.cols + c] = sb[k][e];
            }
    }
}

// dw and db from the CTAs' partial sums: a warp's lanes take 32 neighbouring
// columns, the eight warps every eighth partial each, added up in a fixed order.
__global__ void __launch_bounds__(256) norm_columns_kernel(const NormGradArgs a, int blocks)
{
    __shared__ float part[8][32];
    tc::griddep_wait();
    if (threadIdx.x == 0) tc::griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x * 32 + lane;
    float v = 0.f;
    if (c < 2 * a.cols)
        for (int b = warp; b < blocks; b += 8) v += a.partial[static_cast<int64_t>(b) * 2 * a.cols + c];
    part[warp][lane] = v;
    __syncthreads();
    if (warp != 0 || c >= 2 * a.cols) return;
#pragma unroll
    for (int w = 1; w < 8; ++w) v += part[w][lane];
    if (c < a.cols)
        store_param(a.dweight, a.weight_format, c, v);
    else
        store_param(a.dbias, a.weight_format, c - a.cols, v);
}

struct Shape {
    int tpr, threads, nv;
};

// `slots` pieces of a row over tpr threads of nv slots: four slots a thread
// where that leaves at least a warp's worth of rows, one thread group per row.
Shape norm_shape(int slots)
{
    Shape s;
    s.nv = 4;
    int tpr = 1;
    while (tpr * s.nv < slots) tpr *= 2;
    if (tpr > 1024) {
        tpr = 1024;
        s.nv = 16;
    }
    s.tpr = tpr;
    s.threads = std::max(tpr, 256);
    if (tpr > 32) s.threads = tpr;
    return s;
}

bool vectors_ok(int cols, int epv, const void *const *ptrs, int n, const int64_t *strides)
{
    if (cols % epv) return false;
    for (int i = 0; i < n; ++i)
        if (reinterpret_cast<uintptr_t>(ptrs[i]) % 16 || strides[i] % epv) return false;
    return true;
}

template <typename T>
cudaError_t forward(const NormArgs &a, int sm_count, cudaStream_t s)
{
    constexpr int EPV = 16 / sizeof(T);
    const void *ptrs[] = {a.x, a.y};
    const int64_t strides[] = {a.x_stride, a.y_stride};
    const bool vec = vectors_ok(a.cols, EPV, ptrs, 2, strides);
    const Shape sh = norm_shape(vec ? a.cols / EPV : a.cols);
    const int64_t per = sh.threads / sh.tpr;
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>((a.rows + per - 1) / per, 8 * sm_count)));
    if (vec) return tc::launch_pdl(norm_forward_kernel<T, EPV, 4>, grid, dim3(sh.threads), 0, s, a, sh.tpr);
    if (sh.nv == 4) return tc::launch_pdl(norm_forward_kernel<T, 1, 4>, grid, dim3(sh.threads), 0, s, a, sh.tpr);
    return tc::launch_pdl(norm_forward_kernel<T, 1, 16>, grid, dim3(sh.threads), 0, s, a, sh.tpr);
}

template <typename T>
cudaError_t backward(const NormGradArgs &a, int sm_count, cudaStream_t s)
{
    constexpr int EPV = 16 / sizeof(T);
    const void *ptrs[] = {a.x, a.dy, a.dx};
    const int64_t strides[] = {a.x_stride, a.dy_stride, a.dx_stride};
    const bool vec = vectors_ok(a.cols, EPV, ptrs, 3, strides);
    const Shape sh = norm_shape(vec ? a.cols / EPV : a.cols);
    const dim3 grid(static_cast<unsigned>(layer_norm_blocks(a.rows, a.cols, sm_count)));
    const size_t smem = a.weight && sh.threads > sh.tpr ? 8u * static_cast<size_t>(a.cols) : 0;
    if (vec) return tc::launch_pdl(norm_backward_kernel<T, EPV, 4>, grid, dim3(sh.threads), smem, s, a, sh.tpr);
    if (sh.nv == 4) return tc::launch_pdl(norm_backward_kernel<T, 1, 4>, grid, dim3(sh.threads), smem, s, a, sh.tpr);
    return tc::launch_pdl(norm_backward_kernel<T, 1, 16>, grid, dim3(sh.threads), smem, s, a, sh.tpr);
}

}  // namespace

int layer_norm_blocks(int64_t rows, int, int sm_count)
{
    return static_cast<int>(std::min<int64_t>(rows, 2 * sm_count));
}

cudaError_t launch_layer_norm(const NormArgs &a, int sm_count, cudaStream_t s)
{
    if (a.format == GN_FORMAT_BF16) return forward<__nv_bfloat16>(a, sm_count, s);
    if (a.format == GN_FORMAT_FP16) return forward<__half>(a, sm_count, s);
    return forward<float>(a, sm_count, s);
}

cudaError_t launch_layer_norm_backward(const NormGradArgs &a, int sm_count, cudaStream_t s, int *launches)
{
    cudaError_t e;
    if (a.format == GN_FORMAT_BF16)
        e = backward<__nv_bfloat16>(a, sm_count, s);
    else if (a.format == GN_FORMAT_FP16)
        e = backward<__half>(a, sm_count, s);
    else
        e = backward<float>(a, sm_count, s);
    if (e != cudaSuccess) return e;
    *launches = 1;
    if (!a.weight) return e;
    e = tc::launch_pdl(norm_columns_kernel, dim3((2 * a.cols + 31) / 32), dim3(256), 0, s, a,
                       layer_norm_blocks(a.rows, a.cols, sm_count));
    if (e == cudaSuccess) *launches = 2;
    return e;
}

}  // namespace gn
