// rope_kernels.cu -- sm_103a kernel of rotary positions over several axes.
//
// The first 2 P channels of a head form P pairs (a, b): neighbours
// (2p, 2p + 1), or channel p of either half (p, P + p).  Pair p belongs to one
// position axis and turns by  angle = position[axis] * theta^(-2 i / d)  (i its
// place among the d / 2 pairs of its axis):
//     a' = a cos - b sin,   b' = a sin + b cos
// The inverse (the gradient's rotation) turns back.  Channels from 2 P on pass
// unchanged.
//
// The angle is formed in turns, in fp64 (position x turns per position, less
// its nearest integer), so that far positions keep their phase; the sine and
// cosine of what is left are fp32.  They are computed once per token, in
// shared memory, for all query and key heads.  Products and sums are fp32,
// rounded once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cstdint>

#include "block_internal.h"
#include "block_math.cuh"
#include "tc_common.cuh"

namespace gn {
namespace {

constexpr int kRopeThreads = 256;

template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
    T v[N];
};

__device__ __forceinline__ double position_of(const RopeArgs &a, int64_t token, int axis)
{
    const int64_t at = token * a.axes + axis;
    if (a.position_format == GN_POSITIONS_INT32) return static_cast<double>(static_cast<const int32_t *>(a.positions)[at]);
    if (a.position_format == GN_POSITIONS_INT64) return static_cast<double>(static_cast<const int64_t *>(a.positions)[at]);
    return static_cast<double>(static_cast<const float *>(a.positions)[at]);
}

// A unit of work is EPV pairs of one head (EPV = 1: a single pair, or a
// single channel of the unturned rest).
template <typename T, int EPV>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a)
{
    __shared__ float2 turn[kRopeMaxPairs];
    tc::griddep_wait();
    if (threadIdx.x == 0) tc::griddep_launch_dependents();
    const int heads = a.heads[0] + a.heads[1], rest = a.dim - 2 * a.pairs;
    // units of a head: pieces of EPV channels (neighbours paired: EPV / 2
    // pairs; halves paired: a piece of either half), then pieces of the rest
    constexpr int PV = EPV == 1 ? 1 : EPV;
    const int turned = EPV == 1 ? a.pairs : (a.interleaved ? 2 * a.pairs / PV : a.pairs / PV);
    const int units = turned + rest / PV;
    for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
        __syncthreads();
        for (int p = threadIdx.x; p < a.pairs; p += blockDim.x) {
            const double w = position_of(a, t, a.axis[p]) * a.turns[p];
            float s, c;
            sincospif(2.0f * static_cast<float>(w - rint(w)), &s, &c);
            turn[p] = make_float2(c, a.inverse ? -s : s);
        }
        __syncthreads();
        for (int i = blockIdx.y * blockDim.x + threadIdx.x; i < heads * units; i += gridDim.y * blockDim.x) {
            int h = i / units;
            const int u = i - h * units;
            const int which = h >= a.heads[0];
            if (which) h -= a.heads[0];
            const T *in = static_cast<const T *>(a.in[which]) + t * a.in_token[which] + h * a.in_head[which];
            T *out = static_cast<T *>(a.out[which]) + t * a.out_token[which] + h * a.out_head[which];
            if (u >= turned) {
                const int c = 2 * a.pairs + (u - turned) * PV;
                *reinterpret_cast<Pack<T, PV> *>(out + c) = *reinterpret_cast<const Pack<T, PV> *>(in + c);
            } else if (EPV > 1 && a.interleaved) {
                Pack<T, PV> x = *reinterpret_cast<const Pack<T, PV> *>(in + u * PV);
#pragma unroll
                for (int e = 0; e < PV / 2; ++e) {
                    const float2 w = turn[u * (PV / 2) + e];
                    const float p = to_float(x.v[2 * e]), q = to_float(x.v[2 * e + 1]);
                    x.v[2 * e] = from_float<T>(p * w.x - q * w.y);
                    x.v[2 * e + 1] = from_float<T>(p * w.y + q * w.x);
                }
                *reinterpret_cast<Pack<T, PV> *>(out + u * PV) = x;
            } else {
                const int c0 = a.interleaved ? 2 * u : u * PV, c1 = a.interleaved ? 2 * u + 1 : a.pairs + u * PV;
                Pack<T, PV> x = *reinterpret_cast<const Pack<T, PV> *>(in + c0);
                Pack<T, PV> y = *reinterpret_cast<const Pack<T, PV> *>(in + c1);
#pragma unroll
                for (int e = 0; e < PV; ++e) {
                    const float2 w = turn[u * PV + e];
                    const float p = to_float(x.v[e]), q = to_float(y.v[e]);
                    x.v[e] = from_float<T>(p * w.x - q * w.y);
                    y.v[e] = from_float<T>(p * w.y + q * w.x);
                }
                *reinterpret_cast<Pack<T, PV> *>(out + c0) = x;
                *reinterpret_cast<Pack<T, PV> *>(out + c1) = y;
            }
        }
    }
}

template <typename T>
cudaError_t rope(const RopeArgs &a, int sm_count, cudaStream_t s)
{
    constexpr int EPV = 16 / sizeof(T);
    bool vec = a.dim % EPV == 0 && (a.interleaved ? 2 * a.pairs : a.pairs) % EPV == 0;
    for (int i = 0; i < 2; ++i) {
        if (!a.in[i]) continue;
        vec = vec && reinterpret_cast<uintptr_t>(a.in[i]) % 16 == 0 && reinterpret_cast<uintptr_t>(a.out[i]) % 16 == 0 &&
              a.in_token[i] % EPV == 0 && a.in_head[i] % EPV == 0 && a.out_token[i] % EPV == 0 &&
              a.out_head[i] % EPV == 0;
    }
    const int units = (a.heads[0] + a.heads[1]) * (vec ? (a.dim / EPV) : a.dim - a.pairs);
    const int64_t per_token = (units + kRopeThreads - 1) / kRopeThreads;
    const int64_t want = 8 * sm_count;
    dim3 grid;
    grid.x = static_cast<unsigned>(std::min<int64_t>(a.tokens, want));
    grid.y = static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(per_token, want / grid.x / 2)));
    if (vec) return tc::launch_pdl(rope_kernel<T, EPV>, grid, dim3(kRopeThreads), 0, s, a);
    return tc::launch_pdl(rope_kernel<T, 1>, grid, dim3(kRopeThreads), 0, s, a);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, int sm_count, cudaStream_t s)
{
    if (a.format == GN_FORMAT_BF16) return rope<__nv_bfloat16>(a, sm_count, s);
    if (a.format == GN_FORMAT_FP16) return rope<__half>(a, sm_count, s);
    return rope<float>(a, sm_count, s);
}

}  // namespace gn
