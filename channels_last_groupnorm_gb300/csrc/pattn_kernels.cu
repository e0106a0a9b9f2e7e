// pattn_kernels.cu -- attention of packed documents on sm_103a.
//
// Query i of a document sees a run [lo_i, hi_i) of the document's keys: all of
// them, or (causal) those up to its own position and those of the document's
// prefix.  With t_ij = scale q_i . k_j, capped (t <- cap tanh(t / cap)) and
// biased (t <- t - slope |pos_i - j|):
//   lse_i = log sum_j exp(t_ij),  p_ij = exp(t_ij - lse_i),  out_i = sum_j p_ij v_j
//   delta_i = dout_i . out_i,     ds_ij = p_ij (dout_i . v_j - delta_i) (1 - tanh^2)
//   dq_i = scale sum_j ds_ij k_j, dk_j = scale sum_i ds_ij q_i, dv_j = sum_i p_ij dout_i
// with dk and dv summed over the query heads that share a key / value head.
// A query that sees no key has out = 0, lse = -inf and adds nothing to any
// gradient; what keys outside its run hold has no influence on it.
#include <algorithm>

#include "pattn_common.cuh"
#include "tc_common.cuh"

namespace gn {
namespace {

// No keys at all: zeros, and lse -inf.
__global__ void __launch_bounds__(256) attn_nothing_kernel(const gn_attn_packed_args a)
{
    tc::griddep_wait();
    if (threadIdx.x == 0) tc::griddep_launch_dependents();
    const int64_t n = a.tokens_q * a.heads, step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    for (int64_t i = first; i < n; i += step) a.lse[i] = -INFINITY;
    for (int64_t i = first; i < n * a.dim / 8; i += step) static_cast<uint4 *>(a.out)[i] = make_uint4(0u, 0u, 0u, 0u);
}

// About how long the kernel with tiles of 256 queries of one head takes, in us:
// a tile meets the keys of every document that it touches, 1.6 us for a block of
// 128, and about 4 us besides, one tile per SM at a time.  Few queries per
// document make that long, and the splitting kernel, which reads the keys once
// for all heads that share them, the better one (24 caches of up to 8000 keys, 32
// heads on 8: 1 new token each 77 against 1568 us, 16 each 158 against 1046 us);
// for many short documents of many queries it is the other way round.
double tiles_us(const PackedAttn &p, int sm_count)
{
    const gn_attn_packed_args &a = p.a;
    const double per_doc = static_cast<double>(a.tokens_q) / a.docs, keys = static_cast<double>(a.tokens_k) / a.docs;
    const int64_t tiles = (a.tokens_q + 255) / 256 * a.heads;
    const double blocks = std::max(1.0, 256.0 / std::max(per_doc, 1.0 / 256)) * keys / 128 + 1;
    return static_cast<double>((tiles + sm_count - 1) / sm_count) * (4.0 + 1.6 * blocks);
}

}  // namespace

cudaError_t launch_packed_attn(const PackedAttn &p, int sm_count, const WaitLimit &limit, cudaStream_t s, int *launches)
{
    const gn_attn_packed_args &a = p.a;
    cudaError_t e;
    if (a.tokens_k == 0)
        e = tc::launch_pdl(attn_nothing_kernel, dim3(static_cast<unsigned>(sm_count)), dim3(256), 0, s, a);
    else if (packed_attn_split_us(p, sm_count) < tiles_us(p, sm_count))
        e = launch_packed_attn_split(p, sm_count, limit, s);
    else
        e = launch_packed_attn_tiles(p, limit, s);
    if (e == cudaSuccess) ++*launches;
    return e;
}

}  // namespace gn
