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
// gradient.  Keys outside a query's run are never read for it.
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

}  // namespace

cudaError_t launch_packed_attn(const PackedAttn &p, int sm_count, const WaitLimit &limit, cudaStream_t s, int *launches)
{
    const gn_attn_packed_args &a = p.a;
    cudaError_t e;
    // Few queries per document (with all heads that share its keys no more than
    // one tile's 128 rows): the keys are split and read once for all of them.
    // Else tiles of 128 queries of one head.  24 caches of up to 8000 keys, 32
    // heads on 8: 1 token each 85 against 1031 us (the tiles pack neighbouring
    // documents and meet every one's keys), 16 tokens each 165 against 1031 us.
    if (a.tokens_k == 0)
        e = tc::launch_pdl(attn_nothing_kernel, dim3(static_cast<unsigned>(sm_count)), dim3(256), 0, s, a);
    else if ((a.tokens_q + a.docs - 1) / a.docs * std::min(p.group, 128) <= 128)
        e = launch_packed_attn_split(p, sm_count, limit, s);
    else
        e = launch_packed_attn_tiles(p, limit, s);
    if (e == cudaSuccess) ++*launches;
    return e;
}

}  // namespace gn
