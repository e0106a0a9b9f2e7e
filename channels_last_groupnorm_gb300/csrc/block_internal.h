// block_internal.h -- host-side declarations of the transformer-block kernels
// (norm_kernels.cu, rope_kernels.cu, pattn_kernels.cu) for the C ABI in
// block_capi.cu.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/gnsilu.h"

namespace gn {

// The bound on a kernel's waits, and the words that tell when one ran out.
struct WaitLimit {
    uint64_t timeout_ns;
    unsigned int *status, *host_status;   // device addresses
};

// ---- layer norm (norm_kernels.cu) -------------------------------------------
constexpr int kNormMaxCols = 16384;

// Where rows lie: row n = a inner + b at a outer + b stride elements (flat: n stride).
struct RowsAt {
    int64_t outer, stride;
};

struct NormArgs {
    const void *x, *weight, *bias;
    void *y;
    float *mean, *rstd;
    int64_t rows;
    int cols;
    RowsAt x_at, y_at;
    int64_t inner;                // >= rows: flat
    float eps;
    int format, weight_format;
};

struct NormGradArgs {
    const void *dy, *x, *weight;
    const float *mean, *rstd;
    void *dx, *dweight, *dbias;
    int64_t rows;
    int cols;
    RowsAt dy_at, x_at, dx_at;
    int64_t inner;
    int format, weight_format;
    float *partial;               // [blocks][2][cols] when the weight's gradient is wanted
};

cudaError_t launch_layer_norm(const NormArgs &a, int sm_count, const WaitLimit &limit, cudaStream_t s);
// The most CTAs that launch_layer_norm_backward uses, each with a row of partial sums.
int layer_norm_blocks(int64_t rows, int cols, int sm_count);
cudaError_t launch_layer_norm_backward(const NormGradArgs &a, int sm_count, const WaitLimit &limit, cudaStream_t s,
                                       int *launches);

// ---- rotary positions over several axes (rope_kernels.cu) -------------------
constexpr int kRopeMaxPairs = 128;
constexpr int64_t kRopeMaxElements = 1 << 30;   // of one token: its pieces are counted in an int, plus a grid's step

struct RopeArgs {
    const void *in[2];            // query and key heads (the second may be null)
    void *out[2];
    int64_t in_token[2], in_head[2], out_token[2], out_head[2];   // strides in elements
    int heads[2];
    int64_t tokens;
    int dim, pairs;
    const void *positions;        // [tokens][axes]
    int axes, position_format;
    int interleaved, inverse, format;
    double turns[kRopeMaxPairs];              // turns of a pair per unit of its axis' position
    unsigned char axis[kRopeMaxPairs];
};

cudaError_t launch_rope(const RopeArgs &a, int sm_count, cudaStream_t s);

// ---- attention of packed documents (pattn_*.cu) ------------------------------
struct PackedAttn {
    gn_attn_packed_args a;
    int group;                    // query heads per key / value head
    // backward only
    const void *dout;
    int64_t dout_token, dout_head;
    void *dq, *dk, *dv;
    void *workspace;
};

// On the tensor cores (pattn_forward.cu); tokens_q and tokens_k at least 1.
cudaError_t launch_packed_attn_tiles(const PackedAttn &p, const WaitLimit &limit, cudaStream_t s);
// On the tensor cores for few queries per document (pattn_split.cu); tokens_q and tokens_k at least 1.
// (about how long that takes, for the choice between the two)
double packed_attn_split_us(const PackedAttn &p, int sm_count);
cudaError_t launch_packed_attn_split(const PackedAttn &p, int sm_count, const WaitLimit &limit, cudaStream_t s);
cudaError_t launch_packed_attn(const PackedAttn &p, int sm_count, const WaitLimit &limit, cudaStream_t s, int *launches);
size_t packed_attn_workspace_bytes(int64_t tokens_q, int heads);
cudaError_t launch_packed_attn_backward(const PackedAttn &p, int sm_count, const WaitLimit &limit, cudaStream_t s,
                                        int *launches);

}  // namespace gn
