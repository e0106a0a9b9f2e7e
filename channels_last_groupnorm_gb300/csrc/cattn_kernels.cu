// cattn_kernels.cu -- attention of new tokens over the paged cache: the choice of a
// kernel, the tensor maps of the pages, and the kernel that joins pieces of tiles.
#include <algorithm>

#include "cattn_common.cuh"

namespace gn {
namespace cattn {
namespace {

// Joins the pieces of the tiles that several CTAs shared.  Block (c, y) looks after the
// tile that CTA c began, if others went on with it, and there after some of its rows: a
// warp each, or with many pieces all warps, each with some of the pieces (one token at 131072,
// 38 pieces of a tile: 26 us with a warp for a row).  Four channels a lane; every load of a
// row's outputs is on its way before the first is used.
constexpr int kFewRows = 32, kManyRows = 2 * kTile;
constexpr int kJoinWarps = 8, kJoinMany = 8;

template <typename T>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const __grid_constant__ CattnArgs args)
{
    __shared__ float4 sums[kJoinWarps][32];
    __shared__ float weights[kJoinWarps];
    tc::griddep_wait();
    if (threadIdx.x == 0) tc::griddep_launch_dependents();
    const gn_cache &c = args.p.c;
    const gn_attn_cached_args &a = args.p.a;
    const Shared s = args.shared[blockIdx.x];
    if (s.pieces <= 1 || *reinterpret_cast<volatile unsigned int *>(args.limit.status) != 0u) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool many = s.pieces > kJoinMany && args.rows <= kFewRows;      // (more rows keep the warps busy)
    const float *first = piece_of(args, blockIdx.x, 1), *others = piece_of(args, blockIdx.x, 0);
    const int64_t step = 2 * static_cast<int64_t>(args.rows) * (2 + c.dim);
    const auto piece = [&](int p) { return p == 0 ? first : others + p * step; };
    const int at = min(4 * lane, c.dim - 4);       // (lanes past the width read what another does)
    const int row0 = many ? blockIdx.y : blockIdx.y * kJoinWarps + warp, rows = many ? gridDim.y : gridDim.y * kJoinWarps;
    for (int row = row0; row < s.rows; row += rows) {
        const int i = row / args.heads, h = row - i * args.heads;
        const bool there = h < s.heads;            // (the same for all who share the row)
        float top = -INFINITY, sum = 0.f;
        for (int p = lane; p < s.pieces; p += 32) top = fmaxf(top, piece(p)[row]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        float4 out = make_float4(0.f, 0.f, 0.f, 0.f);
        const int p0 = many ? warp : 0, by = many ? kJoinWarps : 1;
        for (int q = p0; q < s.pieces; q += 8 * by) {
            float4 v[8];
            float f[8], l[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int p = min(q + e * by, s.pieces - 1);
                f[e] = piece(p)[row];
                l[e] = q + e * by < s.pieces ? piece(p)[args.rows + row] : 0.f;
                v[e] = *reinterpret_cast<const float4 *>(piece(p) + 2 * args.rows + row * c.dim + at);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // (a part that saw nothing has a sum of zero)
                if (l[e] == 0.f) continue;
                const float g = ex2_approx(f[e] - top);
                sum = fmaf(g, l[e], sum);
                axpy4(out, g, v[e]);
            }
        }
        if (many) {
            sums[warp][lane] = out;
            if (lane == 0) weights[warp] = sum;
            __syncthreads();
            if (warp == 0) {
                sum = 0.f;
                out = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kJoinWarps; ++w) {
                    sum += weights[w];
                    axpy4(out, 1.0f, sums[w][lane]);
                }
            }
            __syncthreads();
            if (warp != 0) continue;
        }
        if (!there) continue;
        const float inv = sum == 0.f ? 0.f : 1.0f / sum;
        const int64_t token = s.token + i, head = s.head + h;
        store4<T>(a.out, (token * a.heads + head) * c.dim, lane, c.dim, make_float4(out.x * inv, out.y * inv, out.z * inv, out.w * inv));
        if (lane == 0) a.lse[head * a.tokens + token] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
    }
}

// Tensor map over a pool's [pages][heads][tokens][dim] bytes with boxes of 128 channels
// (those past the width read as zeros) x `chunk` tokens.
bool encode_pool(CUtensorMap *map, const void *base, const gn_cache &c, int64_t page, int64_t token, int64_t head, int chunk)
{
    const tc::EncodeTiledFn fn = tc::encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.dim), static_cast<cuuint64_t>(c.page_size),
                                static_cast<cuuint64_t>(c.kv_heads), static_cast<cuuint64_t>(c.pages)};
    // (an axis of one has no stride of its own)
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(token), static_cast<cuuint64_t>(c.kv_heads > 1 ? head : 16),
                                   static_cast<cuuint64_t>(c.pages > 1 ? page : 16)};
    const cuuint32_t box[4] = {128, static_cast<cuuint32_t>(chunk), 1, 1};
    const cuuint32_t step[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(base), dims, strides, box, step,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The tiles of a call and the kernel for them: up to 32 rows on the tensor core's narrow
// side (16 where that is all there is), or 256 on its wide side.
CattnArgs plan(const CachedAttn &p, bool *few)
{
    CattnArgs a = {};
    a.p = p;
    a.scale_log2 = p.a.scale * kLog2e;
    const int64_t each = p.c.cu ? std::max<int64_t>(1, p.a.tokens / p.c.sequences) : p.a.tokens / p.c.sequences;
    *few = each * p.group <= kFewRows;
    a.heads = std::min(p.group, *few ? kFewRows : kManyRows);
    const int most = !*few ? kManyRows : each * a.heads <= 16 ? 16 : kFewRows;
    a.chunks = (p.group + a.heads - 1) / a.heads;
    a.tokens = most / a.heads;
    if (!p.c.cu) a.tokens = static_cast<int>(std::min<int64_t>(a.tokens, each));
    a.rows = !*few ? kManyRows : a.tokens * a.heads <= 16 ? 16 : kFewRows;
    a.extra = *few ? 4 : 8;
    a.chunk = kTile;
    while (p.c.page_size % a.chunk) a.chunk /= 2;
    return a;
}

}  // namespace

cudaError_t launch_join(const CattnArgs &a, int ctas, cudaStream_t s)
{
    return tc::launch_pdl(a.p.a.format == GN_FORMAT_BF16 ? join_kernel<__nv_bfloat16> : join_kernel<__half>,
                          dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(std::min(a.rows, 16))), dim3(32 * kJoinWarps), 0, s, a);
}

}  // namespace cattn

namespace {

// The CTAs' words about tiles that are to be joined, ahead of the pieces.
size_t shared_bytes(int sm_count) { return (2u * static_cast<size_t>(sm_count) * sizeof(cattn::Shared) + 255) / 256 * 256; }

}  // namespace

// (the few rows of two CTAs an SM, or the many of one)
size_t cached_attn_workspace_bytes(int64_t, int, int, int, int dim, int sm_count)
{
    return shared_bytes(sm_count) + 4u * 2u * static_cast<size_t>(sm_count) * cattn::kManyRows * static_cast<size_t>(2 + dim);
}

cudaError_t launch_cached_attn(const CachedAttn &p, int sm_count, const WaitLimit &limit, cudaStream_t s, int *launches)
{
    bool few;
    cattn::CattnArgs a = cattn::plan(p, &few);
    a.limit = limit;
    a.shared = static_cast<cattn::Shared *>(p.workspace);
    a.pieces = reinterpret_cast<float *>(static_cast<char *>(p.workspace) + shared_bytes(sm_count));
    const gn_cache &c = p.c;
    CUtensorMap mk, mv;
    if (!cattn::encode_pool(&mk, c.k_pages, c, c.k_page, c.k_token, c.k_head, a.chunk) ||
        !cattn::encode_pool(&mv, c.v_pages, c, c.v_page, c.v_token, c.v_head, a.chunk))
        return cudaErrorInvalidValue;
    const int ctas = few ? 2 * sm_count : sm_count;
    cudaError_t e = few ? cattn::launch_cached_few(a, mk, mv, ctas, s) : cattn::launch_cached_tiles(a, mk, mv, ctas, s);
    if (e == cudaSuccess) ++*launches, e = cattn::launch_join(a, ctas, s);
    if (e == cudaSuccess) ++*launches;
    return e;
}

}  // namespace gn
