// cattn_kernels.cu -- attention of new tokens over the paged cache: the choice of a
// kernel, the tensor maps of the pages, and the kernel that joins pieces of tiles.
#include <algorithm>

#include "cattn_common.cuh"

namespace gn {
namespace cattn {
namespace {

// Joins the pieces of the tiles that several CTAs shared.  CTA c looks after the tile
// in which the c-th part of the work begins, if it is the second to work on it: part
// c - 1 holds the tile's beginning, and parts c, c + 1, ... go on with it.
template <typename T>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ CattnArgs args)
{
    __shared__ DealRoom room;
    tc::griddep_wait();
    if (threadIdx.x == 0) tc::griddep_launch_dependents();
    const gn_cache &c = args.p.c;
    const gn_attn_cached_args &a = args.p.a;
    const Part part = deal(args, room, gridDim.x);
    if (part.count == 0 || *reinterpret_cast<volatile unsigned int *>(args.limit.status) != 0u) return;
    Walk walk(args);
    walk.start(part.seq, part.offset, part.count);
    Segment g;
    walk.next(g);
    const int64_t begin = part.first - g.b0, end = begin + g.total;     // of the tile, among all units
    const int cta = blockIdx.x;
    if (g.b0 == 0 || part_begin(part.all, part.ctas, cta - 1) > begin) return;
    int others = 0;                       // parts after the first
    while (cta + others < part.ctas && part_begin(part.all, part.ctas, cta + others) < end) ++others;
    const int first_token = g.run * args.tokens, count = min(args.tokens, g.s.end - g.s.begin - first_token);
    const float *first = piece_of(args, cta - 1, 1);
    const int64_t step = 2 * static_cast<int64_t>(args.rows) * (2 + c.dim);
    const float *next = piece_of(args, cta, 0);
    const int quads = c.dim / 4;
    for (int n = threadIdx.x; n < count * args.heads * quads; n += blockDim.x) {
        const int row = n / quads, q = n - row * quads;
        const int h = g.first_head + row % args.heads;
        if (h >= args.p.group) continue;
        float top = first[row], sum = first[args.rows + row];
        float4 o = *reinterpret_cast<const float4 *>(first + 2 * args.rows + row * c.dim + 4 * q);
#pragma unroll 4
        for (int p = 0; p < others; ++p) {
            const float *piece = next + p * step;
            const float m = piece[row], l = piece[args.rows + row];
            const float4 v = *reinterpret_cast<const float4 *>(piece + 2 * args.rows + row * c.dim + 4 * q);
            // (a part that saw nothing has a sum of zero; NaN stays)
            const float now = fmaxf(top, m);
            const float f = sum == 0.f ? 0.f : ex2_approx(top - now), e = l == 0.f ? 0.f : ex2_approx(m - now);
            o.x = fmaf(o.x, f, v.x * e);
            o.y = fmaf(o.y, f, v.y * e);
            o.z = fmaf(o.z, f, v.z * e);
            o.w = fmaf(o.w, f, v.w * e);
            sum = fmaf(sum, f, l * e);
            top = now;
        }
        const float by = sum == 0.f ? 0.f : 1.0f / sum;
        const int64_t token = g.s.begin + first_token + row / args.heads, head = g.hk * args.p.group + h;
        *reinterpret_cast<uint2 *>(static_cast<T *>(a.out) + (token * a.heads + head) * c.dim + 4 * q) =
            make_uint2(Half2<T>::pack(o.x * by, o.y * by), Half2<T>::pack(o.z * by, o.w * by));
        if (q == 0) a.lse[head * a.tokens + token] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
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

constexpr int kFewRows = 32;

// The tiles of a call: up to 32 rows, 16 where that is all there is (half the
// registers, a deeper ring).
CattnArgs plan(const CachedAttn &p)
{
    CattnArgs a = {};
    a.p = p;
    a.scale_log2 = p.a.scale * kLog2e;
    a.heads = std::min(p.group, kFewRows);
    a.chunks = (p.group + a.heads - 1) / a.heads;
    const int64_t each = p.c.cu ? std::max<int64_t>(1, p.a.tokens / p.c.sequences) : p.a.tokens / p.c.sequences;
    const int most = each * a.heads <= 16 ? std::max(16, a.heads) : kFewRows;
    a.tokens = std::max(1, most / a.heads);
    if (!p.c.cu) a.tokens = static_cast<int>(std::min<int64_t>(a.tokens, each));
    a.rows = a.tokens * a.heads <= 16 ? 16 : 32;
    a.chunk = 128;
    while (p.c.page_size % a.chunk) a.chunk /= 2;
    return a;
}

int few_ctas(int sm_count) { return 2 * sm_count; }

}  // namespace

cudaError_t launch_join(const CattnArgs &a, int ctas, cudaStream_t s)
{
    return tc::launch_pdl(a.p.a.format == GN_FORMAT_BF16 ? join_kernel<__nv_bfloat16> : join_kernel<__half>,
                          dim3(static_cast<unsigned>(ctas)), dim3(128), 0, s, a);
}

}  // namespace cattn

size_t cached_attn_workspace_bytes(int64_t, int, int, int, int dim, int sm_count)
{
    return 4u * 2u * static_cast<size_t>(cattn::few_ctas(sm_count)) * cattn::kFewRows * static_cast<size_t>(2 + dim);
}

cudaError_t launch_cached_attn(const CachedAttn &p, int sm_count, const WaitLimit &limit, cudaStream_t s, int *launches)
{
    cattn::CattnArgs a = cattn::plan(p);
    a.limit = limit;
    a.pieces = static_cast<float *>(p.workspace);
    const gn_cache &c = p.c;
    CUtensorMap mk, mv;
    if (!cattn::encode_pool(&mk, c.k_pages, c, c.k_page, c.k_token, c.k_head, a.chunk) ||
        !cattn::encode_pool(&mv, c.v_pages, c, c.v_page, c.v_token, c.v_head, a.chunk))
        return cudaErrorInvalidValue;
    const int ctas = cattn::few_ctas(sm_count);
    cudaError_t e = cattn::launch_cached_few(a, mk, mv, ctas, s);
    if (e == cudaSuccess) ++*launches, e = cattn::launch_join(a, ctas, s);
    if (e == cudaSuccess) ++*launches;
    return e;
}

}  // namespace gn
