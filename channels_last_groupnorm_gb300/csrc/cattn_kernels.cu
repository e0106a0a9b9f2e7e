// cattn_kernels.cu -- attention of new tokens over the paged cache: the choice of a
// kernel, the tensor maps of the pages, and the kernel that joins pieces of tiles.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "cattn_common.cuh"

namespace gn {
namespace cattn {
namespace {

// Joins the pieces of the tiles that several CTAs shared.  A block looks after a
// tile that one CTA began, if others went on with it, and there after some of its rows: a
// warp each, or with many pieces all warps, each with some of the pieces (one token at 131072,
// 38 pieces of a tile: 26 us with a warp for a row).  Four channels a lane; every load of a
// row's outputs is on its way before the first is used.
//
// The first CTAs' blocks look after the kernel for few rows, the others after the one for many.
constexpr int kFewRows = 32;
constexpr int kJoinWarps = 8, kJoinMany = 8;

struct JoinBlocks {
    int few_ctas, few, tiles;     // blocks for a CTA of either kernel
};

template <typename T>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const __grid_constant__ CattnArgs few, const __grid_constant__ CattnArgs tiles, JoinBlocks j)
{
    __shared__ float4 sums[kJoinWarps][32];
    __shared__ float weights[kJoinWarps];
    tc::griddep_wait();
    if (threadIdx.x == 0) tc::griddep_launch_dependents();
    const int block = static_cast<int>(blockIdx.x) - j.few_ctas * j.few;
    const bool narrow = block < 0;
    const int blocks = narrow ? j.few : j.tiles;
    const int cta = (narrow ? blockIdx.x : block) / blocks;
    const int part = (narrow ? blockIdx.x : block) - cta * blocks;
    const CattnArgs &args = narrow ? few : tiles;
    const gn_cache &c = args.p.c;
    const gn_attn_cached_args &a = args.p.a;
    const Shared s = args.shared[cta];
    if (s.pieces <= 1 || *reinterpret_cast<volatile unsigned int *>(args.limit.status) != 0u) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool many = s.pieces > kJoinMany && narrow;      // (more rows keep the warps busy)
    const float *first = piece_of(args, cta, 1), *others = piece_of(args, cta, 0);
    const int64_t step = 2 * static_cast<int64_t>(args.rows) * (2 + c.dim);
    const auto piece = [&](int p) { return p == 0 ? first : others + p * step; };
    const int at = min(4 * lane, c.dim - 4);       // (lanes past the width read what another does)
    const int row0 = many ? part : part * kJoinWarps + warp, rows = many ? blocks : blocks * kJoinWarps;
    for (int row = row0; row < s.rows; row += rows) {
        const int i = row / args.heads, h = row - i * args.heads;
        const bool there = h < s.heads;            // (the same for all who share the row)
        float top = -INFINITY, sum = 0.f;
        for (int p = lane; p < s.pieces; p += 32) top = fmaxf(top, piece(p)[row]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        float4 out = make_float4(0.f, 0.f, 0.f, 0.f);
        const int p0 = many ? warp : 0, by = many ? kJoinWarps : 1;
        // (hardly more loads than there are pieces, two for most tiles: 64 and 64 tokens of 8 heads
        // over 5000 and 7000 keys 34 us, 37 with always eight)
        const auto add = [&](auto count) {
            constexpr int N = decltype(count)::value;
            for (int q = p0; q < s.pieces; q += N * by) {
                float4 v[N];
                float f[N], l[N];
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const int p = min(q + e * by, s.pieces - 1);
                    f[e] = piece(p)[row];
                    l[e] = q + e * by < s.pieces ? piece(p)[args.rows + row] : 0.f;
                    v[e] = *reinterpret_cast<const float4 *>(piece(p) + 2 * args.rows + row * c.dim + at);
                }
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    // (a part that saw nothing has a sum of zero)
                    if (l[e] == 0.f) continue;
                    const float g = ex2_approx(f[e] - top);
                    sum = fmaf(g, l[e], sum);
                    axpy4(out, g, v[e]);
                }
            }
        };
        if (s.pieces <= 2)
            add(std::integral_constant<int, 2>());
        else if (s.pieces <= 4)
            add(std::integral_constant<int, 4>());
        else
            add(std::integral_constant<int, 8>());
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
        const float inv = sum == 0.f ? 0.f : kSumDown / sum;
        const int64_t token = s.token + i, head = s.head + h;
        store4<T>(a.out, (token * a.heads + head) * c.dim, lane, c.dim, make_float4(out.x * inv, out.y * inv, out.z * inv, out.w * inv));
        if (lane == 0) a.lse[head * a.tokens + token] = sum == 0.f ? -INFINITY : (top + kSumUnit + log2f(sum)) * kLn2;
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

// The tiles of one kernel: 16 rows on the tensor core's narrow side (32 there took 195 us for
// four tokens of 8 heads each over 64 x 3000 keys, 177 as two tiles), or 256 on its wide side.
CattnArgs plan(const CachedAttn &p, bool few, int least, int most)
{
    CattnArgs a = {};
    a.p = p;
    // (a cap above every score there can be does nothing, one under fp32's step makes scores equal:
    // within these bounds its quotients and products are ordinary numbers)
    if (a.p.a.cap > 0.f) a.p.a.cap = std::min(std::max(a.p.a.cap, 0x1p-60f), 0x1p60f);
    a.scale_log2 = p.a.scale * kLog2e;
    a.least = least;
    a.most = most;
    a.rows = few ? kFewTile : kManyRows;
    a.heads = std::min(p.group, a.rows);
    a.chunks = (p.group + a.heads - 1) / a.heads;
    a.tokens = a.rows / a.heads;
    a.extra = few ? 4 : 8;
    a.chunk = kTile;
    while (p.c.page_size % a.chunk) a.chunk /= 2;
    return a;
}

// Join blocks for a CTA's tile.  There is one for each row that all its warps share, or for each
// eight rows with a warp of their own, where a tile comes in more than 8 pieces: where the tiles
// are few.  Where they are many most blocks have nothing to do, and a row more for a warp costs
// less than they do.  (8 heads of one token over 20000 keys: 21 us, 26 with 4 blocks; 64 and 64
// tokens of 8 heads over 5000 and 7000: 36 us, 48 with 16; 64 single tokens of 32 heads on 8 over
// 3000: 83 us, 89 with 16.)
int join_blocks(const CattnArgs &a, int ctas, bool few)
{
    const int rows = static_cast<int>(std::min<int64_t>(a.p.a.tokens, a.tokens)) * a.heads;
    const int64_t tiles = std::max<int64_t>(a.p.c.sequences, a.p.a.tokens / a.tokens) * a.p.c.kv_heads * a.chunks;
    const bool many = tiles * kJoinMany < ctas;
    if (few) return many ? rows : std::min(rows, 4);      // (a long sequence among many still has four)
    return many ? (rows + kJoinWarps - 1) / kJoinWarps : 16;
}

// How many of a sequence's tokens are few: up to 32 rows of a head.  (-1: none are in this call,
// INT_MAX: all.)  Only the device knows the counts where they differ, and each kernel then looks
// after its own sequences (a prompt of 2048 and 63 single tokens over 3000 keys each: 175 us, 275
// as tiles of 256 rows; 300 and 63: 108 us, 173 as tiles of 16; a kernel that finds none costs 7).
// Up to 64 rows in all are few: 3, 4, 4 and 5 tokens over 3000 keys 33 us, 38 otherwise, and at
// the worst, 15 and 1 of them over 60000 and 500, 103 us against 101.
int few_tokens(const CachedAttn &p)
{
    const int most = kFewRows / p.group;
    if (most == 0) return -1;
    if (!p.c.cu || p.c.sequences == 1) return p.a.tokens / p.c.sequences <= most ? INT_MAX : -1;
    return p.a.tokens * p.group <= 2 * kFewRows ? INT_MAX : most;
}

}  // namespace
}  // namespace cattn

namespace {

// The workspace: CTAs' words about tiles that are to be joined (two CTAs an SM for few rows, one
// for many), then the two kernels' pieces.
size_t shared_bytes(int sm_count) { return (3u * static_cast<size_t>(sm_count) * sizeof(cattn::Shared) + 255) / 256 * 256; }
size_t piece_bytes(int ctas, int rows, int dim) { return 4u * 2u * static_cast<size_t>(ctas) * static_cast<size_t>(rows) * static_cast<size_t>(2 + dim); }

}  // namespace

size_t cached_attn_workspace_bytes(int64_t, int, int, int, int dim, int sm_count)
{
    return shared_bytes(sm_count) + piece_bytes(2 * sm_count, cattn::kFewTile, dim) + piece_bytes(sm_count, cattn::kManyRows, dim);
}

cudaError_t launch_cached_attn(const CachedAttn &p, int sm_count, const WaitLimit &limit, cudaStream_t s, int *launches)
{
    const int most = cattn::few_tokens(p);
    cattn::CattnArgs few = cattn::plan(p, true, 0, most), tiles = cattn::plan(p, false, most == INT_MAX ? 0 : most + 1, INT_MAX);
    few.limit = tiles.limit = limit;
    few.shared = static_cast<cattn::Shared *>(p.workspace);
    tiles.shared = few.shared + 2 * sm_count;
    few.pieces = reinterpret_cast<float *>(static_cast<char *>(p.workspace) + shared_bytes(sm_count));
    tiles.pieces = few.pieces + piece_bytes(2 * sm_count, cattn::kFewTile, p.c.dim) / 4;
    const gn_cache &c = p.c;
    CUtensorMap mk, mv;
    if (!cattn::encode_pool(&mk, c.k_pages, c, c.k_page, c.k_token, c.k_head, few.chunk) ||
        !cattn::encode_pool(&mv, c.v_pages, c, c.v_page, c.v_token, c.v_head, few.chunk))
        return cudaErrorInvalidValue;
    const int few_ctas = most < 0 ? 0 : 2 * sm_count, tile_ctas = most == INT_MAX ? 0 : sm_count;
    cudaError_t e = cudaSuccess;
    if (tile_ctas) e = cattn::launch_cached_tiles(tiles, mk, mv, tile_ctas, s), *launches += e == cudaSuccess;
    if (e == cudaSuccess && few_ctas) e = cattn::launch_cached_few(few, mk, mv, few_ctas, s), *launches += e == cudaSuccess;
    const cattn::JoinBlocks j = {few_ctas, cattn::join_blocks(few, few_ctas, true), cattn::join_blocks(tiles, tile_ctas, false)};
    if (e == cudaSuccess)
        e = tc::launch_pdl(p.a.format == GN_FORMAT_BF16 ? cattn::join_kernel<__nv_bfloat16> : cattn::join_kernel<__half>,
                           dim3(static_cast<unsigned>(few_ctas * j.few + tile_ctas * j.tiles)), dim3(32 * cattn::kJoinWarps), 0, s, few,
                           tiles, j),
        *launches += e == cudaSuccess;
    return e;
}

}  // namespace gn
