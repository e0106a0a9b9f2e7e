// pattn_forward.cu -- packed attention's forward pass on the tensor cores.
//
// A CTA takes two tiles of 128 queries of one head (packed along the token
// axis, whatever documents they belong to: a query's keys are one run, so a
// tile's keys are the run from its queries' first to their last) and streams
// the keys and values in blocks of 128 through a ring of shared memory:
//   S_t = Q_t K^T            tcgen05, fp32 in tensor memory (128 columns a tile)
//   P_t = 2^(S_t c - m)      one query per thread of tile t's four warps; the
//                            half-precision weights go back to tensor memory,
//                            over the scores
//   O_t += P_t V             P from tensor memory, V read MN-major
// While the warps of one tile turn scores into weights, the tensor core works
// for the other.  m is a running maximum that only moves when a score is more
// than 2^8 above it (the weights stay below 2^8), which is when O and the row
// sum are rescaled; the row sum adds the unrounded weights, so lse is exact to
// fp32.  fp16 weights are kept 2^7 higher, away from its subnormals.
// Only blocks that some query of the tile sees in part are masked; there the
// values are also looked over for infinities and NaN (0 x NaN is not 0).
#include <algorithm>

#include "pattn_tiles.cuh"

namespace gn {

namespace {

using namespace pattn;

constexpr int kThreads = 384;    // warps: 0 loads, 1 MMA, 2 the MMA's waits, 4-7 and 8-11 the two tiles' softmax
constexpr int kStages = 4;       // ring of key and value tiles, in the order K0 V0 K1 V1 ...

// kPFull: per tile the weights of the block's first and last 64 keys
enum Bar { kQFull = 0, kFull = 2, kEmpty = kFull + kStages, kSFull = kEmpty + kStages, kPFull = kSFull + 2,
           kOFull = kPFull + 4, kDrain = kOFull + 2, kBars };

struct Layout {
    uint32_t q, ring, bars, words, total;
};

__host__ __device__ inline Layout layout(int halves)
{
    Layout l;
    const uint32_t tile = kHalfBytes * static_cast<uint32_t>(halves);
    l.q = 0;
    l.ring = 2 * tile;
    l.bars = l.ring + kStages * tile;
    l.words = l.bars + 8 * kBars;      // tensor-memory slot, abort, bad[2], 2 x 4 x 4 range words
    l.total = l.words + 4 * (4 + 32);
    return l;
}

template <typename T, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    attn_forward_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ CUtensorMap map_v, const __grid_constant__ TileArgs args)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *const gbase = smem_raw + (base - raw);
    const gn_attn_packed_args &a = args.p.a;
    const int halves = a.dim > 64 ? 2 : 1;
    const Layout lay = layout(halves);
    const uint32_t tile_bytes = kHalfBytes * static_cast<uint32_t>(halves);
    const auto bar = [&](int i) { return base + lay.bars + 8u * static_cast<uint32_t>(i); };
    volatile uint32_t *words = reinterpret_cast<volatile uint32_t *>(gbase + lay.words);
    volatile int *abort = reinterpret_cast<volatile int *>(words + 1);
    int *bad = reinterpret_cast<int *>(gbase + lay.words + 8);
    volatile int *range = reinterpret_cast<volatile int *>(words + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.x % a.heads, hk = h / args.p.group;
    // the last tiles first: with causal runs they have the most keys (without, a
    // document's length decides, which no order of the tiles knows)
    const int row0 = (args.tiles - 1 - static_cast<int>(blockIdx.x / a.heads)) * 2 * kTile;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kBars; ++i) mbar_init(bar(i), i >= kPFull && i < kPFull + 4 ? 4 : 1);
        *abort = (*reinterpret_cast<volatile unsigned int *>(args.limit.status) != 0u) ? 1 : 0;
        bad[0] = 0x7fffffff;
        bad[1] = -1;
        mbar_init_fence();
        prefetch_tensormap(&map_q);
        prefetch_tensormap(&map_k);
        prefetch_tensormap(&map_v);
    }
    if (warp == 1) {
        tmem_alloc(base + lay.words, 512);
        tmem_relinquish();
    }
    tc::griddep_wait();
    if (threadIdx.x == 0) tc::griddep_launch_dependents();

    // every query's run of keys, and what the tiles make of them: the keys that
    // any query sees, and those that all see
    Span span = {0, 0, 0};
    const int tile = warp >= 8 ? 1 : 0, row = row0 + tile * kTile + (warp & 3) * 32 + lane;
    if (warp >= 4) {
        span = query_span_warp(a, row, lane);
        const bool live = row < a.tokens_q, some = live && span.lo < span.hi;
        const int lo = __reduce_min_sync(0xffffffffu, some ? span.lo : 0x7fffffff);
        const int hi = __reduce_max_sync(0xffffffffu, some ? span.hi : 0);
        const int all_lo = __reduce_max_sync(0xffffffffu, !live ? 0 : (some ? span.lo : 0x7fffffff));
        const int all_hi = __reduce_min_sync(0xffffffffu, !live ? 0x7fffffff : (some ? span.hi : 0));
        if (lane == 0) {
            volatile int *w = range + ((warp - 4) * 4);
            w[0] = lo;
            w[1] = hi;
            w[2] = all_lo;
            w[3] = all_hi;
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = words[0];
    int key0 = 0x7fffffff, key1 = 0, lo[2], hi[2], all_lo = 0, all_hi = 0x7fffffff;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        lo[t] = 0x7fffffff;
        hi[t] = 0;
        for (int w = 0; w < 4; ++w) {
            volatile int *r = range + (t * 4 + w) * 4;
            lo[t] = min(lo[t], r[0]);
            hi[t] = max(hi[t], r[1]);
            if (t == tile) {
                all_lo = max(all_lo, r[2]);
                all_hi = min(all_hi, r[3]);
            }
        }
        key0 = min(key0, lo[t]);
        key1 = max(key1, hi[t]);
    }
    // blocks of 128 keys from key0; tile t works on blocks [first[t], last[t])
    int first[2], last[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        first[t] = lo[t] < hi[t] ? (lo[t] - key0) / kTile : 0;
        last[t] = lo[t] < hi[t] ? (hi[t] - key0 + kTile - 1) / kTile : 0;
    }
    const int blocks = key0 < key1 ? (key1 - key0 + kTile - 1) / kTile : 0;
    const bool skip = *abort != 0;

    if (warp >= 4) {
        many_registers();
        // ---- softmax: one query per thread ----
        constexpr float kShift = weight_shift<T>();
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + 128 * tile, to = tmem + lanes + 256 + 128 * tile;
        const int b0 = tile ? first[1] : first[0], b1 = tile ? last[1] : last[0];
        const float slope2 = (MODE & kBias) && a.slopes ? __ldg(a.slopes + h) * kLog2e : 0.f;
        float m = -INFINITY, l = 0.f;
        bool go = !skip;
        for (int b = b0; go && b < b1; ++b) {
            const int j0 = key0 + b * kTile;
            const bool masked = j0 < all_lo || j0 + kTile > all_hi;
            go = wait_warp(bar(kSFull + tile), (b - b0) & 1, abort, args.limit);
            if (!go) break;
            tc_fence_after_sync();
            float s[kTile];
            tmem_ld_all(ts, s);
            const float c = bend_scores<MODE>(s, a, args.scale_log2, slope2, span.pos - j0);
            if (masked) mask_scores(s, span.lo - j0, static_cast<unsigned>(max(0, span.hi - span.lo)));
            const float mx = top_score(s) * c;
            const bool grew = mx > m + (kShift + kRescaleLog2) || (b == b0 && mx > m);
            if (__any_sync(0xffffffffu, grew)) {
                const float to_m = grew ? mx - kShift : m;
                const float f = grew && m != -INFINITY ? ex2_approx(m - to_m) : 1.0f;
                m = to_m;
                l *= f;
                if (b > b0) rescale_columns(to, f);
            }
            // the weights, 32 keys at a time; the first 64 are handed over early
            const float m_use = m == -INFINITY ? 0.f : m;
            const uint64_t c2 = pack2(c, c), m2 = pack2(-m_use, -m_use);
            uint64_t sum2[2] = {0, 0};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t pk[16];
                weigh_32<T>(s + 32 * q, c2, m2, sum2, pk);
                tmem_st16(ts + 16 * q, pk);
                if (q == 1 && !masked) {
                    tmem_wait_st();
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kPFull + 2 * tile));
                }
            }
            const float2 sums = unpack2(add2(sum2[0], sum2[1]));
            l += sums.x + sums.y;
            if (masked) {
                const int nv = 2 * b + 1, r = (warp & 3) * 32 + lane;
                go = wait_warp(bar(kFull + nv % kStages), (nv / kStages) & 1, abort, args.limit);
                if (go)
                    clear_not_finite<T>(base + lay.ring + (nv % kStages) * tile_bytes, r, j0 + r, key0, key1, halves, bad);
            }
            tmem_wait_st();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                if (masked) mbar_arrive(bar(kPFull + 2 * tile));   // (not before the values were looked over)
                mbar_arrive(bar(kPFull + 2 * tile + 1));
            }
        }
        if (b0 < b1 && go) go = wait_warp(bar(kOFull + tile), 0, abort, args.limit);
        named_sync(1, 256);   // both tiles are done with looking at the values
        if (go) {
            tc_fence_after_sync();
            const float inv = l == 0.f ? 0.f : 1.0f / l;
            T *dst = static_cast<T *>(a.out) + (static_cast<int64_t>(row) * a.heads + h) * a.dim;
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
                if (32 * q >= a.dim) break;
                float o[32];
                if (b0 < b1) {
                    tmem_ld32(to + 32 * q, o);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int ch = 32 * q + 8 * k;
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = l == 0.f ? 0u : Half2<T>::pack(o[8 * k + 2 * e] * inv, o[8 * k + 2 * e + 1] * inv);
                    if (row < a.tokens_q && ch < a.dim)
                        *reinterpret_cast<uint4 *>(dst + ch) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            if (row < a.tokens_q)
                a.lse[static_cast<int64_t>(h) * a.tokens_q + row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
            // queries that see a value row which was cleared
            __syncwarp();
            unsigned again = __ballot_sync(0xffffffffu, row < a.tokens_q && span.lo < span.hi && span.lo <= bad[1] &&
                                                            span.hi > bad[0]);
            for (; again; again &= again - 1) {
                const int n = __ffs(again) - 1;
                const int j0 = max(__shfl_sync(0xffffffffu, span.lo, n), bad[0]);
                const int j1 = min(__shfl_sync(0xffffffffu, span.hi, n), bad[1] + 1);
                if (any_not_finite<T>(a.v, a.v_token, hk * a.v_head, j0, j1, a.dim))
                    row_forward<T>(a, args.p.group, row - lane + n, h);
            }
        }
        tc_fence_before_sync();
    } else {
        few_registers();
        if (warp == 0) {
            if (lane == 0 && !skip) {
                // ---- loads ----
                for (int t = 0; t < 2; ++t)
                    if (first[t] < last[t]) {
                        mbar_arrive_expect_tx(bar(kQFull + t), tile_bytes);
                        load_tile(base + lay.q + t * tile_bytes, &map_q, halves, h, row0 + t * kTile, bar(kQFull + t));
                    }
                int n = 0;
                bool go = true;
                for (; go && n < 2 * blocks; ++n) {
                    const int st = n % kStages;
                    if (n >= kStages && !wait(bar(kEmpty + st), (n / kStages - 1) & 1, abort, args.limit)) {
                        go = false;
                        break;
                    }
                    mbar_arrive_expect_tx(bar(kFull + st), tile_bytes);
                    load_tile(base + lay.ring + st * tile_bytes, (n & 1) ? &map_v : &map_k, halves, hk,
                              key0 + (n >> 1) * kTile, bar(kFull + st));
                }
                // nothing is left in flight when the CTA ends, whatever became of the others
                for (int k = max(0, n - kStages); k < n; ++k)
                    tc::drain(bar(kFull + k % kStages), (k / kStages) & 1, args.limit.timeout_ns);
                for (int t = 0; t < 2; ++t)
                    if (first[t] < last[t]) tc::drain(bar(kQFull + t), 0, args.limit.timeout_ns);
            }
        } else if (warp == 1 || warp == 2) {
            if (!skip) {
                // ---- MMA: per block and tile the weighted values of the block
                // before, then the scores of this one ----
                const bool waits = warp == 2;
                const int steps = (a.dim + 15) / 16;
                const uint32_t is = instruction<T>(kTile, false), io = instruction<T>(steps * 16, true);
                const auto loaded = [&](int n) { wait_warp(bar(kFull + n % kStages), (n / kStages) & 1, abort, args.limit); };
                for (int b = 0; b <= blocks; ++b) {
                    const int nv = 2 * b - 1, nk = 2 * b;
                    const uint32_t v_tile = base + lay.ring + (nv % kStages) * tile_bytes;
                    const uint32_t k_tile = base + lay.ring + (nk % kStages) * tile_bytes;
                    // (a tile may have no part in a block: its loads are waited for all the same)
                    if (waits) {
                        if (b > 0) loaded(nv);
                        if (b < blocks) loaded(nk);
                    }
    #pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const bool weigh = b - 1 >= first[t] && b - 1 < last[t], score = b >= first[t] && b < last[t];
                        if (weigh) {
    #pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                if (waits) wait_warp(bar(kPFull + 2 * t + half), (b - 1 - first[t]) & 1, abort, args.limit);
                                hand_over();
                                if (waits) continue;
                                tc_fence_after_sync();
                                mma_channels(tmem + 256 + 128 * t, tmem + 128 * t + 32 * half, v_tile, half, io,
                                             b - 1 > first[t] || half);
                            }
                            if (!waits && b == last[t]) commit(bar(kOFull + t));
                        }
                        if (score) {
                            if (waits && b == first[t]) wait_warp(bar(kQFull + t), 0, abort, args.limit);
                            if (!weigh) hand_over();
                            if (waits) continue;
                            mma_tokens(tmem + 128 * t, base + lay.q + t * tile_bytes, k_tile, steps, is);
                            commit(bar(kSFull + t));
                        }
                    }
                    hand_over();
                    if (!waits) {
                        if (b > 0) commit(bar(kEmpty + nv % kStages));
                        if (b < blocks) commit(bar(kEmpty + nk % kStages));
                    }
                }
                if (!waits) {
                    commit(bar(kDrain));
                    tc::drain(bar(kDrain), 0, args.limit.timeout_ns);
                }
            }
        }
    }
    __syncwarp();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

template <typename T, int MODE>
cudaError_t launch(const TileArgs &args, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                   cudaStream_t s)
{
    const int halves = args.p.a.dim > 64 ? 2 : 1;
    const size_t smem = layout(halves).total + 1024;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_shared(reinterpret_cast<const void *>(attn_forward_kernel<T, MODE>),
                                       layout(2).total + 1024, done);
    if (e != cudaSuccess) return e;
    const int64_t grid = static_cast<int64_t>(args.tiles) * args.p.a.heads;
    return tc::launch_pdl(attn_forward_kernel<T, MODE>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), smem, s, mq,
                          mk, mv, args);
}

template <typename T>
cudaError_t launch_mode(int mode, const TileArgs &args, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                        cudaStream_t s)
{
    if (mode == 0) return launch<T, 0>(args, mq, mk, mv, s);
    if (mode == kCap) return launch<T, kCap>(args, mq, mk, mv, s);
    if (mode == kBias) return launch<T, kBias>(args, mq, mk, mv, s);
    return launch<T, kCap | kBias>(args, mq, mk, mv, s);
}

}  // namespace

cudaError_t launch_packed_attn_tiles(const PackedAttn &p, const WaitLimit &limit, cudaStream_t s)
{
    const gn_attn_packed_args &a = p.a;
    const bool bf16 = a.format == GN_FORMAT_BF16;
    CUtensorMap mq, mk, mv;
    if (!encode_heads(&mq, a.q, bf16, a.tokens_q, a.q_token, a.heads, a.q_head, a.dim) ||
        !encode_heads(&mk, a.k, bf16, a.tokens_k, a.k_token, a.kv_heads, a.k_head, a.dim) ||
        !encode_heads(&mv, a.v, bf16, a.tokens_k, a.v_token, a.kv_heads, a.v_head, a.dim))
        return cudaErrorInvalidValue;
    TileArgs args = {};
    args.p = p;
    args.scale_log2 = a.scale * kLog2e;
    args.limit = limit;
    args.tiles = static_cast<int>((a.tokens_q + 2 * kTile - 1) / (2 * kTile));
    const int mode = score_mode(a);
    return bf16 ? launch_mode<__nv_bfloat16>(mode, args, mq, mk, mv, s) : launch_mode<__half>(mode, args, mq, mk, mv, s);
}

}  // namespace gn
