// pattn_split.cu -- packed attention for few queries per document (single new
// tokens beside a cache, short chunks), on the tensor cores.
//
// Such a call is bound by reading the keys and values once (4 bytes per key,
// head and channel at the memory's rate), so
//  * a tile's 128 rows are the query heads that share a key / value head, times
//    a few neighbouring tokens: all of them meet the same keys, which are read
//    once for all;
//  * the keys are split between the CTAs of a cluster (up to 16), each with
//    its own blocks of 128, and the parts are joined over distributed shared
//    memory at the end: one launch, no workspace;
//  * two CTAs share an SM where their shared memory lets them (plan), so that
//    one's start, softmax or end is covered by the other's loads.
// Two kernels, by the number of rows:
//  * up to 32 (attn_few_kernel): the keys are the accumulator's lanes and the
//    rows its columns, S^T = K Q^T and O^T += V^T P^T, so that every thread of
//    the softmax warps has a key, and a block costs a thread as many
//    exponentials as there are rows.
//  * more (attn_split_kernel): as in the kernel for long runs of queries, one
//    row per thread and 128 keys each.  With 4 rows, 4 lanes of one warp would do
//    128 exponentials each: 1.5 us for a block that takes 0.35 us to load (85 us
//    against 75 us for 24 single tokens over caches of up to 8000 keys).
// Rows past the tile's count read whatever lies there; nobody reads what becomes
// of them.
#include <algorithm>

#include "pattn_tiles.cuh"

namespace gn {
namespace {

using namespace pattn;

constexpr int kThreads = 256;   // warps: 0 loads, 1 MMA, 2 the MMA's waits, 4-7 softmax
constexpr int kMaxStages = 5;
constexpr int kMaxSplits = 16;

struct SplitArgs {
    PackedAttn p;
    float scale_log2;
    WaitLimit limit;
    int tokens, heads, chunks;    // of a tile: its tokens, its query heads; chunks of heads per key / value head
    int splits, stages;
};

enum Bar { kQ = 0, kFull, kEmpty = kFull + kMaxStages, kS = kEmpty + kMaxStages, kP, kO, kDrain, kBars };

struct Layout {
    uint32_t q, q_half, ring, stats, bars, words, total;
};

__host__ __device__ inline Layout layout(int halves, int rows, int stages)
{
    Layout l;
    const uint32_t tile = kHalfBytes * static_cast<uint32_t>(halves);
    l.q = 0;
    l.q_half = static_cast<uint32_t>((rows + 7) / 8) * 1024u;
    l.ring = l.q_half * static_cast<uint32_t>(halves);
    l.stats = l.ring + static_cast<uint32_t>(stages) * tile;    // 128 row maxima, 128 row sums
    l.bars = l.stats + 2 * kTile * 4;
    l.words = l.bars + 8 * kBars;                               // tensor-memory slot, abort, bad[2], 4 x 4 range words
    l.total = l.words + 4 * (4 + 16);
    return l;
}

// The end of either kernel: the cluster's parts (per row a maximum and a sum at
// `stats`, unnormalised outputs [rows][dim] at `parts`, first and last cleared
// key at `cleared`) joined, every CTA writing some of the channels; then the
// rows that see a value row which any CTA cleared, one by one.  `live`, `span`:
// of row r, held by the threads of warps 4 on.
template <typename T>
__device__ __forceinline__ void join_parts(const SplitArgs &args, uint32_t stats, uint32_t parts, uint32_t cleared,
                                           bool failed, int split, int token0, int hk, int first_head, bool live, Span span,
                                           int r)
{
    const gn_attn_packed_args &a = args.p.a;
    const int rows = args.tokens * args.heads, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (args.splits > 1) cluster_sync_all();
    if (!failed) {
        for (int n = split * kThreads + static_cast<int>(threadIdx.x); n < rows * a.dim; n += args.splits * kThreads) {
            const int row = n / a.dim, c = n - row * a.dim;
            const int token = token0 + row / args.heads, g = first_head + row % args.heads;
            if (token >= a.tokens_q || g >= args.p.group) continue;
            // (all the peers' values are asked for before the first is used)
            float ms[kMaxSplits], ls[kMaxSplits], vs[kMaxSplits];
#pragma unroll
            for (int s = 0; s < kMaxSplits; ++s) {
                ms[s] = -INFINITY;
                ls[s] = vs[s] = 0.f;
                if (s < args.splits) {
                    ms[s] = peer_float(stats + 4u * row, s);
                    ls[s] = peer_float(stats + 4u * (kTile + row), s);
                    vs[s] = peer_float(parts + 4u * static_cast<uint32_t>(n), s);
                }
            }
            float top = -INFINITY, sum = 0.f, v = 0.f;
#pragma unroll
            for (int s = 0; s < kMaxSplits; ++s) top = fmaxf(top, ms[s]);
#pragma unroll
            for (int s = 0; s < kMaxSplits; ++s) {
                // (a part that saw nothing has a sum of zero, and may have written no outputs)
                const float f = ls[s] == 0.f ? 0.f : ex2_approx(ms[s] - top);
                sum = fmaf(f, ls[s], sum);
                v += ls[s] == 0.f ? 0.f : f * vs[s];
            }
            const int head = hk * args.p.group + g;
            static_cast<T *>(a.out)[(static_cast<int64_t>(token) * a.heads + head) * a.dim + c] =
                static_cast<T>(sum == 0.f ? 0.f : v / sum);
            if (c == 0)
                a.lse[static_cast<int64_t>(head) * a.tokens_q + token] =
                    sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
        }
    }
    int bad_lo = 0x7fffffff, bad_hi = -1;
    if (split == 0 && warp >= 4 && lane < args.splits) {
        bad_lo = __float_as_int(peer_float(cleared, lane));
        bad_hi = __float_as_int(peer_float(cleared + 4, lane));
    }
    bad_lo = __reduce_min_sync(0xffffffffu, bad_lo);
    bad_hi = __reduce_max_sync(0xffffffffu, bad_hi);
    if (args.splits > 1)
        cluster_sync_all();      // a CTA's parts stay until every peer has read them
    else
        __syncthreads();
    if (split == 0 && warp >= 4 && !failed) {
        unsigned again = __ballot_sync(0xffffffffu, live && span.lo < span.hi && span.lo <= bad_hi && span.hi > bad_lo);
        for (; again; again &= again - 1) {
            const int n = __ffs(again) - 1, row = r - lane + n;
            const int j0 = max(__shfl_sync(0xffffffffu, span.lo, n), bad_lo);
            const int j1 = min(__shfl_sync(0xffffffffu, span.hi, n), bad_hi + 1);
            if (!any_not_finite<T>(a.v, a.v_token, hk * a.v_head, j0, j1, a.dim)) continue;
            row_forward<T>(a, args.p.group, token0 + row / args.heads, hk * args.p.group + first_head + row % args.heads);
        }
    }
}

template <typename T, int MODE>
__global__ void __launch_bounds__(kThreads, 2)
    attn_split_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_v, const __grid_constant__ SplitArgs args)
{
    extern __shared__ __align__(1024) uint8_t gbase[];
    const uint32_t base = smem_addr(gbase);
    const gn_attn_packed_args &a = args.p.a;
    const int halves = a.dim > 64 ? 2 : 1, rows = args.tokens * args.heads;
    const Layout lay = layout(halves, rows, args.stages);
    const uint32_t tile_bytes = kHalfBytes * static_cast<uint32_t>(halves);
    const auto bar = [&](int i) { return base + lay.bars + 8u * static_cast<uint32_t>(i); };
    const auto stage = [&](int n) { return base + lay.ring + static_cast<uint32_t>(n % args.stages) * tile_bytes; };
    volatile uint32_t *words = reinterpret_cast<volatile uint32_t *>(gbase + lay.words);
    volatile int *abort = reinterpret_cast<volatile int *>(words + 1);
    int *bad = reinterpret_cast<int *>(gbase + lay.words + 8);
    volatile int *range = reinterpret_cast<volatile int *>(words + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // splits innermost (a cluster), then the heads: CTAs that run at the same time
    // read the same tokens, whose heads lie next to each other
    const int split = static_cast<int>(blockIdx.x) % args.splits, part = static_cast<int>(blockIdx.x) / args.splits;
    const int parts = a.kv_heads * args.chunks, token0 = part / parts * args.tokens;
    const int hk = part % parts / args.chunks, first_head = part % args.chunks * args.heads;   // within the group

    if (threadIdx.x == 0) {
        for (int i = 0; i < kBars; ++i) mbar_init(bar(i), i == kP ? 4 : 1);
        *abort = (*reinterpret_cast<volatile unsigned int *>(args.limit.status) != 0u) ? 1 : 0;
        bad[0] = 0x7fffffff;
        bad[1] = -1;
        mbar_init_fence();
        prefetch_tensormap(&map_q);
        prefetch_tensormap(&map_k);
        prefetch_tensormap(&map_v);
    }
    if (warp == 1) {
        tmem_alloc(base + lay.words, 256);
        tmem_relinquish();
    }
    tc::griddep_wait();

    const int r = (warp & 3) * 32 + lane, i = token0 + r / args.heads, g = first_head + r % args.heads;
    const int h = hk * args.p.group + g;
    const bool live = warp >= 4 && r < rows && i < a.tokens_q && g < args.p.group;
    Span span = {0, 0, 0};
    if (warp >= 4) {
        span = query_span_warp(a, i, lane);
        const bool some = live && span.lo < span.hi;
        const int lo = __reduce_min_sync(0xffffffffu, some ? span.lo : 0x7fffffff);
        const int hi = __reduce_max_sync(0xffffffffu, some ? span.hi : 0);
        const int all_lo = __reduce_max_sync(0xffffffffu, !live ? 0 : (some ? span.lo : 0x7fffffff));
        const int all_hi = __reduce_min_sync(0xffffffffu, !live ? 0x7fffffff : (some ? span.hi : 0));
        if (lane == 0) {
            volatile int *w = range + (warp - 4) * 4;
            w[0] = lo;
            w[1] = hi;
            w[2] = all_lo;
            w[3] = all_hi;
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    // (only now: a kernel that starts early must not find tensor memory that a
    // CTA of this one has yet to take)
    if (threadIdx.x == 0) tc::griddep_launch_dependents();
    const uint32_t tmem = words[0];
    int key0 = 0x7fffffff, key1 = 0, all_lo = 0, all_hi = 0x7fffffff;
    for (int w = 0; w < 4; ++w) {
        key0 = min(key0, range[4 * w]);
        key1 = max(key1, range[4 * w + 1]);
        all_lo = max(all_lo, range[4 * w + 2]);
        all_hi = min(all_hi, range[4 * w + 3]);
    }
    // this CTA's blocks [b0, b1) of the tile's
    const int total = key0 < key1 ? (key1 - key0 + kTile - 1) / kTile : 0;
    const int share = (total + args.splits - 1) / args.splits;
    const int b0 = min(total, split * share), b1 = min(total, b0 + share), blocks = b1 - b0;
    const bool skip = *abort != 0;
    const int k_first = key0 + b0 * kTile;     // (of no use without blocks)
    const uint32_t t_s = tmem, t_o = tmem + 128;
    float m = -INFINITY, l = 0.f;

    if (warp == 0) {
        if (lane == 0 && !skip && blocks > 0) {
            mbar_arrive_expect_tx(bar(kQ), static_cast<uint32_t>(rows * halves) * 128u);
            for (int n = 0; n < halves; ++n)
                tma_load_3d(base + lay.q + n * lay.q_half, &map_q, n * 64, hk * args.p.group + first_head, token0, bar(kQ));
            int n = 0;
            for (; n < 2 * blocks; ++n) {
                const int st = n % args.stages;
                if (n >= args.stages && !wait(bar(kEmpty + st), (n / args.stages - 1) & 1, abort, args.limit)) break;
                mbar_arrive_expect_tx(bar(kFull + st), tile_bytes);
                load_tile(stage(n), (n & 1) ? &map_v : &map_k, halves, hk, k_first + (n >> 1) * kTile, bar(kFull + st));
            }
            // nothing is left in flight when the CTA goes on, whatever became of the others
            for (int k = max(0, n - args.stages); k < n; ++k)
                tc::drain(bar(kFull + k % args.stages), (k / args.stages) & 1, args.limit.timeout_ns);
            tc::drain(bar(kQ), 0, args.limit.timeout_ns);
        }
        __syncwarp();
    } else if (warp == 1 || warp == 2) {
        if (!skip && blocks > 0) {
            const bool waits = warp == 2;
            const int steps = (a.dim + 15) / 16;
            const uint32_t is = instruction<T>(kTile, false), io = instruction<T>(steps * 16, true);
            const auto loaded = [&](int n) {
                wait_warp(bar(kFull + n % args.stages), (n / args.stages) & 1, abort, args.limit);
            };
            if (waits) wait_warp(bar(kQ), 0, abort, args.limit);
            for (int b = 0; b < blocks; ++b) {
                if (waits) loaded(2 * b);
                hand_over();
                if (!waits) {
                    mma_tokens(t_s, base + lay.q, stage(2 * b), steps, is, lay.q_half);
                    commit(bar(kS));
                    commit(bar(kEmpty + 2 * b % args.stages));
                }
                if (waits) {
                    loaded(2 * b + 1);
                    wait_warp(bar(kP), b & 1, abort, args.limit);
                }
                hand_over();
                if (!waits) {
                    tc_fence_after_sync();
                    mma_channels(t_o, t_s, stage(2 * b + 1), 0, io, b > 0);
                    mma_channels(t_o, t_s + 64, stage(2 * b + 1), 1, io, true);
                    commit(bar(kEmpty + (2 * b + 1) % args.stages));
                }
            }
            if (!waits) {
                commit(bar(kO));
                commit(bar(kDrain));
                tc::drain(bar(kDrain), 0, args.limit.timeout_ns);
            }
        }
    } else if (warp >= 4 && !skip) {
        constexpr float kShift = weight_shift<T>();
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = t_s + lanes, to = t_o + lanes;
        const bool busy = (warp & 3) * 32 < rows;    // has any row
        const float slope2 = (MODE & kBias) && a.slopes && live ? __ldg(a.slopes + h) * kLog2e : 0.f;
        for (int b = 0; b < blocks; ++b) {
            const int j0 = k_first + b * kTile;
            const bool masked = j0 < all_lo || j0 + kTile > all_hi;
            // (a wait that ran out sets the abort flag: the later ones return at
            // once, and nothing is written at the end)
            wait_warp(bar(kS), b & 1, abort, args.limit);
            tc_fence_after_sync();
            if (busy) {
                // the scores of one half of the keys at a time, twice: their
                // maximum first, then (the second half still at hand) the weights
                float s[64], c = 1.0f;
                const auto scores = [&](int q) {
                    tmem_ld_all(ts + 64 * q, s);
                    c = bend_scores<MODE>(s, a, args.scale_log2, slope2, span.pos - j0 - 64 * q);
                    if (masked) mask_scores(s, span.lo - j0 - 64 * q, static_cast<unsigned>(max(0, span.hi - span.lo)));
                };
                scores(0);
                float mx = top_score(s);
                scores(1);
                mx = fmaxf(mx, top_score(s)) * c;
                const bool grew = mx > m + (kShift + kRescaleLog2) || (b == 0 && mx > m);
                if (__any_sync(0xffffffffu, grew)) {
                    const float top = grew ? mx - kShift : m;
                    const float f = grew && m != -INFINITY ? ex2_approx(m - top) : 1.0f;
                    m = top;
                    l *= f;
                    if (b > 0) rescale_columns(to, f);
                }
                const float m_use = m == -INFINITY ? 0.f : m;
                const uint64_t c2 = pack2(c, c), m2 = pack2(-m_use, -m_use);
                uint64_t sum2[2] = {0, 0};
#pragma unroll 1
                for (int q = 1; q >= 0; --q) {
                    if (q == 0) scores(0);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t pk[16];
                        weigh_32<T>(s + 32 * e, c2, m2, sum2, pk);
                        tmem_st16(ts + 64 * q + 16 * e, pk);
                    }
                }
                const float2 sums = unpack2(add2(sum2[0], sum2[1]));
                l += sums.x + sums.y;
            }
            if (masked) {
                const int nv = 2 * b + 1;
                wait_warp(bar(kFull + nv % args.stages), (nv / args.stages) & 1, abort, args.limit);
                clear_not_finite<T>(stage(nv), r, j0 + r, key0, key1, halves, bad);
            }
            tmem_wait_st();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kP));
        }
        if (blocks > 0) wait_warp(bar(kO), 0, abort, args.limit);
        tc_fence_after_sync();
        // (the ring is free: every product is done; a failed call reads nothing of it)
        if (blocks > 0 && busy) {
            float *o = reinterpret_cast<float *>(gbase + lay.ring) + static_cast<int64_t>(r) * a.dim;
            for (int q = 0; 32 * q < a.dim; ++q) {
                float v[32];
                tmem_ld32(to + 32 * q, v);
                tmem_wait_ld();
                if (r < rows)
#pragma unroll
                    for (int k = 0; k < 32; k += 4)
                        if (32 * q + k < a.dim)
                            *reinterpret_cast<float4 *>(o + 32 * q + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
            }
        }
        float *stats = reinterpret_cast<float *>(gbase + lay.stats);
        stats[r] = m;
        stats[kTile + r] = l;
        tc_fence_before_sync();
    }
    __syncwarp();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 256);
    }
    __syncwarp();
    join_parts<T>(args, base + lay.stats, base + lay.ring, base + lay.words + 8, *abort != 0, split, token0, hk, first_head,
                  live, span, r);
}

// ---------------------------------------------------------------------------
// up to N = 16 or 32 rows: keys on the lanes
// ---------------------------------------------------------------------------
struct FewLayout {
    uint32_t q, weights, ring, info, stats, tops, bars, words, total;
};

__host__ __device__ inline FewLayout few_layout(int halves, int n, int stages)
{
    FewLayout l;
    const uint32_t tile = kHalfBytes * static_cast<uint32_t>(halves), rows = static_cast<uint32_t>(n) * 128u;
    l.q = 0;                                    // [halves][n][64 channels]
    l.weights = l.q + 2 * rows;                 // [2][n][64 keys], swizzled like a tile
    l.ring = l.weights + 2 * rows;
    // (with one half of channels the product with V reads another half past the last tile)
    l.info = l.ring + static_cast<uint32_t>(stages) * tile + (halves == 1 ? kHalfBytes : 0u);
    l.stats = l.info + static_cast<uint32_t>(n) * 16u;          // n runs of keys and slopes
    l.tops = l.stats + 2 * kTile * 4;                           // 4 x n row maxima (or sums) of a warp
    l.bars = l.tops + 4u * static_cast<uint32_t>(n) * 4u;
    l.words = l.bars + 8 * kBars;
    l.total = l.words + 4 * (4 + 16);
    return l;
}

// An order-preserving whole number of a float, for the warp-wide maximum.
__device__ __forceinline__ int ordered(float v)
{
    const int i = __float_as_int(v);
    return i >= 0 ? i : i ^ 0x7fffffff;
}
__device__ __forceinline__ float from_ordered(int i) { return __int_as_float(i >= 0 ? i : i ^ 0x7fffffff); }

template <int N>
__device__ __forceinline__ void tmem_ld_rows(uint32_t taddr, float (&v)[N])
{
#pragma unroll
    for (int q = 0; q < N / 16; ++q) {
        uint32_t u[16];
        tmem_ld16(taddr + 16 * q, u);
#pragma unroll
        for (int k = 0; k < 16; ++k) v[16 * q + k] = __uint_as_float(u[k]);
    }
    tmem_wait_ld();
}

template <typename T, int MODE, int N>
__global__ void __launch_bounds__(kThreads, 2)
    attn_few_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                    const __grid_constant__ CUtensorMap map_v, const __grid_constant__ SplitArgs args)
{
    extern __shared__ __align__(1024) uint8_t gbase[];
    const uint32_t base = smem_addr(gbase);
    const gn_attn_packed_args &a = args.p.a;
    const int halves = a.dim > 64 ? 2 : 1, rows = args.tokens * args.heads;
    const FewLayout lay = few_layout(halves, N, args.stages);
    const uint32_t tile_bytes = kHalfBytes * static_cast<uint32_t>(halves), n_bytes = N * 128u;
    const auto bar = [&](int i) { return base + lay.bars + 8u * static_cast<uint32_t>(i); };
    const auto stage = [&](int n) { return base + lay.ring + static_cast<uint32_t>(n % args.stages) * tile_bytes; };
    volatile uint32_t *words = reinterpret_cast<volatile uint32_t *>(gbase + lay.words);
    volatile int *abort = reinterpret_cast<volatile int *>(words + 1);
    int *bad = reinterpret_cast<int *>(gbase + lay.words + 8);
    volatile int *range = reinterpret_cast<volatile int *>(words + 4);
    int4 *info = reinterpret_cast<int4 *>(gbase + lay.info);
    float *tops = reinterpret_cast<float *>(gbase + lay.tops);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // splits innermost (a cluster), then the heads: CTAs that run at the same time
    // read the same tokens, whose heads lie next to each other
    const int split = static_cast<int>(blockIdx.x) % args.splits, part = static_cast<int>(blockIdx.x) / args.splits;
    const int parts = a.kv_heads * args.chunks, token0 = part / parts * args.tokens;
    const int hk = part % parts / args.chunks, first_head = part % args.chunks * args.heads;   // within the group

    if (threadIdx.x == 0) {
        for (int i = 0; i < kBars; ++i) mbar_init(bar(i), i == kP ? 4 : 1);
        *abort = (*reinterpret_cast<volatile unsigned int *>(args.limit.status) != 0u) ? 1 : 0;
        bad[0] = 0x7fffffff;
        bad[1] = -1;
        mbar_init_fence();
        prefetch_tensormap(&map_q);
        prefetch_tensormap(&map_k);
        prefetch_tensormap(&map_v);
    }
    if (warp == 1) {
        tmem_alloc(base + lay.words, 64);
        tmem_relinquish();
    }
    tc::griddep_wait();

    // the rows (of which the first warp of four has all)
    const int r = (warp & 3) * 32 + lane, i = token0 + r / args.heads, g = first_head + r % args.heads;
    const int h = hk * args.p.group + g;
    const bool live = warp >= 4 && r < rows && i < a.tokens_q && g < args.p.group;
    Span span = {0, 0, 0};
    if (warp == 4) {
        span = query_span_warp(a, i, lane);
        const bool some = live && span.lo < span.hi;
        if (!some) span.lo = span.hi = 0;
        if (r < N)
            info[r] = make_int4(span.lo, span.hi, span.pos,
                                __float_as_int((MODE & kBias) && a.slopes && live ? __ldg(a.slopes + h) * kLog2e : 0.f));
        const int lo = __reduce_min_sync(0xffffffffu, some ? span.lo : 0x7fffffff);
        const int hi = __reduce_max_sync(0xffffffffu, some ? span.hi : 0);
        const int all_lo = __reduce_max_sync(0xffffffffu, !live ? 0 : (some ? span.lo : 0x7fffffff));
        const int all_hi = __reduce_min_sync(0xffffffffu, !live ? 0x7fffffff : (some ? span.hi : 0));
        if (lane == 0) {
            range[0] = lo;
            range[1] = hi;
            range[2] = all_lo;
            range[3] = all_hi;
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    // (only now: a kernel that starts early must not find tensor memory that a
    // CTA of this one has yet to take)
    if (threadIdx.x == 0) tc::griddep_launch_dependents();
    const uint32_t tmem = words[0], t_s = tmem, t_o = tmem + 32;
    const int key0 = range[0], key1 = range[1], all_lo = range[2], all_hi = range[3];
    // this CTA's blocks [b0, b1) of the tile's
    const int total = key0 < key1 ? (key1 - key0 + kTile - 1) / kTile : 0;
    const int share = (total + args.splits - 1) / args.splits;
    const int b0 = min(total, split * share), b1 = min(total, b0 + share), blocks = b1 - b0;
    const bool skip = *abort != 0;
    const int k_first = key0 + b0 * kTile;     // (of no use without blocks)

    if (warp == 0) {
        if (lane == 0 && !skip && blocks > 0) {
            mbar_arrive_expect_tx(bar(kQ), static_cast<uint32_t>(rows * halves) * 128u);
            for (int n = 0; n < halves; ++n)
                tma_load_3d(base + lay.q + n * n_bytes, &map_q, n * 64, hk * args.p.group + first_head, token0, bar(kQ));
            int n = 0;
            for (; n < 2 * blocks; ++n) {
                const int st = n % args.stages;
                if (n >= args.stages && !wait(bar(kEmpty + st), (n / args.stages - 1) & 1, abort, args.limit)) break;
                mbar_arrive_expect_tx(bar(kFull + st), tile_bytes);
                load_tile(stage(n), (n & 1) ? &map_v : &map_k, halves, hk, k_first + (n >> 1) * kTile, bar(kFull + st));
            }
            // nothing is left in flight when the CTA goes on, whatever became of the others
            for (int k = max(0, n - args.stages); k < n; ++k)
                tc::drain(bar(kFull + k % args.stages), (k / args.stages) & 1, args.limit.timeout_ns);
            tc::drain(bar(kQ), 0, args.limit.timeout_ns);
        }
        __syncwarp();
    } else if (warp == 1 || warp == 2) {
        if (!skip && blocks > 0) {
            const bool waits = warp == 2;
            const int steps = (a.dim + 15) / 16;
            // the rows are N; V is the A operand, read MN-major (bit 15)
            const uint32_t is = instruction<T>(N, false), io = instruction<T>(N, false) | 1u << 15;
            const auto loaded = [&](int n) {
                wait_warp(bar(kFull + n % args.stages), (n / args.stages) & 1, abort, args.limit);
            };
            if (waits) wait_warp(bar(kQ), 0, abort, args.limit);
            for (int b = 0; b < blocks; ++b) {
                if (waits) loaded(2 * b);
                hand_over();
                if (!waits) {
                    mma_tokens(t_s, stage(2 * b), base + lay.q, steps, is, kHalfBytes, n_bytes);
                    commit(bar(kS));
                    commit(bar(kEmpty + 2 * b % args.stages));
                }
                if (waits) {
                    loaded(2 * b + 1);
                    wait_warp(bar(kP), b & 1, abort, args.limit);
                }
                hand_over();
                if (!waits) {
                    tc_fence_after_sync();
                    mma_values(t_o, stage(2 * b + 1), base + lay.weights, n_bytes, io, b > 0);
                    commit(bar(kEmpty + (2 * b + 1) % args.stages));
                }
            }
            if (!waits) {
                commit(bar(kO));
                commit(bar(kDrain));
                tc::drain(bar(kDrain), 0, args.limit.timeout_ns);
            }
        }
    } else if (warp >= 4 && !skip) {
        constexpr float kShift = weight_shift<T>();
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        // this thread's key within the block: its place in the weights' rows
        const uint32_t place = base + lay.weights + static_cast<uint32_t>(r >> 6) * n_bytes + static_cast<uint32_t>(r & 7) * 2u;
        const uint32_t chunk = static_cast<uint32_t>(r >> 3) & 7u;
        float m[N], l[N];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            m[n] = -INFINITY;
            l[n] = 0.f;
        }
        float by = args.scale_log2, inv_cap = 0.f;
        if (MODE & kCap) {
            by = a.cap * kLog2e;
            inv_cap = a.scale / a.cap;
        }
        for (int b = 0; b < blocks; ++b) {
            const int first = k_first + b * kTile, j = first + r;
            const bool masked = first < all_lo || first + kTile > all_hi;
            wait_warp(bar(kS), b & 1, abort, args.limit);
            tc_fence_after_sync();
            float s[N];
            tmem_ld_rows<N>(t_s + lanes, s);
            bool grew = b == 0;
#pragma unroll
            for (int n = 0; n < N; ++n) {
                if (n >= rows) break;             // (the same for all: rows that are not there cost nothing)
                if ((MODE & kCap) && n % 4 == 0) {
                    float x[4] = {s[n], s[n + 1], s[n + 2], s[n + 3]};
                    tanh_all(x, inv_cap);
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[n + e] = x[e];
                }
                s[n] *= by;
                if ((MODE & kBias) || masked) {
                    const int4 w = info[n];
                    if (MODE & kBias) s[n] = fmaf(-__int_as_float(w.w), fabsf(static_cast<float>(w.z - j)), s[n]);
                    if (masked) s[n] = j >= w.x && j < w.y ? s[n] : -INFINITY;
                }
                grew = grew || s[n] > m[n] + (kShift + kRescaleLog2);
            }
            // the maxima are the same in all threads, and only looked for when a
            // score is far above one of them
            if (bar_any(1, 128, grew)) {
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    if (n >= rows) break;
                    const int top = __reduce_max_sync(0xffffffffu, ordered(s[n] == s[n] ? s[n] : -INFINITY));
                    if (lane == 0) tops[(warp & 3) * N + n] = from_ordered(top);
                }
                named_sync(1, 128);
                float f[N];
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    f[n] = 1.0f;
                    if (n >= rows) continue;
                    const float top = fmaxf(fmaxf(tops[n], tops[N + n]), fmaxf(tops[2 * N + n], tops[3 * N + n]));
                    // (a row's maximum moves for its own scores only: not by what another row's keys hold)
                    const bool up = top > m[n] + (kShift + kRescaleLog2);
                    f[n] = up && m[n] != -INFINITY ? ex2_approx(m[n] - (top - kShift)) : 1.0f;
                    if (up) m[n] = top - kShift;
                    l[n] *= f[n];
                }
                if (b > 0) {
                    float o[N];
                    tmem_ld_rows<N>(t_o + lanes, o);
#pragma unroll
                    for (int q = 0; q < N / 16; ++q) {
                        uint32_t u[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) u[k] = __float_as_uint(o[16 * q + k] * f[16 * q + k]);
                        tmem_st16(t_o + lanes + 16 * q, u);
                    }
                    tmem_wait_st();
                }
            }
#pragma unroll
            for (int n = 0; n < N; ++n) {
                if (n >= rows) break;
                const float p = ex2_approx(s[n] - (m[n] == -INFINITY ? 0.f : m[n]));
                l[n] += p;
                sts_u16(place + n * 128u + ((chunk ^ (n & 7u)) << 4), Half2<T>::pack(p, 0.f));
            }
            if (masked) {
                const int nv = 2 * b + 1;
                wait_warp(bar(kFull + nv % args.stages), (nv / args.stages) & 1, abort, args.limit);
                clear_not_finite<T>(stage(nv), r, j, key0, key1, halves, bad);
            }
            fence_proxy_async_smem();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kP));
        }
        if (blocks > 0) wait_warp(bar(kO), 0, abort, args.limit);
        tc_fence_after_sync();
        // (the ring is free: every product is done; a failed call reads nothing of it)
        float *out = reinterpret_cast<float *>(gbase + lay.ring), *stats = reinterpret_cast<float *>(gbase + lay.stats);
        if (blocks > 0) {
            float o[N];
            tmem_ld_rows<N>(t_o + lanes, o);
#pragma unroll
            for (int n = 0; n < N; ++n)
                if (n < rows && r < a.dim) out[n * a.dim + r] = o[n];
        }
        named_sync(1, 128);           // the maxima in `tops` have been read
#pragma unroll
        for (int n = 0; n < N; ++n) {
            if (n >= rows) break;
            const float sum = warp_sum(l[n]);
            if (lane == 0) tops[(warp & 3) * N + n] = sum;
        }
        named_sync(1, 128);
#pragma unroll
        for (int n = 0; n < N; ++n)
            if (r == n) {
                stats[n] = m[n];
                stats[kTile + n] = (tops[n] + tops[N + n]) + (tops[2 * N + n] + tops[3 * N + n]);
            }
        tc_fence_before_sync();
    }
    __syncwarp();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 64);
    }
    __syncwarp();
    join_parts<T>(args, base + lay.stats, base + lay.ring, base + lay.words + 8, *abort != 0, split, token0, hk, first_head,
                  live, span, r);
}

using Kernel = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const SplitArgs);

template <typename T, int MODE>
cudaError_t launch(const SplitArgs &args, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, cudaStream_t s)
{
    const int halves = args.p.a.dim > 64 ? 2 : 1, rows = args.tokens * args.heads;
    static std::atomic<uint64_t> done[3], wide[3];
    const int which = rows <= 16 ? 0 : (rows <= 32 ? 1 : 2);
    const Kernel kernels[3] = {attn_few_kernel<T, MODE, 16>, attn_few_kernel<T, MODE, 32>, attn_split_kernel<T, MODE>};
    const Kernel kernel = kernels[which];
    // (never so little that three CTAs would share an SM: attn_split_kernel's
    // take 256 columns of its 512 of tensor memory each)
    const size_t smem = std::max<size_t>(which < 2 ? few_layout(halves, which ? 32 : 16, args.stages).total
                                                   : layout(halves, rows, args.stages).total, 80 * 1024);
    cudaError_t e = allow_shared(reinterpret_cast<const void *>(kernel), 160 * 1024, done[which]);
    if (e == cudaSuccess) e = allow_clusters(reinterpret_cast<const void *>(kernel), wide[which]);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = static_cast<unsigned>(args.splits);
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    const int64_t tiles = (args.p.a.tokens_q + args.tokens - 1) / args.tokens;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * args.splits * args.p.a.kv_heads * args.chunks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = args.splits > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, mq, mk, mv, args);
}

template <typename T>
cudaError_t launch_mode(int mode, const SplitArgs &args, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                        cudaStream_t s)
{
    if (mode == 0) return launch<T, 0>(args, mq, mk, mv, s);
    if (mode == kCap) return launch<T, kCap>(args, mq, mk, mv, s);
    if (mode == kBias) return launch<T, kBias>(args, mq, mk, mv, s);
    return launch<T, kCap | kBias>(args, mq, mk, mv, s);
}

// A call's tiles and splits, and about how long it takes (us).
//
// Splits: the number that should end first.  CTAs are taken to run in rounds of
// two per SM (also where an SM holds one), and one takes as long as its blocks and
// about seven more (start, first loads and join: 9 us where a block of its stream
// takes 1.3 us, or 2.2 us with more than 32 rows); documents are taken for half as long again as their average,
// since the longest ends last.  (24 caches of 2880 keys, 8 heads: 192 tiles, 3
// splits: two rounds.)
SplitArgs plan(const PackedAttn &p, int sm_count, double *us)
{
    const gn_attn_packed_args &a = p.a;
    SplitArgs args = {};
    args.p = p;
    args.scale_log2 = a.scale * kLog2e;
    args.heads = std::min(p.group, kTile);
    args.chunks = (p.group + args.heads - 1) / args.heads;
    const int64_t per_doc = (a.tokens_q + a.docs - 1) / a.docs;
    args.tokens = static_cast<int>(std::min<int64_t>(kTile / args.heads, per_doc));
    // (with up to 16 rows two CTAs' shared memory fits an SM, and so it does with 33
    // to 56, or with more of up to 64 channels; otherwise an SM holds one)
    args.stages = a.dim > 64 ? 3 : 5;
    const int64_t tiles = (a.tokens_q + args.tokens - 1) / args.tokens * a.kv_heads * args.chunks;
    const double blocks = 1.5 * static_cast<double>(a.tokens_k) / a.docs / kTile;
    double best = 0.0;
    for (int s = 1; s <= kMaxSplits && (s == 1 || s <= blocks); ++s) {
        const double cost = static_cast<double>((tiles * s + 2 * sm_count - 1) / (2 * sm_count)) * (7.0 + blocks / s);
        if (s == 1 || cost < best) {
            best = cost;
            args.splits = s;
        }
    }
    *us = best * (args.tokens * args.heads > 32 ? 2.2 : 1.3);
    return args;
}

}  // namespace

double packed_attn_split_us(const PackedAttn &p, int sm_count)
{
    double us;
    plan(p, sm_count, &us);
    return us;
}

cudaError_t launch_packed_attn_split(const PackedAttn &p, int sm_count, const WaitLimit &limit, cudaStream_t s)
{
    const gn_attn_packed_args &a = p.a;
    double us;
    SplitArgs args = plan(p, sm_count, &us);
    args.limit = limit;
    const bool bf16 = a.format == GN_FORMAT_BF16;
    CUtensorMap mq, mk, mv;
    if (!encode_heads(&mq, a.q, bf16, a.tokens_q, a.q_token, a.heads, a.q_head, a.dim, args.heads, args.tokens) ||
        !encode_heads(&mk, a.k, bf16, a.tokens_k, a.k_token, a.kv_heads, a.k_head, a.dim) ||
        !encode_heads(&mv, a.v, bf16, a.tokens_k, a.v_token, a.kv_heads, a.v_head, a.dim))
        return cudaErrorInvalidValue;
    const int mode = score_mode(a);
    return bf16 ? launch_mode<__nv_bfloat16>(mode, args, mq, mk, mv, s) : launch_mode<__half>(mode, args, mq, mk, mv, s);
}

}  // namespace gn
