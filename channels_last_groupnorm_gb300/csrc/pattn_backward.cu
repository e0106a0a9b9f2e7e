// pattn_backward.cu -- packed attention's backward pass on the tensor cores:
// three launches, every product a tcgen05 one and every sum in a fixed order.
//
//   attn_rows_info_kernel   per query: its run of keys; per query and head:
//                           lse in units of log2 and delta = dout . out
//   attn_dkv_kernel         a CTA owns 128 keys of one key / value head and
//                           goes over the queries that see them, in blocks of
//                           128, for every query head of the group (or, where
//                           those CTAs would be few, a cluster of CTAs shares
//                           the heads and adds up over distributed shared
//                           memory at the end):
//     S^T = K Q^T, dP^T = V dO^T           (keys are the lanes)
//     P^T = 2^(c S^T - lse),  dS^T = P^T (dP^T - delta) (1 - tanh^2)
//     dV += P^T dO,  dK += dS^T Q          (P^T, dS^T from tensor memory)
//   attn_dq_kernel          a CTA owns 128 queries of one head and goes over
//                           their keys:  S = Q K^T, dP = dO V^T, dS, dQ += dS K
//
// Roundings: P and dS are rounded to the half format, as the tensor cores take
// them (half a step of each weight, under the outputs' own rounding), and delta is
// formed from the forward pass' rounded output; scores, lse, the sums and the
// accumulators are fp32.  In fp16 a dS under 2^-14 loses bits and one under 2^-25
// is lost: 16384 tokens, D = 128, dout of 0.1 gives dq within 3.2e-4 of its norm,
// of 0.01 1.5e-3, of 0.001 1.5e-2 (dq itself, rounded, 2.1e-4, 2.2e-4, 1.3e-3).  A
// factor that lifts them without any overflow would have to be found for each
// key, and a training step in fp16 scales its loss anyway.
//
// Computing the scores in both costs 7 products of 128 x 128 x D per block
// instead of 5, but dK, dV and dQ stay in tensor memory to the end: no fp32
// atomics, so the same inputs give the same bits, and the shared heads' sums
// are part of the accumulation.
//
// In either kernel the tensor core always has the other half of the work in
// hand while the eight softmax warps (two per lane quarter, 64 columns each)
// do theirs: weights are made while dK and the next dP run, score gradients
// while dV and the next S run.  P and dS overwrite S and dP in place, every
// warp within the columns that it has read.
#include <algorithm>

#include "pattn_tiles.cuh"

namespace gn {
namespace {

using namespace pattn;

constexpr int kThreads = 384;    // warps: 0 loads, 1 MMA, 2 the MMA's waits, 4-11 softmax
// Tiles in flight: of the ones that two products far apart in a step read (Q for
// dK and dV, K for dQ), and of the ones that are done with sooner (dO, V).
// With two of each, released together, the loads were waited for (dQ: 2300 of
// 3900 cycles a step).
constexpr int kLongStages = 3;
constexpr int kShortStages = 2;

// Per query: the run of keys it sees and where it stands; per query and head:
// -lse in units of log2, and -delta.  Padded to whole blocks so that 128 rows can be copied
// from any multiple of 4; padding rows see nothing.
struct Info {
    float *lse, *delta;   // [heads][padded]
    int4 *span;           // [padded]
    int64_t padded;
};

__host__ __device__ inline int64_t padded_rows(int64_t tokens_q) { return (tokens_q + 2 * kTile - 1) / kTile * kTile; }

template <typename T>
__global__ void __launch_bounds__(256) attn_rows_info_kernel(const __grid_constant__ PackedAttn p, const Info info)
{
    tc::griddep_wait();
    if (threadIdx.x == 0) tc::griddep_launch_dependents();
    const gn_attn_packed_args &a = p.a;
    // sixteen lanes (eight channels each) per query and head
    const int lane = threadIdx.x & 31, place = lane & 15;
    const int64_t n = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 4;
    const int64_t i = n / a.heads;
    const int h = static_cast<int>(n % a.heads);
    if (n >= info.padded * a.heads) return;
    if (h == 0 && place == 0) {
        Span s = {0, 0, 0};
        if (i < a.tokens_q) s = query_span(a, static_cast<int>(i));
        info.span[i] = make_int4(s.lo, s.hi, s.pos, 0);
    }
    float s = 0.f;
    if (i < a.tokens_q && place * 8 < a.dim) {
        float x[8], g[8];
        unpack8<T>(__ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(a.out) + n * a.dim + place * 8)), x);
        unpack8<T>(__ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(p.dout) + i * p.dout_token + h * p.dout_head + place * 8)), g);
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(x[e], g[e], s);
    }
    const unsigned group = 0xffffu << (lane & 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(group, s, o);
    if (place == 0) {
        // a row without keys (lse -inf) weighs nothing anywhere
        float lse = i < a.tokens_q ? a.lse[static_cast<int64_t>(h) * a.tokens_q + i] * kLog2e : INFINITY;
        if (lse == -INFINITY) lse = INFINITY;
        info.lse[static_cast<int64_t>(h) * info.padded + i] = -lse;
        info.delta[static_cast<int64_t>(h) * info.padded + i] = -s;
    }
}

// ---- one row by one warp, for what sees a row that was cleared -----------------
template <typename T>
__device__ __noinline__ void row_dq(const PackedAttn &p, const Info &info, int i, int h)
{
    const gn_attn_packed_args &a = p.a;
    const int lane = threadIdx.x & 31, hk = h / p.group;
    const int4 s = info.span[i];
    const int64_t at = static_cast<int64_t>(h) * info.padded + i;
    const float nlse = info.lse[at], ndelta = info.delta[at];
    const float slope = a.slopes ? a.slopes[h] : 0.f;
    const float4 q = load4<T>(a.q, i * a.q_token + h * a.q_head, lane, a.dim);
    const float4 g = load4<T>(p.dout, i * p.dout_token + h * p.dout_head, lane, a.dim);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = s.x; j < s.y; ++j) {
        const float4 k = load4<T>(a.k, j * a.k_token + hk * a.k_head, lane, a.dim);
        const float4 v = load4<T>(a.v, j * a.v_token + hk * a.v_head, lane, a.dim);
        float slack;
        const float t = score_log2(a, slope, warp_sum(dot4(q, k)), s.z, j, slack);
        axpy4(acc, ex2_approx(t + nlse) * (warp_sum(dot4(g, v)) + ndelta) * slack * a.scale, k);
        if (all_nan(acc, lane, a.dim)) break;
    }
    store4<T>(p.dq, (static_cast<int64_t>(i) * a.heads + h) * a.dim, lane, a.dim, acc);
}

template <typename T>
__device__ __noinline__ void row_dkv(const PackedAttn &p, const Info &info, int j, int hk)
{
    const gn_attn_packed_args &a = p.a;
    const int lane = threadIdx.x & 31;
    const Span s = key_span(a, j);
    const float4 k = load4<T>(a.k, j * a.k_token + hk * a.k_head, lane, a.dim);
    const float4 v = load4<T>(a.v, j * a.v_token + hk * a.v_head, lane, a.dim);
    float4 dk = make_float4(0.f, 0.f, 0.f, 0.f), dv = dk;
    bool settled = false;
    for (int h = hk * p.group; !settled && h < (hk + 1) * p.group; ++h) {
        const float slope = a.slopes ? a.slopes[h] : 0.f;
        for (int i = s.lo; !settled && i < s.hi; ++i) {
            const float4 q = load4<T>(a.q, i * a.q_token + h * a.q_head, lane, a.dim);
            const float4 g = load4<T>(p.dout, i * p.dout_token + h * p.dout_head, lane, a.dim);
            const int64_t at = static_cast<int64_t>(h) * info.padded + i;
            float slack;
            const float t = score_log2(a, slope, warp_sum(dot4(q, k)), info.span[i].z, j, slack);
            const float w = ex2_approx(t + info.lse[at]);
            axpy4(dv, w, g);
            axpy4(dk, w * (warp_sum(dot4(g, v)) + info.delta[at]) * slack * a.scale, q);
            settled = all_nan(dk, lane, a.dim) && all_nan(dv, lane, a.dim);
        }
    }
    store4<T>(p.dk, (static_cast<int64_t>(j) * a.kv_heads + hk) * a.dim, lane, a.dim, dk);
    store4<T>(p.dv, (static_cast<int64_t>(j) * a.kv_heads + hk) * a.dim, lane, a.dim, dv);
}

// Scores of N pairs (raw, in place) to what times the returned factor is in
// units of log2 before lse, capped, and biased by the distance |at + DIR n| (or,
// for queries of several documents, by what far(n) says).  slack[n], with a cap:
// its slope there.
template <int MODE, int DIR, int N, typename Far>
__device__ __forceinline__ float bend(float (&s)[N], float (&slack)[N], const TileArgs &args, float slope2, int at,
                                      bool several, Far far)
{
    const gn_attn_packed_args &a = args.p.a;
    float by = args.scale_log2;
    if (MODE & kCap) {
        tanh_all(s, a.scale / a.cap);
        by = a.cap * kLog2e;
#pragma unroll
        for (int n = 0; n < N; n += 2) {
            const uint64_t v = pack2(s[n], s[n + 1]);
            const float2 r = unpack2(fma2(mul2(v, pack2(-1.0f, -1.0f)), v, pack2(1.0f, 1.0f)));
            slack[n] = r.x;
            slack[n + 1] = r.y;
        }
    }
    if (!(MODE & kBias)) return by;
    if (several) {
#pragma unroll
        for (int n = 0; n < N; ++n) s[n] = fmaf(-slope2, fabsf(far(n)), s[n] * by);
    } else {
        take_distance<DIR>(s, by, slope2, at);
    }
    return 1.0f;
}

// The weights times the cap's slopes, which is all that the scores' gradients
// want of either (and keeps 64 registers free for dP).
template <int MODE, int N>
__device__ __forceinline__ void fold_slack(float (&w)[N], const float (&slack)[N])
{
    if (MODE & kCap) {
#pragma unroll
        for (int n = 0; n < N; n += 2) {
            const float2 v = unpack2(mul2(pack2(w[n], w[n + 1]), pack2(slack[n], slack[n + 1])));
            w[n] = v.x;
            w[n + 1] = v.y;
        }
    }
}

// Barriers and words of either kernel.  Own: the tiles a CTA owns; Long /
// Short: a streamed tile is there, is done with; Info: a block's row records;
// S / Dp: an MMA result is there; P / Ds: the softmax warps have put theirs in
// its place; Out: the accumulators are done.  A phase of a barrier must have been
// seen by all that wait for it before the next one can complete.  dK and dV issue
// S of a block only after P of the block before, one S is enough; dQ issues it a
// block earlier, into the other buffer of scores, and has an S for each: S of block
// n + 2 follows Ds of block n, whose warps have seen S of block n.
enum Bar { kOwn = 0, kLong, kLongFree = kLong + kLongStages, kShort = kLongFree + kLongStages,
           kShortFree = kShort + kShortStages, kInfo = kShortFree + kShortStages, kS = kInfo + 2, kDp = kS + 2, kP, kDs, kOut,
           kDrain, kBars };
constexpr int kSoftWarps = 8;

__device__ __forceinline__ void init_bars(uint32_t bars)
{
    for (int i = 0; i < kBars; ++i) mbar_init(bars + 8u * i, i == kP || i == kDs ? kSoftWarps : 1);
    mbar_init_fence();
}

// Shared memory of either kernel: the two tiles it owns, the two rings, for dK
// and dV the row records of two blocks.  (It begins on a 1 KB boundary, as the
// swizzled tiles need: there is no static shared memory ahead of it.)
struct Layout {
    uint32_t own, longs, shorts, rows, bars, words, total;
};

__host__ __device__ inline Layout layout(int halves)
{
    Layout l;
    const uint32_t tile = kHalfBytes * static_cast<uint32_t>(halves);
    l.own = 0;
    l.longs = 2 * tile;
    l.shorts = l.longs + kLongStages * tile;
    l.rows = l.shorts + kShortStages * tile;    // 2 x (128 -lse, 128 -delta)
    l.bars = l.rows + 2 * kTile * 8;
    l.words = l.bars + 8 * kBars;               // tensor-memory slot, abort, bad[2], 8 x 4 range words
    l.total = l.words + 4 * (4 + 32);
    return l;
}

// How many of each load a CTA has issued; when it ends nothing is left in
// flight, whatever became of the others.
struct Loads {
    int longs, shorts, infos;
};

__device__ __forceinline__ void drain_loads(uint32_t bars, const Loads &got, uint64_t timeout_ns)
{
    const auto ring = [&](int first, int stages, int n) {
        for (int k = max(0, n - stages); k < n; ++k)
            tc::drain(bars + 8u * (first + k % stages), (k / stages) & 1, timeout_ns);
    };
    tc::drain(bars + 8u * kOwn, 0, timeout_ns);
    ring(kLong, kLongStages, got.longs);
    ring(kShort, kShortStages, got.shorts);
    ring(kInfo, 2, got.infos);
}

// Writes one accumulator's rows: 64 channels (half 0 or 1) of the warp's 32
// tokens, scaled and rounded once.
template <typename T>
__device__ __forceinline__ void store_half(void *out, int64_t row_offset, bool live, bool any, uint32_t taddr, int half,
                                           int dim, float scale)
{
#pragma unroll 1
    for (int q = 2 * half; q < 2 * half + 2; ++q) {
        if (32 * q >= dim) break;
        float o[32];
        if (any) {
            tmem_ld32(taddr + 32 * q, o);
            tmem_wait_ld();
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                w[e] = any ? Half2<T>::pack(o[8 * k + 2 * e] * scale, o[8 * k + 2 * e + 1] * scale) : 0u;
            if (live && 32 * q + 8 * k < dim)
                *reinterpret_cast<uint4 *>(static_cast<T *>(out) + row_offset + 32 * q + 8 * k) =
                    make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// ---------------------------------------------------------------------------
// dK and dV
// ---------------------------------------------------------------------------
template <typename T, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    attn_dkv_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                    const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_do,
                    const __grid_constant__ TileArgs args, const Info info)
{
    extern __shared__ __align__(1024) uint8_t gbase[];
    const uint32_t base = smem_addr(gbase);
    const gn_attn_packed_args &a = args.p.a;
    const int halves = a.dim > 64 ? 2 : 1, group = args.p.group;
    const Layout lay = layout(halves);
    const uint32_t tile_bytes = kHalfBytes * static_cast<uint32_t>(halves);
    const auto bar = [&](int i) { return base + lay.bars + 8u * static_cast<uint32_t>(i); };
    volatile uint32_t *words = reinterpret_cast<volatile uint32_t *>(gbase + lay.words);
    volatile int *abort = reinterpret_cast<volatile int *>(words + 1);
    int *bad = reinterpret_cast<int *>(gbase + lay.words + 8);
    volatile int *range = reinterpret_cast<volatile int *>(words + 4);
    const auto long_tile = [&](int n) { return base + lay.longs + static_cast<uint32_t>(n % kLongStages) * tile_bytes; };
    const auto short_tile = [&](int n) { return base + lay.shorts + static_cast<uint32_t>(n % kShortStages) * tile_bytes; };
    // streamed tile n is there (a whole warp asks) / is done with (n < 0: there was none)
    const auto has_long = [&](int n) { return wait_warp(bar(kLong + n % kLongStages), (n / kLongStages) & 1, abort, args.limit); };
    const auto has_short = [&](int n) { return wait_warp(bar(kShort + n % kShortStages), (n / kShortStages) & 1, abort, args.limit); };
    const auto long_free = [&](int n) {
        return n < 0 || wait(bar(kLongFree + n % kLongStages), (n / kLongStages) & 1, abort, args.limit);
    };
    const auto short_free = [&](int n) {
        return n < 0 || wait(bar(kShortFree + n % kShortStages), (n / kShortStages) & 1, abort, args.limit);
    };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // a cluster's CTAs take `heads` of the group's query heads each
    const int parts = args.parts, part = static_cast<int>(blockIdx.x) % parts, heads = group / parts;
    const int hk = static_cast<int>(blockIdx.x) / parts % a.kv_heads, first_head = hk * group + part * heads;
    // the first tiles first: with causal runs the most queries see them
    const int key0 = static_cast<int>(blockIdx.x) / parts / a.kv_heads * kTile;

    if (threadIdx.x == 0) {
        init_bars(bar(0));
        *abort = (*reinterpret_cast<volatile unsigned int *>(args.limit.status) != 0u) ? 1 : 0;
        bad[0] = 0x7fffffff;
        bad[1] = -1;
        prefetch_tensormap(&map_q);
        prefetch_tensormap(&map_k);
        prefetch_tensormap(&map_v);
        prefetch_tensormap(&map_do);
    }
    if (warp == 1) {
        tmem_alloc(base + lay.words, 512);
        tmem_relinquish();
    }
    tc::griddep_wait();
    if (threadIdx.x == 0) tc::griddep_launch_dependents();

    // the queries that see any of the tile's keys, and those that see all
    const int row = (warp & 3) * 32 + lane, key = key0 + row;
    Span span = {0, 0, 0};
    if (warp >= 4) {
        if (key < a.tokens_k) span = key_span(a, key);
        const bool live = key < a.tokens_k, some = live && span.lo < span.hi;
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
    int q_lo = 0x7fffffff, q_hi = 0, all_lo = 0, all_hi = 0x7fffffff;
    for (int w = 0; w < 4; ++w) {
        q_lo = min(q_lo, range[4 * w]);
        q_hi = max(q_hi, range[4 * w + 1]);
        all_lo = max(all_lo, range[4 * w + 2]);
        all_hi = min(all_hi, range[4 * w + 3]);
    }
    const bool any = q_lo < q_hi;
    const int q0 = q_lo & ~3;                   // the rows' records are copied from a multiple of 32 bytes
    const int blocks = any ? (q_hi - q0 + kTile - 1) / kTile : 0;
    const int steps_all = blocks * heads;       // query heads outermost
    const bool skip = *abort != 0;
    const uint32_t k_tile = base + lay.own, v_tile = k_tile + tile_bytes;
    const uint32_t t_s = tmem, t_dp = tmem + 128, t_dk = tmem + 256, t_dv = tmem + 384;

    if (warp >= 4) {
        many_registers();
        // ---- softmax: one key per thread, 64 of a block's queries per warp ----
        const int half = (warp - 4) >> 2;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        bool go = !skip;
        float slope2 = 0.f;
        for (int n = 0; go && n < steps_all; ++n) {
            const int i0 = q0 + (n % blocks) * kTile;
            const bool masked = i0 < all_lo || i0 + kTile > all_hi;
            if ((MODE & kBias) && n % blocks == 0) slope2 = __ldg(a.slopes + first_head + n / blocks) * kLog2e;
            const float4 *nlse = reinterpret_cast<const float4 *>(gbase + lay.rows + (n & 1) * kTile * 8) + 16 * half;
            const float4 *ndelta = nlse + kTile / 4;
            const int4 *spans = info.span + i0 + 64 * half;
            go = wait_warp(bar(kInfo + (n & 1)), (n >> 1) & 1, abort, args.limit) &&
                 wait_warp(bar(kS), n & 1, abort, args.limit);
            if (!go) break;
            tc_fence_after_sync();
            float w[64], slack[64];              // scores, then weights; the cap's slopes
            tmem_ld_all(t_s + lanes + 64 * half, w);
            // (queries that all see the same keys stand one after the other)
            const int at = (MODE & kBias) ? __ldg(&spans->z) - key : 0;
            const float c = bend<MODE, 1>(w, slack, args, slope2, at, masked,
                                             [&](int k) { return static_cast<float>(__ldg(&spans[k].z) - key); });
            const uint64_t c2 = pack2(c, c);
#pragma unroll
            for (int k = 0; k < 64; k += 4) {
                const float4 e = nlse[k / 4];
                const float2 x = unpack2(fma2(pack2(w[k], w[k + 1]), c2, pack2(e.x, e.y)));
                const float2 y = unpack2(fma2(pack2(w[k + 2], w[k + 3]), c2, pack2(e.z, e.w)));
                w[k] = ex2_approx(x.x);
                w[k + 1] = ex2_approx(x.y);
                w[k + 2] = ex2_approx(y.x);
                w[k + 3] = ex2_approx(y.y);
            }
            if (masked) {
#pragma unroll
                for (int k = 0; k < 64; ++k) {
                    const int2 sp = __ldg(reinterpret_cast<const int2 *>(spans + k));
                    const bool sees = key >= sp.x && key < sp.y;
                    w[k] = sees ? w[k] : 0.f;
                    if (MODE & kCap) slack[k] = sees ? slack[k] : 0.f;    // (of an unseen NaN: 0 x NaN is not 0)
                }
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t pk[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) pk[k] = Half2<T>::pack(w[32 * q + 2 * k], w[32 * q + 2 * k + 1]);
                tmem_st16(t_s + lanes + 64 * half + 16 * q, pk);
            }
            fold_slack<MODE>(w, slack);
            if (masked) {
                const int r = (warp & 3) * 32 + lane;
                if (half == 0 || has_short(n))
                    clear_not_finite<T>(half ? short_tile(n) : long_tile(n), r, i0 + r, q_lo, q_hi, halves, bad);
            }
            tmem_wait_st();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kP));

            go = wait_warp(bar(kDp), n & 1, abort, args.limit);
            if (!go) break;
            tc_fence_after_sync();
            float dp[64];
            tmem_ld_all(t_dp + lanes + 64 * half, dp);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t pk[16];
#pragma unroll
                for (int k = 0; k < 16; k += 2) {
                    const int n0 = 32 * q + 2 * k;
                    const float4 e = ndelta[n0 / 4];
                    const float2 x = unpack2(mul2(pack2(w[n0], w[n0 + 1]), add2(pack2(dp[n0], dp[n0 + 1]), pack2(e.x, e.y))));
                    const float2 y = unpack2(mul2(pack2(w[n0 + 2], w[n0 + 3]), add2(pack2(dp[n0 + 2], dp[n0 + 3]), pack2(e.z, e.w))));
                    float d[4] = {x.x, x.y, y.x, y.y};
                    if (masked) {
                        // a weight of zero times what an unseen row holds
#pragma unroll
                        for (int i = 0; i < 4; ++i) d[i] = w[n0 + i] == 0.f ? 0.f : d[i];
                    }
                    pk[k] = Half2<T>::pack(d[0], d[1]);
                    pk[k + 1] = Half2<T>::pack(d[2], d[3]);
                }
                tmem_st16(t_dp + lanes + 64 * half + 16 * q, pk);
            }
            tmem_wait_st();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kDs));
        }
        if (any && go) go = wait_warp(bar(kOut), 0, abort, args.limit);
        const bool failed = bar_any(1, 256, !go), live = key < a.tokens_k;   // one answer for all: barriers follow
        const int64_t at = (static_cast<int64_t>(key) * a.kv_heads + hk) * a.dim;
        int bad_lo = 0x7fffffff, bad_hi = -1;
        tc_fence_after_sync();
        if (parts == 1) {
            if (!failed) {
                store_half<T>(args.p.dk, at, live, any, t_dk + lanes, half, a.dim, a.scale);
                store_half<T>(args.p.dv, at, live, any, t_dv + lanes, half, a.dim, 1.0f);
            }
            named_sync(1, 256);
            bad_lo = bad[0];
            bad_hi = bad[1];
        } else {
            // this CTA's sums into its shared memory (all of which is free now:
            // every product is done), [dk, dv][channels][keys]; then every CTA
            // adds up all parts of some of the channels, in the parts' order
            float *sums = reinterpret_cast<float *>(gbase);
            if (any && !failed)
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    const int c = 64 * half + 32 * (q & 1);
                    if (c >= a.dim) continue;
                    float o[32];
                    tmem_ld32((q < 2 ? t_dk : t_dv) + lanes + c, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (c + k < a.dim) sums[((q < 2 ? 0 : a.dim) + c + k) * kTile + row] = o[k];
                }
            cluster_sync_all();
            const int eighths = 2 * a.dim / 8;
            if (!failed)
                for (int n = 2 * part + half; n < eighths; n += 2 * parts) {
                    float v[8] = {};
                    if (any)
                        for (int p = 0; p < parts; ++p)
#pragma unroll
                            for (int e = 0; e < 8; ++e) v[e] += peer_float(base + ((n * 8 + e) * kTile + row) * 4u, p);
                    const int c = n * 8 % a.dim;
                    const float by = n * 8 < a.dim ? a.scale : 1.0f;
                    if (live)
                        *reinterpret_cast<uint4 *>(static_cast<T *>(n * 8 < a.dim ? args.p.dk : args.p.dv) + at + c) =
                            make_uint4(Half2<T>::pack(v[0] * by, v[1] * by), Half2<T>::pack(v[2] * by, v[3] * by),
                                       Half2<T>::pack(v[4] * by, v[5] * by), Half2<T>::pack(v[6] * by, v[7] * by));
                }
            if (lane < parts) {
                bad_lo = __float_as_int(peer_float(base + lay.words + 8, lane));
                bad_hi = __float_as_int(peer_float(base + lay.words + 12, lane));
            }
            bad_lo = __reduce_min_sync(0xffffffffu, bad_lo);
            bad_hi = __reduce_max_sync(0xffffffffu, bad_hi);
            cluster_sync_all();
        }
        unsigned again = failed || part ? 0u : __ballot_sync(0xffffffffu, live && span.lo < span.hi && span.lo <= bad_hi &&
                                                                              span.hi > bad_lo);
        for (int n = 0; again; again &= again - 1, ++n) {
            if ((n & 1) != half) continue;
            const int from = __ffs(again) - 1;
            const int i0 = max(__shfl_sync(0xffffffffu, span.lo, from), bad_lo);
            const int i1 = min(__shfl_sync(0xffffffffu, span.hi, from), bad_hi + 1);
            bool bad_seen = false;
            for (int h = hk * group; !bad_seen && h < (hk + 1) * group; ++h)
                bad_seen = any_not_finite<T>(a.q, a.q_token, h * a.q_head, i0, i1, a.dim) ||
                           any_not_finite<T>(args.p.dout, args.p.dout_token, h * args.p.dout_head, i0, i1, a.dim);
            if (bad_seen) row_dkv<T>(args.p, info, key - lane + from, hk);
        }
        tc_fence_before_sync();
    } else {
        few_registers();
        if (warp == 0) {
            if (lane == 0 && !skip && any) {
                mbar_arrive_expect_tx(bar(kOwn), 2 * tile_bytes);
                load_tile(k_tile, &map_k, halves, hk, key0, bar(kOwn));
                load_tile(v_tile, &map_v, halves, hk, key0, bar(kOwn));
                Loads got = {};
                for (int n = 0; n < steps_all; ++n) {
                    const int h = first_head + n / blocks, i0 = q0 + (n % blocks) * kTile;
                    if (!long_free(n - kLongStages)) break;
                    mbar_arrive_expect_tx(bar(kLong + n % kLongStages), tile_bytes);
                    load_tile(long_tile(n), &map_q, halves, h, i0, bar(kLong + n % kLongStages));
                    ++got.longs;
                    if (!short_free(n - kShortStages)) break;
                    mbar_arrive_expect_tx(bar(kShort + n % kShortStages), tile_bytes);
                    load_tile(short_tile(n), &map_do, halves, h, i0, bar(kShort + n % kShortStages));
                    ++got.shorts;
                    // the records are done with when the scores' gradients of their block are, as Q is
                    if (!long_free(n - 2)) break;
                    const int64_t at = static_cast<int64_t>(h) * info.padded + i0;
                    const uint32_t rows = base + lay.rows + (n & 1) * kTile * 8;
                    mbar_arrive_expect_tx(bar(kInfo + (n & 1)), kTile * 8);
                    bulk_load(rows, info.lse + at, kTile * 4, bar(kInfo + (n & 1)));
                    bulk_load(rows + kTile * 4, info.delta + at, kTile * 4, bar(kInfo + (n & 1)));
                    ++got.infos;
                }
                drain_loads(bar(0), got, args.limit.timeout_ns);
            }
        } else if (warp == 1 || warp == 2) {
            if (!skip && any) {
                const bool waits = warp == 2;
                const int steps = (a.dim + 15) / 16;
                const uint32_t is = instruction<T>(kTile, false), io = instruction<T>(steps * 16, true);
                if (waits) {
                    wait_warp(bar(kOwn), 0, abort, args.limit);
                    has_long(0);
                    has_short(0);
                }
                hand_over();
                if (!waits) {
                    mma_tokens(t_s, k_tile, long_tile(0), steps, is);
                    commit(bar(kS));
                    mma_tokens(t_dp, v_tile, short_tile(0), steps, is);
                    commit(bar(kDp));
                }
                for (int n = 0; n < steps_all; ++n) {
                    const bool more = n + 1 < steps_all;
                    if (waits) wait_warp(bar(kP), n & 1, abort, args.limit);
                    hand_over();
                    if (!waits) {
                        tc_fence_after_sync();
                        mma_channels(t_dv, t_s, short_tile(n), 0, io, n > 0);
                        mma_channels(t_dv, t_s + 64, short_tile(n), 1, io, true);
                        commit(bar(kShortFree + n % kShortStages));
                    }
                    if (more) {
                        if (waits) has_long(n + 1);
                        hand_over();
                        if (!waits) {
                            mma_tokens(t_s, k_tile, long_tile(n + 1), steps, is);
                            commit(bar(kS));
                        }
                    }
                    if (waits) wait_warp(bar(kDs), n & 1, abort, args.limit);
                    hand_over();
                    if (!waits) {
                        tc_fence_after_sync();
                        mma_channels(t_dk, t_dp, long_tile(n), 0, io, n > 0);
                        mma_channels(t_dk, t_dp + 64, long_tile(n), 1, io, true);
                        commit(bar(kLongFree + n % kLongStages));
                    }
                    if (more) {
                        if (waits) has_short(n + 1);
                        hand_over();
                        if (!waits) {
                            mma_tokens(t_dp, v_tile, short_tile(n + 1), steps, is);
                            commit(bar(kDp));
                        }
                    }
                }
                if (!waits) {
                    commit(bar(kOut));
                    commit(bar(kDrain));
                    tc::drain(bar(kDrain), 0, args.limit.timeout_ns);
                }
            }
        }
        __syncwarp();
        if (parts > 1) {        // (the softmax warps' two)
            cluster_sync_all();
            cluster_sync_all();
        }
    }
    __syncwarp();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------------------
// dQ
// ---------------------------------------------------------------------------
template <typename T, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    attn_dq_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_do,
                   const __grid_constant__ TileArgs args, const Info info)
{
    extern __shared__ __align__(1024) uint8_t gbase[];
    const uint32_t base = smem_addr(gbase);
    const gn_attn_packed_args &a = args.p.a;
    const int halves = a.dim > 64 ? 2 : 1;
    const Layout lay = layout(halves);
    const uint32_t tile_bytes = kHalfBytes * static_cast<uint32_t>(halves);
    const auto bar = [&](int i) { return base + lay.bars + 8u * static_cast<uint32_t>(i); };
    volatile uint32_t *words = reinterpret_cast<volatile uint32_t *>(gbase + lay.words);
    volatile int *abort = reinterpret_cast<volatile int *>(words + 1);
    int *bad = reinterpret_cast<int *>(gbase + lay.words + 8);
    volatile int *range = reinterpret_cast<volatile int *>(words + 4);
    const auto long_tile = [&](int n) { return base + lay.longs + static_cast<uint32_t>(n % kLongStages) * tile_bytes; };
    const auto short_tile = [&](int n) { return base + lay.shorts + static_cast<uint32_t>(n % kShortStages) * tile_bytes; };
    // streamed tile n is there (a whole warp asks) / is done with (n < 0: there was none)
    const auto has_long = [&](int n) { return wait_warp(bar(kLong + n % kLongStages), (n / kLongStages) & 1, abort, args.limit); };
    const auto has_short = [&](int n) { return wait_warp(bar(kShort + n % kShortStages), (n / kShortStages) & 1, abort, args.limit); };
    const auto long_free = [&](int n) {
        return n < 0 || wait(bar(kLongFree + n % kLongStages), (n / kLongStages) & 1, abort, args.limit);
    };
    const auto short_free = [&](int n) {
        return n < 0 || wait(bar(kShortFree + n % kShortStages), (n / kShortStages) & 1, abort, args.limit);
    };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.x % a.heads, hk = h / args.p.group;
    const int row0 = (args.tiles - 1 - static_cast<int>(blockIdx.x / a.heads)) * kTile;

    if (threadIdx.x == 0) {
        init_bars(bar(0));
        *abort = (*reinterpret_cast<volatile unsigned int *>(args.limit.status) != 0u) ? 1 : 0;
        bad[0] = 0x7fffffff;
        bad[1] = -1;
        prefetch_tensormap(&map_q);
        prefetch_tensormap(&map_k);
        prefetch_tensormap(&map_v);
        prefetch_tensormap(&map_do);
    }
    if (warp == 1) {
        tmem_alloc(base + lay.words, 512);
        tmem_relinquish();
    }
    tc::griddep_wait();
    if (threadIdx.x == 0) tc::griddep_launch_dependents();

    const int r = (warp & 3) * 32 + lane, row = row0 + r;   // (row < info.padded)
    int4 span = make_int4(0, 0, 0, 0);
    float nlse = -INFINITY, ndelta = 0.f;
    if (warp >= 4) {
        span = info.span[row];
        nlse = info.lse[static_cast<int64_t>(h) * info.padded + row];
        ndelta = info.delta[static_cast<int64_t>(h) * info.padded + row];
        const bool live = row < a.tokens_q, some = live && span.x < span.y;
        const int lo = __reduce_min_sync(0xffffffffu, some ? span.x : 0x7fffffff);
        const int hi = __reduce_max_sync(0xffffffffu, some ? span.y : 0);
        const int all_lo = __reduce_max_sync(0xffffffffu, !live ? 0 : (some ? span.x : 0x7fffffff));
        const int all_hi = __reduce_min_sync(0xffffffffu, !live ? 0x7fffffff : (some ? span.y : 0));
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
    int key0 = 0x7fffffff, key1 = 0, all_lo = 0, all_hi = 0x7fffffff;
    for (int w = 0; w < 4; ++w) {
        key0 = min(key0, range[4 * w]);
        key1 = max(key1, range[4 * w + 1]);
        all_lo = max(all_lo, range[4 * w + 2]);
        all_hi = min(all_hi, range[4 * w + 3]);
    }
    const bool any = key0 < key1;
    const int blocks = any ? (key1 - key0 + kTile - 1) / kTile : 0;
    const bool skip = *abort != 0;
    const uint32_t q_tile = base + lay.own, do_tile = q_tile + tile_bytes;
    // two buffers of scores (their gradients go over them)
    const uint32_t t_s = tmem, t_dp = tmem + 256, t_dq = tmem + 384;

    if (warp >= 4) {
        many_registers();
        // ---- softmax: one query per thread, 64 of a block's keys per warp ----
        const int half = (warp - 4) >> 2;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const float slope2 = (MODE & kBias) ? __ldg(a.slopes + h) * kLog2e : 0.f;
        bool go = !skip;
        for (int n = 0; go && n < blocks; ++n) {
            const int j0 = key0 + n * kTile;
            const bool masked = j0 < all_lo || j0 + kTile > all_hi;
            const int lo = span.x - j0, len = max(0, span.y - span.x);
            const uint32_t ts = t_s + lanes + 128 * (n & 1) + 64 * half;
            go = wait_warp(bar(kS + (n & 1)), (n >> 1) & 1, abort, args.limit);
            if (!go) break;
            tc_fence_after_sync();
            float w[64], slack[64];              // scores, then weights; the cap's slopes
            tmem_ld_all(ts, w);
            const float c = bend<MODE, -1>(w, slack, args, slope2, span.z - j0 - 64 * half, false, [](int) { return 0.f; });
            const uint64_t c2 = pack2(c, c), e2 = pack2(nlse, nlse);
#pragma unroll
            for (int k = 0; k < 64; k += 2) {
                const float2 x = unpack2(fma2(pack2(w[k], w[k + 1]), c2, e2));
                w[k] = ex2_approx(x.x);
                w[k + 1] = ex2_approx(x.y);
            }
            fold_slack<MODE>(w, slack);
            if (masked) {
#pragma unroll
                for (int k = 0; k < 64; ++k)
                    w[k] = static_cast<unsigned>(k + 64 * half - lo) < static_cast<unsigned>(len) ? w[k] : 0.f;
            }
            go = wait_warp(bar(kDp), n & 1, abort, args.limit);
            if (!go) break;
            tc_fence_after_sync();
            float dp[64];
            tmem_ld_all(t_dp + lanes + 64 * half, dp);
            const uint64_t d2 = pack2(ndelta, ndelta);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t pk[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const int n0 = 32 * q + 2 * k;
                    float2 x = unpack2(mul2(pack2(w[n0], w[n0 + 1]), add2(pack2(dp[n0], dp[n0 + 1]), d2)));
                    if (masked) {
                        x.x = w[n0] == 0.f ? 0.f : x.x;
                        x.y = w[n0 + 1] == 0.f ? 0.f : x.y;
                    }
                    pk[k] = Half2<T>::pack(x.x, x.y);
                }
                tmem_st16(ts + 16 * q, pk);
            }
            if (masked && half == 0)
                clear_not_finite<T>(long_tile(n), r, j0 + r, key0, key1, halves, bad);
            tmem_wait_st();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kDs));
        }
        if (any && go) go = wait_warp(bar(kOut), 0, abort, args.limit);
        if (!bar_any(1, 256, !go)) {   // one answer for all: there is another barrier inside
            tc_fence_after_sync();
            const bool live = row < a.tokens_q;
            store_half<T>(args.p.dq, (static_cast<int64_t>(row) * a.heads + h) * a.dim, live, any, t_dq + lanes, half, a.dim,
                          a.scale);
            named_sync(1, 256);
            unsigned again = __ballot_sync(0xffffffffu, live && span.x < span.y && span.x <= bad[1] && span.y > bad[0]);
            for (int n = 0; again; again &= again - 1, ++n) {
                if ((n & 1) != half) continue;
                const int from = __ffs(again) - 1;
                const int j0 = max(__shfl_sync(0xffffffffu, span.x, from), bad[0]);
                const int j1 = min(__shfl_sync(0xffffffffu, span.y, from), bad[1] + 1);
                if (any_not_finite<T>(a.k, a.k_token, hk * a.k_head, j0, j1, a.dim)) row_dq<T>(args.p, info, row - lane + from, h);
            }
        }
        tc_fence_before_sync();
    } else {
        few_registers();
        if (warp == 0) {
            if (lane == 0 && !skip && any) {
                mbar_arrive_expect_tx(bar(kOwn), 2 * tile_bytes);
                load_tile(q_tile, &map_q, halves, h, row0, bar(kOwn));
                load_tile(do_tile, &map_do, halves, h, row0, bar(kOwn));
                Loads got = {};
                for (int n = 0; n < blocks; ++n) {
                    if (!long_free(n - kLongStages)) break;
                    mbar_arrive_expect_tx(bar(kLong + n % kLongStages), tile_bytes);
                    load_tile(long_tile(n), &map_k, halves, hk, key0 + n * kTile, bar(kLong + n % kLongStages));
                    ++got.longs;
                    if (!short_free(n - kShortStages)) break;
                    mbar_arrive_expect_tx(bar(kShort + n % kShortStages), tile_bytes);
                    load_tile(short_tile(n), &map_v, halves, hk, key0 + n * kTile, bar(kShort + n % kShortStages));
                    ++got.shorts;
                }
                drain_loads(bar(0), got, args.limit.timeout_ns);
            }
        } else if (warp == 1 || warp == 2) {
            if (!skip && any) {
                const bool waits = warp == 2;
                const int steps = (a.dim + 15) / 16;
                const uint32_t is = instruction<T>(kTile, false), io = instruction<T>(steps * 16, true);
                if (waits) {
                    wait_warp(bar(kOwn), 0, abort, args.limit);
                    has_long(0);
                    has_short(0);
                }
                hand_over();
                if (!waits) {
                    mma_tokens(t_s, q_tile, long_tile(0), steps, is);
                    commit(bar(kS));
                    mma_tokens(t_dp, do_tile, short_tile(0), steps, is);
                    commit(bar(kDp));
                    commit(bar(kShortFree));
                }
                for (int n = 0; n < blocks; ++n) {
                    const bool more = n + 1 < blocks;
                    if (more) {
                        if (waits) has_long(n + 1);
                        hand_over();
                        if (!waits) {
                            mma_tokens(t_s + 128 * ((n + 1) & 1), q_tile, long_tile(n + 1), steps, is);
                            commit(bar(kS + ((n + 1) & 1)));
                        }
                    }
                    if (waits) {
                        if (more) has_short(n + 1);
                        wait_warp(bar(kDs), n & 1, abort, args.limit);
                    }
                    hand_over();
                    if (!waits) {
                        tc_fence_after_sync();
                        if (more) {
                            mma_tokens(t_dp, do_tile, short_tile(n + 1), steps, is);
                            commit(bar(kDp));
                            commit(bar(kShortFree + (n + 1) % kShortStages));
                        }
                        mma_channels(t_dq, t_s + 128 * (n & 1), long_tile(n), 0, io, n > 0);
                        mma_channels(t_dq, t_s + 128 * (n & 1) + 64, long_tile(n), 1, io, true);
                        commit(bar(kLongFree + n % kLongStages));
                    }
                }
                if (!waits) {
                    commit(bar(kOut));
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
cudaError_t launch(const TileArgs &args, const CUtensorMap (&map)[4], const Info &info, int sm_count, cudaStream_t s,
                   int *launches)
{
    const gn_attn_packed_args &a = args.p.a;
    const int halves = a.dim > 64 ? 2 : 1;
    static std::atomic<uint64_t> done_kv{0}, done_q{0};
    cudaError_t e = allow_shared(reinterpret_cast<const void *>(attn_dkv_kernel<T, MODE>), layout(2).total, done_kv);
    if (e == cudaSuccess)
        e = allow_shared(reinterpret_cast<const void *>(attn_dq_kernel<T, MODE>), layout(2).total, done_q);
    if (e != cudaSuccess) return e;
    const int64_t rows = info.padded * a.heads;
    e = tc::launch_pdl(attn_rows_info_kernel<T>, dim3(static_cast<unsigned>((rows + 15) / 16)), dim3(256), 0, s, args.p, info);
    if (e != cudaSuccess) return e;
    ++*launches;
    TileArgs kv = args, q = args;
    kv.tiles = static_cast<int>((a.tokens_k + kTile - 1) / kTile);
    // Shared heads: one CTA for all query heads of a key / value head and tile,
    // or (a divisor up to 8 of them) a cluster, when those CTAs are fewer than
    // four for each SM and the longest would be waited for: 4360 tokens, 16 heads
    // on 4, D = 64 (prefix mask, cap): 133 us in 560 CTAs; the backward call took
    // 437 us with 140 and 267 us with 560 when the cluster was added.
    kv.parts = 1;
    while (kv.parts < 8 && args.p.group % (2 * kv.parts) == 0 &&
           static_cast<int64_t>(kv.tiles) * a.kv_heads * kv.parts < 4 * sm_count)
        kv.parts *= 2;
    for (const int odd : {7, 5, 3})
        if (kv.parts == 1 && args.p.group % odd == 0 && static_cast<int64_t>(kv.tiles) * a.kv_heads < 4 * sm_count) kv.parts = odd;
    q.tiles = static_cast<int>((a.tokens_q + kTile - 1) / kTile);
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = static_cast<unsigned>(kv.parts);
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(static_cast<int64_t>(kv.tiles) * a.kv_heads * kv.parts));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = layout(halves).total;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = kv.parts > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, attn_dkv_kernel<T, MODE>, map[0], map[1], map[2], map[3], kv, info);
    if (e != cudaSuccess) return e;
    ++*launches;
    e = tc::launch_pdl(attn_dq_kernel<T, MODE>, dim3(static_cast<unsigned>(static_cast<int64_t>(q.tiles) * a.heads)),
                       dim3(kThreads), layout(halves).total, s, map[0], map[1], map[2], map[3], q, info);
    if (e == cudaSuccess) ++*launches;
    return e;
}

template <typename T>
cudaError_t launch_mode(int mode, const TileArgs &args, const CUtensorMap (&map)[4], const Info &info, int sm_count,
                        cudaStream_t s, int *launches)
{
    if (mode == 0) return launch<T, 0>(args, map, info, sm_count, s, launches);
    if (mode == kCap) return launch<T, kCap>(args, map, info, sm_count, s, launches);
    if (mode == kBias) return launch<T, kBias>(args, map, info, sm_count, s, launches);
    return launch<T, kCap | kBias>(args, map, info, sm_count, s, launches);
}

}  // namespace

size_t packed_attn_workspace_bytes(int64_t tokens_q, int heads)
{
    return static_cast<size_t>(padded_rows(tokens_q)) * (16 + 8 * static_cast<size_t>(heads));
}

cudaError_t launch_packed_attn_backward(const PackedAttn &p, int sm_count, const WaitLimit &limit, cudaStream_t s,
                                        int *launches)
{
    const gn_attn_packed_args &a = p.a;
    if (a.tokens_q == 0 || a.tokens_k == 0) {
        const size_t q = 2u * static_cast<size_t>(a.tokens_q) * a.heads * a.dim;
        const size_t k = 2u * static_cast<size_t>(a.tokens_k) * a.kv_heads * a.dim;
        cudaError_t e = q ? cudaMemsetAsync(p.dq, 0, q, s) : cudaSuccess;
        if (e == cudaSuccess && k) e = cudaMemsetAsync(p.dk, 0, k, s);
        if (e == cudaSuccess && k) e = cudaMemsetAsync(p.dv, 0, k, s);
        return e;
    }
    const bool bf16 = a.format == GN_FORMAT_BF16;
    CUtensorMap map[4];
    if (!encode_heads(&map[0], a.q, bf16, a.tokens_q, a.q_token, a.heads, a.q_head, a.dim) ||
        !encode_heads(&map[1], a.k, bf16, a.tokens_k, a.k_token, a.kv_heads, a.k_head, a.dim) ||
        !encode_heads(&map[2], a.v, bf16, a.tokens_k, a.v_token, a.kv_heads, a.v_head, a.dim) ||
        !encode_heads(&map[3], p.dout, bf16, a.tokens_q, p.dout_token, a.heads, p.dout_head, a.dim))
        return cudaErrorInvalidValue;
    TileArgs args = {};
    args.p = p;
    args.scale_log2 = a.scale * kLog2e;
    args.limit = limit;
    Info info;
    info.padded = padded_rows(a.tokens_q);
    info.span = static_cast<int4 *>(p.workspace);
    info.lse = reinterpret_cast<float *>(info.span + info.padded);
    info.delta = info.lse + info.padded * a.heads;
    const int mode = (a.cap > 0.f ? kCap : 0) | (a.slopes ? kBias : 0);
    return bf16 ? launch_mode<__nv_bfloat16>(mode, args, map, info, sm_count, s, launches)
                : launch_mode<__half>(mode, args, map, info, sm_count, s, launches);
}

}  // namespace gn
