// cattn_few.cu -- attention over the paged cache for few rows: single new tokens, a few
// proposed ones.
//
// Such a call is bound by reading the cache once (2 bytes per token, head and
// channel).  The pages go from memory to the tensor cores as they are: a block of 128
// keys is the A operand of S^T = K Q^T (keys are the accumulator's lanes, rows its
// columns) and, read MN-major, of O^T += V^T P^T.  What has more than 4 bits is on the
// narrow side, and is split into e4m3 numbers that add up to it: a query (its largest
// channel at 2^7) into 2 of bf16's 8 bits, 3 of fp16's 11, whose products go into the same
// accumulator; the weights into 2 or 3, each next one times 2^4, with accumulators of
// their own.  That costs the tensor core's time, of which there is plenty, and no pass
// over the keys: converted to half precision they would cross shared memory three
// times more, which it has no room for at this rate (141 of 128 bytes a cycle).
//
// A page's scales stay out of the products: a thread of the softmax warps has one key,
// and multiplies its scores by the key's; the value's scale goes into the weight as
// 2^(t + log2 scale - m), with m the running maximum of t + log2 scale, and out of the
// weights' sum again.
//
// Each CTA (two on an SM) does an equal part of all blocks (cattn_common.cuh), its
// loads running ahead over the ends of tiles.
#include <algorithm>

#include "cattn_common.cuh"

namespace gn {
namespace cattn {
namespace {

constexpr int kThreads = 256;   // warps: 0 loads, 1 MMA, 2 the MMA's waits, 4-7 softmax
constexpr int kMaxStages = 6;
// Weights: the row's largest at 2^6 when the maximum moves, which it does once a score
// is 2^2 above it: below 448 = 2^8.8, and as far as can be from e4m3's smallest step.
constexpr float kShift = 6.0f, kRescale = 2.0f;
constexpr float kLeastScale = 0x1p-100f;

enum Bar { kQ = 0, kFull, kEmpty = kFull + kMaxStages, kS = kEmpty + kMaxStages, kP = kS + 2, kO = kP + 2, kDrain = kO + 2, kBars };

struct Layout {
    uint32_t q, weights, weights_bytes, ring, rows, tops, bars, words, deal, total;
};

__host__ __device__ inline Layout layout(int n, int parts, int stages)
{
    Layout l;
    const uint32_t operand = static_cast<uint32_t>(parts) * static_cast<uint32_t>(n) * 128u;
    l.q = 0;
    l.weights = operand;
    l.weights_bytes = operand;
    l.ring = 3 * operand;
    l.rows = l.ring + static_cast<uint32_t>(stages) * kTileBytes;   // n x (factor, maximum, rescaling, slope), n x (end, position)
    l.tops = l.rows + static_cast<uint32_t>(n) * 24u;               // 4 x n maxima or sums of a warp
    l.bars = l.tops + 16u * static_cast<uint32_t>(n);
    l.words = l.bars + 8 * kBars;                                   // tensor-memory slot, abort
    l.deal = l.words + 16;
    l.total = l.deal + sizeof(DealRoom);
    return l;
}

struct Row {
    float factor, top, grow, slope;
};

__device__ __forceinline__ int ordered(float v)
{
    const int i = __float_as_int(v);
    return i >= 0 ? i : i ^ 0x7fffffff;
}
__device__ __forceinline__ float from_ordered(int i) { return __int_as_float(i >= 0 ? i : i ^ 0x7fffffff); }

__device__ __forceinline__ void sts_u8(uint32_t addr, uint32_t v)
{
    asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, float (&v)[N])
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

// A key's scales and where they are.
struct KeyScale {
    float k, v;
};

template <typename T, int MODE, int N>
__global__ void __launch_bounds__(kThreads, 2)
    cached_few_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                      const __grid_constant__ CattnArgs args)
{
    constexpr int PARTS = IsBf16<T>::value ? 2 : 3;
    extern __shared__ __align__(1024) uint8_t gbase[];
    const uint32_t base = smem_addr(gbase);
    const gn_cache &c = args.p.c;
    const gn_attn_cached_args &a = args.p.a;
    const Layout lay = layout(N, PARTS, args.stages);
    const auto bar = [&](int i) { return base + lay.bars + 8u * static_cast<uint32_t>(i); };
    const auto stage = [&](int n) { return base + lay.ring + static_cast<uint32_t>(n % args.stages) * kTileBytes; };
    volatile uint32_t *words = reinterpret_cast<volatile uint32_t *>(gbase + lay.words);
    volatile int *abort = reinterpret_cast<volatile int *>(words + 1);
    Row *rows = reinterpret_cast<Row *>(gbase + lay.rows);
    int2 *ends = reinterpret_cast<int2 *>(gbase + lay.rows + N * sizeof(Row));
    float *tops = reinterpret_cast<float *>(gbase + lay.tops);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kBars; ++i) mbar_init(bar(i), i == kQ || i == kP || i == kP + 1 ? 4 : 1);
        *abort = (*reinterpret_cast<volatile unsigned int *>(args.limit.status) != 0u) ? 1 : 0;
        mbar_init_fence();
        prefetch_tensormap(&map_k);
        prefetch_tensormap(&map_v);
    }
    constexpr uint32_t kColumns = 2 * N + PARTS * N <= 128 ? 128 : 256;
    if (warp == 1) {
        tmem_alloc(base + lay.words, kColumns);
        tmem_relinquish();
    }
    tc::griddep_wait();
    const Part part = deal(args, *reinterpret_cast<DealRoom *>(gbase + lay.deal), gridDim.x);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    // (only now: a kernel that starts early must not find tensor memory that a
    // CTA of this one has yet to take)
    if (threadIdx.x == 0) tc::griddep_launch_dependents();
    const uint32_t tmem = words[0], t_s = tmem, t_o = tmem + 2 * N;
    const bool skip = *abort != 0;

    Walk walk(args);
    walk.start(part.seq, part.offset, skip ? 0 : part.count);
    Segment g;
    if (warp == 0) {
        int n = 0;                    // tiles so far: keys and values by turns
        bool go = true;
        while (go && walk.next(g)) {
            const int keys = keys_of(args, g.s, g.run);
            int key = g.b0 * kTile + lane * args.chunk;
            bool mine = lane * args.chunk < kTile && key < keys;
            int page = mine ? page_for(args, g.seq, key) : 0;
            for (int b = g.b0; go && b < g.b1; ++b) {
                const int key_now = key, page_now = page;
                const bool now = mine;
                key += kTile;
                mine = lane * args.chunk < kTile && key < keys && b + 1 < g.b1;
                if (mine) page = page_for(args, g.seq, key);
                for (int e = 0; go && e < 2; ++e, ++n) {
                    const int st = n % args.stages;
                    if (n >= args.stages && !wait_warp(bar(kEmpty + st), (n / args.stages - 1) & 1, abort, args.limit)) {
                        go = false;
                        break;
                    }
                    load_pages(stage(n), e ? &map_v : &map_k, args, key_now, page_now, g.hk, bar(kFull + st), now);
                }
            }
        }
        // nothing is left in flight when the CTA goes on, whatever became of the others
        for (int k = max(0, n - args.stages); k < n; ++k)
            tc::drain(bar(kFull + k % args.stages), (k / args.stages) & 1, args.limit.timeout_ns);
        __syncwarp();
    } else if (warp == 1 || warp == 2) {
        const bool waits = warp == 2;
        const int steps = (c.dim + 31) / 32;
        const uint32_t is = instruction_e4m3(N, false), io = instruction_e4m3(PARTS * N, true);
        const auto loaded = [&](int n) { wait_warp(bar(kFull + n % args.stages), (n / args.stages) & 1, abort, args.limit); };
        const auto scores = [&](int n) {              // block n's, into buffer n & 1
            if (elect_one()) {
#pragma unroll
                for (int p = 0; p < PARTS; ++p) {
                    const uint64_t dk = sw128_kmajor_desc(stage(2 * n)), dq = sw128_kmajor_desc(base + lay.q + p * N * 128u);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (k >= steps) break;
                        umma_e4m3(t_s + (n & 1) * N, dk + 2 * k, dq + 2 * k, is, p > 0 || k > 0);
                    }
                }
            }
            __syncwarp();
            commit(bar(kS + (n & 1)));
            commit(bar(kEmpty + 2 * n % args.stages));
        };
        int n = 0, segment = 0;                       // blocks, tiles so far
        for (; walk.next(g); ++segment) {
            if (waits) {
                wait_warp(bar(kQ), segment & 1, abort, args.limit);
                loaded(2 * n);
            }
            hand_over();
            if (!waits) {
                tc_fence_after_sync();
                scores(n);
            }
            for (int b = g.b0; b < g.b1; ++b, ++n) {
                if (b + 1 < g.b1) {
                    // (the buffer's last scores have been read: their weights were waited for)
                    if (waits) loaded(2 * n + 2);
                    hand_over();
                    if (!waits) scores(n + 1);
                }
                if (waits) {
                    loaded(2 * n + 1);
                    wait_warp(bar(kP + (n & 1)), (n >> 1) & 1, abort, args.limit);
                }
                hand_over();
                if (!waits) {
                    tc_fence_after_sync();
                    const uint64_t dv = sw128_mnmajor_desc(stage(2 * n + 1));
                    const uint64_t dw = sw128_kmajor_desc(base + lay.weights + (n & 1) * lay.weights_bytes);
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) umma_e4m3(t_o, dv + k * (4096u >> 4), dw + 2 * k, io, b > g.b0 || k > 0);
                    }
                    __syncwarp();
                    commit(bar(kEmpty + (2 * n + 1) % args.stages));
                    commit(bar(kO + (n & 1)));
                }
            }
        }
        if (!waits && n > 0) {
            commit(bar(kDrain));
            tc::drain(bar(kDrain), 0, args.limit.timeout_ns);
        }
    } else if (warp >= 4) {
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const int r = (warp & 3) * 32 + lane;
        // this thread's key within the block: its place in the weights' rows
        const uint32_t place = base + lay.weights + static_cast<uint32_t>(r & 15);
        const uint32_t piece = static_cast<uint32_t>(r >> 4);
        float by = args.scale_log2, inv_cap = 0.f;
        if (MODE & kCap) {
            by = a.cap * kLog2e;
            inv_cap = a.scale / a.cap;
        }
        int n = 0;
        while (walk.next(g)) {
            const int first_token = g.run * args.tokens, count = min(args.tokens, g.s.end - g.s.begin - first_token);
            const int live = count * args.heads, keys = keys_of(args, g.s, g.run);
            // the tile's rows: what they see, and their queries in parts
            if (r < live) {
                const int pos = g.s.first_place() + first_token + r / args.heads, h = g.first_head + r % args.heads;
                ends[r] = make_int2(a.causal ? min(max(pos + 1, 0), g.s.length) : g.s.length, pos);
                rows[r].top = -INFINITY;
                rows[r].slope = (MODE & kBias) && a.slopes && h < args.p.group ? __ldg(a.slopes + g.hk * args.p.group + h) * kLog2e : 0.f;
            }
            const int all = a.causal ? min(max(g.s.first_place() + first_token + 1, 0), g.s.length) : g.s.length;
            for (int q = warp & 3; q < live; q += 4) {
                const int h = g.first_head + q % args.heads;
                const int64_t token = g.s.begin + first_token + q / args.heads;
                const bool there = h < args.p.group && 4 * lane < c.dim;
                const float4 f = there ? load4<T>(a.q, token * a.q_token + (g.hk * args.p.group + h) * a.q_head, lane, c.dim)
                                       : make_float4(0.f, 0.f, 0.f, 0.f);
                float x[4] = {f.x, f.y, f.z, f.w}, most = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) most = max_nan(most, fabsf(x[e]));
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, o));
                const int shift = most < INFINITY ? query_shift(most) : 0;
                const float up = most < INFINITY ? power_of_two(shift) : NAN;
                uint32_t w[PARTS];
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] *= up;
                split_e4m3<PARTS>(x, w);
                const uint32_t at = base + lay.q + q * 128u + (((lane >> 2) ^ (q & 7u)) << 4) + (lane & 3u) * 4u;
#pragma unroll
                for (int p = 0; p < PARTS; ++p)
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + p * N * 128u), "r"(w[p]) : "memory");
                if (lane == 0) rows[q].factor = power_of_two(-shift);
            }
            fence_proxy_async_smem();
            named_sync(1, 128);
            if (lane == 0) mbar_arrive(bar(kQ));
            float l[N];
#pragma unroll
            for (int i = 0; i < N; ++i) l[i] = 0.f;
            // the scales of this thread's key, a block ahead
            const auto scales_of = [&](int j) {
                KeyScale s = {0.f, 0.f};
                const int page = j < keys ? cache::page_of(c, g.seq, j / c.page_size) : -1;
                if (page >= 0) {
                    s.k = __ldg(c.k_scales + static_cast<int64_t>(page) * c.kv_heads + g.hk);
                    s.v = __ldg(c.v_scales + static_cast<int64_t>(page) * c.kv_heads + g.hk);
                }
                return s;
            };
            KeyScale ahead = scales_of(g.b0 * kTile + r);
            for (int b = g.b0; b < g.b1; ++b, ++n) {
                const int first = b * kTile, j = first + r;
                const bool masked = first + kTile > all;
                const KeyScale key = ahead;
                if (b + 1 < g.b1) ahead = scales_of(j + kTile);
                const float vs = key.v < kLeastScale ? kLeastScale : key.v, inv_vs = 1.0f / vs, log_vs = log2f(vs);
                const float ks = (MODE & kCap) ? key.k * inv_cap : key.k * by;
                wait_warp(bar(kS + (n & 1)), (n >> 1) & 1, abort, args.limit);
                tc_fence_after_sync();
                float s[N];
                tmem_ld_cols<N>(t_s + (n & 1) * N + lanes, s);
                bool grew = b == g.b0;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    if (i >= live) break;             // (the same for all: rows that are not there cost nothing)
                    const Row row = rows[i];
                    float t = s[i] * (ks * row.factor);
                    if (MODE & kCap) t = tanh_fast(t) * by;
                    if ((MODE & kBias) || masked) {
                        const int2 e = ends[i];
                        if (MODE & kBias) t = fmaf(-row.slope, fabsf(static_cast<float>(e.y - j)), t);
                        t = t + log_vs;
                        if (masked) t = j < e.x ? t : -INFINITY;
                    } else {
                        t = t + log_vs;
                    }
                    s[i] = t;
                    grew = grew || t > row.top + (kShift + kRescale);
                }
                // the maxima are only looked for when a score is far above one of them
                if (bar_any(1, 128, grew)) {
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        if (i >= live) break;
                        const int top = __reduce_max_sync(0xffffffffu, ordered(s[i] == s[i] ? s[i] : -INFINITY));
                        if (lane == 0) tops[(warp & 3) * N + i] = from_ordered(top);
                    }
                    named_sync(1, 128);
                    if (r < live) {
                        const float old = rows[r].top;
                        const float top = fmaxf(fmaxf(tops[r], tops[N + r]), fmaxf(tops[2 * N + r], tops[3 * N + r]));
                        // (a row's maximum moves for its own scores only: not by what another row's keys hold)
                        const bool up = top > old + (kShift + kRescale);
                        rows[r].grow = up && old != -INFINITY ? ex2_approx(old - (top - kShift)) : 1.0f;
                        if (up) rows[r].top = top - kShift;
                    }
                    named_sync(1, 128);
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        if (i >= live) break;
                        l[i] *= rows[i].grow;
                    }
                    if (b > g.b0) {
                        wait_warp(bar(kO + ((n - 1) & 1)), ((n - 1) >> 1) & 1, abort, args.limit);
                        tc_fence_after_sync();
#pragma unroll 1
                        for (int q = 0; q < PARTS * N / 16; ++q) {
                            uint32_t u[16];
                            tmem_ld16(t_o + lanes + 16 * q, u);
                            tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < 16; ++k) u[k] = __float_as_uint(__uint_as_float(u[k]) * rows[(16 * q + k) % N].grow);
                            tmem_st16(t_o + lanes + 16 * q, u);
                        }
                        tmem_wait_st();
                    }
                }
                // the weights' buffer is free once the products of two blocks ago are done
                if (n >= 2) wait_warp(bar(kO + (n & 1)), ((n - 2) >> 1) & 1, abort, args.limit);
                const uint32_t to = place + (n & 1) * lay.weights_bytes;
#pragma unroll
                for (int i = 0; i < N; i += 2) {
                    if (i >= live) break;
                    float p[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float top = rows[i + e].top;
                        // (0 x inv_vs would not be 0 if an unseen key's scale is no number)
                        const bool seen = s[i + e] != -INFINITY;
                        p[e] = seen ? ex2_approx(s[i + e] - (top == -INFINITY ? 0.f : top)) : 0.f;
                        l[i + e] = seen ? fmaf(p[e], inv_vs, l[i + e]) : l[i + e];
                    }
#pragma unroll
                    for (int q = 0; q < PARTS; ++q) {
                        const uint32_t w = e4m3_pair(p[0], p[1]);
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            sts_u8(to + static_cast<uint32_t>(q * N + i + e) * 128u + ((piece ^ ((i + e) & 7u)) << 4), w >> (8 * e));
                        const float2 v = e4m3_values(w);
                        p[0] = (p[0] - v.x) * 16.0f;
                        p[1] = (p[1] - v.y) * 16.0f;
                    }
                }
                if (first + kTile > keys) {
                    // what lies behind the sequence has weight 0, but 0 x NaN is not 0
                    const int nv = 2 * n + 1;
                    wait_warp(bar(kFull + nv % args.stages), (nv / args.stages) & 1, abort, args.limit);
                    if (j >= keys) zero_tile_row(stage(nv), r);
                }
                fence_proxy_async_smem();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kP + (n & 1)));
            }
            wait_warp(bar(kO + ((n - 1) & 1)), ((n - 1) >> 1) & 1, abort, args.limit);
            tc_fence_after_sync();
            named_sync(1, 128);           // the maxima in `tops` have been read
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (i >= live) break;
                const float sum = warp_sum(l[i]);
                if (lane == 0) tops[(warp & 3) * N + i] = sum;
            }
            named_sync(1, 128);
            const bool whole = g.b0 == 0 && g.b1 == g.total, good = *abort == 0;
            float *to = piece_of(args, blockIdx.x, g.b0 == 0 ? 1 : 0);
            float o[N];
            tmem_ld_cols<N>(t_o + lanes, o);
            float step = 1.0f / 16.0f;
#pragma unroll
            for (int q = 1; q < PARTS; ++q, step *= 1.0f / 16.0f) {
                float more[N];
                tmem_ld_cols<N>(t_o + q * N + lanes, more);
#pragma unroll
                for (int i = 0; i < N; ++i) o[i] = fmaf(more[i], step, o[i]);
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (i >= live) break;
                const int h = g.first_head + i % args.heads;
                const int64_t token = g.s.begin + first_token + i / args.heads;
                if (h >= args.p.group || !good) continue;
                const float sum = (tops[i] + tops[N + i]) + (tops[2 * N + i] + tops[3 * N + i]), top = rows[i].top;
                if (whole) {
                    const int64_t head = g.hk * args.p.group + h;
                    if (r < c.dim) static_cast<T *>(a.out)[(token * a.heads + head) * c.dim + r] = from_float<T>(sum == 0.f ? 0.f : o[i] / sum);
                    if (r == 0) a.lse[head * a.tokens + token] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
                } else {
                    if (r < c.dim) to[2 * N + i * c.dim + r] = o[i];
                    if (r == 0) {
                        to[i] = top;
                        to[N + i] = sum;
                    }
                }
            }
            tc_fence_before_sync();
            named_sync(1, 128);           // rows and tops are free
        }
    }
    __syncwarp();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, kColumns);
    }
}

using Kernel = void (*)(const CUtensorMap, const CUtensorMap, const CattnArgs);

template <typename T, int MODE, int N>
cudaError_t launch(const CattnArgs &args, const CUtensorMap &mk, const CUtensorMap &mv, int ctas, cudaStream_t s)
{
    constexpr int PARTS = IsBf16<T>::value ? 2 : 3;
    CattnArgs a = args;
    // (two CTAs on an SM: 113 KB each)
    a.stages = kMaxStages;
    while (layout(N, PARTS, a.stages).total > 113 * 1024) --a.stages;
    static std::atomic<uint64_t> done{0}, wide{0};
    const Kernel kernel = cached_few_kernel<T, MODE, N>;
    cudaError_t e = allow_shared(reinterpret_cast<const void *>(kernel), 113 * 1024, done);
    if (e == cudaSuccess) e = allow_clusters(reinterpret_cast<const void *>(kernel), wide);
    if (e != cudaSuccess) return e;
    return tc::launch_pdl(kernel, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), layout(N, PARTS, a.stages).total, s, mk, mv, a);
}

template <typename T, int MODE>
cudaError_t launch_rows(const CattnArgs &a, const CUtensorMap &mk, const CUtensorMap &mv, int ctas, cudaStream_t s)
{
    return a.rows == 16 ? launch<T, MODE, 16>(a, mk, mv, ctas, s) : launch<T, MODE, 32>(a, mk, mv, ctas, s);
}

template <typename T>
cudaError_t launch_mode(const CattnArgs &a, const CUtensorMap &mk, const CUtensorMap &mv, int ctas, cudaStream_t s)
{
    const int mode = (a.p.a.cap > 0.f ? kCap : 0) | (a.p.a.slopes ? kBias : 0);
    if (mode == 0) return launch_rows<T, 0>(a, mk, mv, ctas, s);
    if (mode == kCap) return launch_rows<T, kCap>(a, mk, mv, ctas, s);
    if (mode == kBias) return launch_rows<T, kBias>(a, mk, mv, ctas, s);
    return launch_rows<T, kCap | kBias>(a, mk, mv, ctas, s);
}

}  // namespace

cudaError_t launch_cached_few(const CattnArgs &a, const CUtensorMap &mk, const CUtensorMap &mv, int ctas, cudaStream_t s)
{
    return a.p.a.format == GN_FORMAT_BF16 ? launch_mode<__nv_bfloat16>(a, mk, mv, ctas, s) : launch_mode<__half>(a, mk, mv, ctas, s);
}

}  // namespace cattn
}  // namespace gn
