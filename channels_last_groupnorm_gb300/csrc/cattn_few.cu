// cattn_few.cu -- attention over the paged cache for few rows: single new tokens, a few
// proposed ones.
//
// Such a call is bound by reading the cache once (2 bytes per token, head and
// channel).  The pages go from memory to the tensor cores as they are: a block of 128
// keys is the A operand of S^T = K Q^T (keys are the accumulator's lanes, rows its
// columns) and, read MN-major, of O^T += V^T P^T.  What has more bits is on the
// narrow side, and is split into numbers of 8 bits that add up to it: a query (its largest
// channel at 2^7) into 2 (bf16's 8 bits) or 3 (fp16's 11) of e4m3, whose products go into the same
// accumulator; the weights, rounded to fp16, into 3 or 4 of e5m2, each next one times 2^3, with
// accumulators of their own.  (e5m2 for its range: a long context's small weights, together
// most of a sum, are held to as many bits as the large ones.  Two or three parts of e4m3, which
// hold none under 2^-18 of the largest, took as long for single tokens -- 64 of 32 heads on 8 over
// 3000 keys 85 us replayed either way -- and 176 us instead of 182 for 64 x 4 tokens of 64
// heads.)  That costs the tensor core's time, of which there is plenty, and no pass
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

constexpr int kThreads = 256;   // warps: 0 loads, 1 MMA, 2 the MMA's waits, 3 the next tile's rows, 4-7 softmax
constexpr int kSegments = 32;  // that are found at a time
constexpr int kScales = 4;      // blocks whose scales are in shared memory
constexpr int kMaxStages = 6;
// Weights: the row's largest at 2^11 when the maximum moves, which it does once a score
// is 2^4 above it: fp16's largest number is under 2^16, its least normal one 2^-14, so weights of
// 2^-25 of the row's largest still have all their bits.
constexpr float kShift = 11.0f, kRescale = 4.0f;
constexpr float kLeastScale = 0x1p-100f;

enum Bar { kQ = 0, kQFree = 2, kFull = kQFree + 2, kEmpty = kFull + kMaxStages, kS = kEmpty + kMaxStages, kP = kS + 2, kO = kP + 2,
           kScale = kO + 2, kDrain = kScale + kScales, kBars };

// One row of a tile: its scores' factor, its running maximum, the bias and the first place of
// the block of 128 that the query stands in; what the maximum's last move makes of sums, and the
// keys that it sees; where its results go (-1: it has none); the query's place in its block.
// (Apart, since fp32 holds no odd place past 2^24: what blocks are away and what places within
// one are is exact.)
struct __align__(16) Row {
    float factor, top, slope, block;
    float grow;
    int end;
    int64_t out, lse;
    float within, pad;
};

struct Layout {
    uint32_t q, operand, weights, ring, rows, tops, scales, bars, words, deal, work, total;
};

// Weights lie as the threads have them, a key's next to each other ([128 keys][parts][n],
// MN-major, swizzled over rows of 64 bytes): whole vectors are stored, where
// [rows][keys] would take a byte at a time (48 of them a thread in three parts).
constexpr uint32_t kWeightRow = 64, kWeightBytes = kTile * kWeightRow;

// Descriptor of the weights as the B operand: 8 keys after 8 keys (stride offset); the
// swizzle mode is 4 for 64 bytes.
__device__ __forceinline__ uint64_t weights_desc(uint32_t smem)
{
    uint64_t d = static_cast<uint64_t>((smem & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(1u) << 16;
    d |= static_cast<uint64_t>((8u * kWeightRow) >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(4u) << 61;
    return d;
}

__host__ __device__ constexpr Layout layout(int n, int parts, int stages)
{
    Layout l = {};
    const uint32_t operand = static_cast<uint32_t>(parts) * static_cast<uint32_t>(n) * 128u;
    l.operand = operand;
    l.q = 0;                                                        // two of each: this tile's and the next one's,
    l.weights = 2 * operand;                                        // this block's and the next one's
    l.ring = l.weights + 2 * kWeightBytes;
    l.rows = l.ring + static_cast<uint32_t>(stages) * kTileBytes;   // 2 x n Row
    l.tops = l.rows + 2 * static_cast<uint32_t>(n) * sizeof(Row);   // 4 x n maxima or sums of a warp
    l.scales = l.tops + 16u * static_cast<uint32_t>(n);             // kScales x 16 chunks
    l.bars = l.scales + kScales * 16 * sizeof(float4);
    l.words = l.bars + 8 * kBars;                                   // tensor-memory slot, abort
    l.deal = l.words + 16;
    l.work = l.deal + sizeof(DealRoom);
    l.total = l.work + sizeof(WorkList<kSegments>);
    return l;
}

// (two CTAs on an SM: 113 KB each)
constexpr uint32_t kRoom = 113 * 1024;
__host__ __device__ constexpr int stages_of(int n, int parts)
{
    int stages = kMaxStages;
    while (layout(n, parts, stages).total > kRoom) --stages;
    return stages;
}

__device__ __forceinline__ int ordered(float v)
{
    const int i = __float_as_int(v);
    return i >= 0 ? i : i ^ 0x7fffffff;
}
__device__ __forceinline__ float from_ordered(int i) { return __int_as_float(i >= 0 ? i : i ^ 0x7fffffff); }

// e5m2 is the upper half of fp16: four values' bytes, cut off there, ...
__device__ __forceinline__ uint32_t e5m2_four(uint32_t lo, uint32_t hi) { return __byte_perm(lo, hi, 0x7531); }

// ... 8 times what that leaves of two of them (exact: at most 8 bits, under a quarter of the value), ...
__device__ __forceinline__ uint32_t eight_times_rest(uint32_t v)
{
    const uint32_t near = v & 0xff00ff00u;
    const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&v), *reinterpret_cast<const __half2 *>(&near));
    const __half2 r = __hmul2(d, __float2half2_rn(8.0f));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// ... and for the last of the parts rounded to nearest.
__device__ __forceinline__ uint32_t e5m2_four_rounded(uint32_t lo, uint32_t hi)
{
    return e5m2_pair_half(lo) | e5m2_pair_half(hi) << 16;
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

template <typename T>
__host__ __device__ constexpr int query_parts() { return IsBf16<T>::value ? 2 : 3; }

template <typename T, int MODE>
__global__ void __launch_bounds__(kThreads, 2)
    cached_few_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                      const __grid_constant__ CattnArgs args)
{
    constexpr int N = kFewTile, PARTS = query_parts<T>(), WEIGHTS = PARTS + 1, STAGES = stages_of(N, PARTS);
    constexpr Layout lay = layout(N, PARTS, STAGES);
    constexpr int SIDE = 4;      // rows that are worked on side by side
    extern __shared__ __align__(1024) uint8_t gbase[];
    const uint32_t base = smem_addr(gbase);
    const gn_cache &c = args.p.c;
    const gn_attn_cached_args &a = args.p.a;
    const auto bar = [&](int i) { return base + lay.bars + 8u * static_cast<uint32_t>(i); };
    const auto stage = [&](int n) { return base + lay.ring + static_cast<uint32_t>(n % STAGES) * kTileBytes; };
    volatile uint32_t *words = reinterpret_cast<volatile uint32_t *>(gbase + lay.words);
    volatile int *abort = reinterpret_cast<volatile int *>(words + 1);
    Row *all_rows = reinterpret_cast<Row *>(gbase + lay.rows);
    float4 *scales = reinterpret_cast<float4 *>(gbase + lay.scales);
    float *tops = reinterpret_cast<float *>(gbase + lay.tops);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kBars; ++i) mbar_init(bar(i), i == kQFree || i == kQFree + 1 || i == kP || i == kP + 1 ? 4 : 1);
        *abort = (*reinterpret_cast<volatile unsigned int *>(args.limit.status) != 0u) ? 1 : 0;
        mbar_init_fence();
        prefetch_tensormap(&map_k);
        prefetch_tensormap(&map_v);
    }
    constexpr uint32_t kColumns = 128;
    static_assert(2 * N + WEIGHTS * N <= kColumns, "a CTA's tensor memory");
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

    Reader<kSegments> work(*reinterpret_cast<WorkList<kSegments> *>(gbase + lay.work));
    Segment g;
    if (warp == 0) {
        // The pages, and each chunk's scales by the lane that brings it: a block's are
        // asked for ahead of its loads and stored behind them.  (Their slot was last read
        // by the softmax kScales blocks ago, whose products the values' stage has waited for.)
        const float by = (MODE & kCap) ? a.scale / a.cap : args.scale_log2;
        int n = 0, block = 0;         // tiles so far (keys and values by turns), blocks so far
        bool go = true;
        begin_work(args);
        Walk walk(args);
        walk.start(part.seq, part.offset, skip ? 0 : part.count, part.first);
        while (work.next(g, [&](WorkList<kSegments> &w) { fill_work(w, walk, part); })) {
            if (!go) continue;
            const int keys = keys_of(args, g.s, g.run);
            int key = g.b0 * kTile + lane * args.chunk;
            bool mine = lane * args.chunk < kTile && key < keys;
            int page = mine ? page_for(args, g.seq, key) : 0;
            for (int b = g.b0; go && b < g.b1; ++b, ++block) {
                const int key_now = key, page_now = page;
                const bool now = mine;
                float ks = 0.f, vs = 0.f;
                if (now && page_now < c.pages) {
                    ks = __ldg(c.k_scales + static_cast<int64_t>(page_now) * c.kv_heads + g.hk);
                    vs = __ldg(c.v_scales + static_cast<int64_t>(page_now) * c.kv_heads + g.hk);
                }
                key += kTile;
                mine = lane * args.chunk < kTile && key < keys && b + 1 < g.b1;
                if (mine) page = page_for(args, g.seq, key);
                for (int e = 0; go && e < 2; ++e, ++n) {
                    const int st = n % STAGES;
                    if (n >= STAGES && !wait_warp(bar(kEmpty + st), (n / STAGES - 1) & 1, abort, args.limit)) {
                        go = false;
                        break;
                    }
                    load_pages(stage(n), e ? &map_v : &map_k, args, key_now, page_now, g.hk, bar(kFull + st), now);
                }
                vs = vs < kLeastScale ? kLeastScale : vs;
                if (lane < 16) scales[(block % kScales) * 16 + lane] = make_float4(ks * by, log2f(vs), kSumDown / vs, 0.f);
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kScale + block % kScales));
            }
        }
        // nothing is left in flight when the CTA goes on, whatever became of the others
        for (int k = max(0, n - STAGES); k < n; ++k)
            tc::drain(bar(kFull + k % STAGES), (k / STAGES) & 1, args.limit.timeout_ns);
        __syncwarp();
    } else if (warp == 1 || warp == 2) {
        const bool waits = warp == 2;
        const int steps = (c.dim + 31) / 32;
        const uint32_t is = instruction_e4m3(N, false), io = instruction_e4m3(WEIGHTS * N, true) | 1u << 16 | 1u << 10;
        const auto loaded = [&](int n) { wait_warp(bar(kFull + n % STAGES), (n / STAGES) & 1, abort, args.limit); };
        const auto scores = [&](int n, int q) {       // block n's with query buffer q, into buffer n & 1
            if (elect_one()) {
#pragma unroll
                for (int p = 0; p < PARTS; ++p) {
                    const uint64_t dk = sw128_kmajor_desc(stage(2 * n)), dq = sw128_kmajor_desc(base + lay.q + q * lay.operand + p * N * 128u);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (k >= steps) break;
                        umma_e4m3(t_s + (n & 1) * N, dk + 2 * k, dq + 2 * k, is, p > 0 || k > 0);
                    }
                }
            }
            __syncwarp();
            commit(bar(kS + (n & 1)));
            commit(bar(kEmpty + 2 * n % STAGES));
        };
        int n = 0, segment = 0;                       // blocks, tiles so far
        for (; work.next(g); ++segment) {
            if (waits) {
                wait_warp(bar(kQ + (segment & 1)), (segment >> 1) & 1, abort, args.limit);
                loaded(2 * n);
            }
            hand_over();
            if (!waits) {
                tc_fence_after_sync();
                scores(n, segment & 1);
            }
            for (int b = g.b0; b < g.b1; ++b, ++n) {
                if (b + 1 < g.b1) {
                    // (the buffer's last scores have been read: their weights were waited for)
                    if (waits) loaded(2 * n + 2);
                    hand_over();
                    if (!waits) scores(n + 1, segment & 1);
                }
                if (waits) {
                    loaded(2 * n + 1);
                    wait_warp(bar(kP + (n & 1)), (n >> 1) & 1, abort, args.limit);
                }
                hand_over();
                if (!waits) {
                    tc_fence_after_sync();
                    const uint64_t dv = sw128_mnmajor_desc(stage(2 * n + 1));
                    const uint64_t dw = weights_desc(base + lay.weights + (n & 1) * kWeightBytes);
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) umma_e4m3(t_o, dv + k * (4096u >> 4), dw + k * (32u * kWeightRow >> 4), io, b > g.b0 || k > 0);
                    }
                    __syncwarp();
                    commit(bar(kEmpty + (2 * n + 1) % STAGES));
                    commit(bar(kO + (n & 1)));
                }
            }
        }
        if (!waits && n > 0) {
            commit(bar(kDrain));
            tc::drain(bar(kDrain), 0, args.limit.timeout_ns);
        }
    } else if (warp == 3) {
        // the rows of a tile while the one before it is worked on
        for (int segment = 0; work.next(g); ++segment) {
            const int buffer = segment & 1;
            Row *rows = all_rows + buffer * N;
            const int first_token = g.run * args.tokens, live = min(args.tokens, g.s.end - g.s.begin - first_token) * args.heads;
            if (segment >= 2) wait_warp(bar(kQFree + buffer), ((segment >> 1) - 1) & 1, abort, args.limit);
            if (lane < N) {
                const int h = g.first_head + lane % args.heads, i = first_token + lane / args.heads, place = g.s.first_place() + i;
                const int64_t token = g.s.begin + i, head = g.hk * args.p.group + h;
                const bool there = lane < live && h < args.p.group;
                Row row;
                row.factor = row.grow = 1.0f;
                // (the last four rows that are worked on together may be past the tile's: no score is above
                // their maximum, and nothing is made of their weights)
                row.top = lane < live ? -INFINITY : INFINITY;
                row.slope = (MODE & kBias) && a.slopes && there ? __ldg(a.slopes + head) * kLog2e : 0.f;
                row.block = static_cast<float>(place & ~(kTile - 1));
                row.within = static_cast<float>(place & (kTile - 1));
                row.end = a.causal ? min(max(place + 1, 0), g.s.held) : g.s.held;
                row.out = there ? token * a.heads + head : -1;
                row.lse = head * a.tokens + token;
                rows[lane] = row;
            }
            __syncwarp();
            // (eight rows on their way together, and the next eight while these are split)
            int h = g.first_head;
            int64_t token = g.s.begin + first_token;
            float4 ahead[8];
            const auto load_rows = [&](int q0) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const bool there = q0 + e < live && h < args.p.group && 4 * lane < c.dim;
                    ahead[e] = there ? load4<T>(a.q, token * a.q_token + (g.hk * args.p.group + h) * a.q_head, lane, c.dim)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
                    if (++h == g.first_head + args.heads) {
                        h = g.first_head;
                        ++token;
                    }
                }
            };
            load_rows(0);
#pragma unroll 1
            for (int q0 = 0; q0 < live; q0 += 8) {
                float4 f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = ahead[e];
                if (q0 + 8 < live) load_rows(q0 + 8);
                float most[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) most[e] = max_nan3(max_nan(fabsf(f[e].x), fabsf(f[e].y)), f[e].z, f[e].w);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
#pragma unroll
                    for (int e = 0; e < 8; ++e) most[e] = max_nan(most[e], __shfl_xor_sync(0xffffffffu, most[e], o));
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int q = q0 + e;
                    if (q >= live) break;
                    // (infinities too: their products with keys of either sign are no numbers)
                    const int shift = most[e] < INFINITY ? query_shift(most[e]) : 0;
                    const float up = most[e] < INFINITY ? power_of_two(shift) : NAN;
                    uint32_t lo[PARTS], hi[PARTS];
                    split_e4m3<PARTS>(f[e].x * up, f[e].y * up, lo);
                    split_e4m3<PARTS>(f[e].z * up, f[e].w * up, hi);
                    const uint32_t at = base + lay.q + buffer * lay.operand + q * 128u + (((lane >> 2) ^ (q & 7u)) << 4) + (lane & 3u) * 4u;
#pragma unroll
                    for (int p = 0; p < PARTS; ++p)
                        asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + p * N * 128u), "r"(lo[p] | hi[p] << 16) : "memory");
                    if (lane == 0) rows[q].factor = power_of_two(-shift);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kQ + buffer));
        }
    } else if (warp >= 4) {
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const int r = (warp & 3) * 32 + lane;
        // this thread's key within the block: its row of weights, and what its 16-byte pieces'
        // numbers are swizzled with
        const uint32_t place = base + lay.weights + static_cast<uint32_t>(r) * kWeightRow;
        const uint32_t flip = r >> 1 & 3u;
        const int my_chunk = r / args.chunk;
        int n = 0;
        for (int segment = 0; work.next(g); ++segment) {
            Row *rows = all_rows + (segment & 1) * N;
            const int first_token = g.run * args.tokens, live = min(args.tokens, g.s.end - g.s.begin - first_token) * args.heads;
            const int keys = keys_of(args, g.s, g.run);
            const int all = a.causal ? min(max(g.s.first_place() + first_token + 1, 0), g.s.held) : g.s.held;
            wait_warp(bar(kQ + (segment & 1)), (segment >> 1) & 1, abort, args.limit);
            float l[N];
#pragma unroll
            for (int i = 0; i < N; ++i) l[i] = 0.f;
            for (int b = g.b0; b < g.b1; ++b, ++n) {
                const int first = b * kTile, j = first + r;
                const bool masked = first + kTile > all;
                wait_warp(bar(kScale + n % kScales), (n / kScales) & 1, abort, args.limit);
                const float4 key = scales[(n % kScales) * 16 + my_chunk];
                const float ks = key.x, log_vs = key.y, inv_vs = key.z;
                wait_warp(bar(kS + (n & 1)), (n >> 1) & 1, abort, args.limit);
                tc_fence_after_sync();
                float s[N];
                tmem_ld_cols<N>(t_s + (n & 1) * N + lanes, s);
                bool grew = b == g.b0;
                // (some rows at a time: the tile may have fewer, what the others hold goes
                // nowhere, and they run side by side)
#pragma unroll
                for (int i = 0; i < N; i += SIDE) {
                    if (i >= live) break;
                    float4 row[SIDE];
                    int end[SIDE];
#pragma unroll
                    for (int e = 0; e < SIDE; ++e) {
                        row[e] = *reinterpret_cast<const float4 *>(&rows[i + e]);
                        if (masked) end[e] = rows[i + e].end;
                    }
                    float x[SIDE];
#pragma unroll
                    for (int e = 0; e < SIDE; ++e) x[e] = s[i + e] * (ks * row[e].x);
                    if (MODE & kCap) tanh_all(x, 1.0f);
#pragma unroll
                    for (int e = 0; e < SIDE; ++e) {
                        float t = x[e];
                        if (MODE & kCap) t *= a.cap * kLog2e;
                        if (MODE & kBias) {
                            const float away = (row[e].w - static_cast<float>(first)) + (rows[i + e].within - static_cast<float>(r));
                            t = fmaf(-row[e].z, fabsf(away), t);
                        }
                        t += log_vs;
                        if (masked) t = j < end[e] ? t : -INFINITY;
                        s[i + e] = t;
                        grew = grew || t > row[e].y + (kShift + kRescale);
                    }
                }
                // the maxima are only looked for when a score is far above one of them
                if (bar_any(1, 128, grew)) {
#pragma unroll
                    for (int i = 0; i < N; i += 4) {
                        if (i >= live) break;
                        int top[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            top[e] = __reduce_max_sync(0xffffffffu, ordered(s[i + e] == s[i + e] ? s[i + e] : -INFINITY));
                        if (lane == 0)
                            *reinterpret_cast<float4 *>(tops + (warp & 3) * N + i) =
                                make_float4(from_ordered(top[0]), from_ordered(top[1]), from_ordered(top[2]), from_ordered(top[3]));
                    }
                    named_sync(1, 128);
                    if (r < N && r < live) {
                        const float old = rows[r].top;
                        const float top = fmaxf(fmaxf(tops[r], tops[N + r]), fmaxf(tops[2 * N + r], tops[3 * N + r]));
                        // (a row's maximum moves for its own scores only: not by what another row's keys hold)
                        const bool up = top > old + (kShift + kRescale);
                        rows[r].grow = up && old != -INFINITY ? ex2_approx(old - (top - kShift)) : 1.0f;
                        if (up) rows[r].top = top - kShift;
                    }
                    named_sync(1, 128);
#pragma unroll
                    for (int i = 0; i < N; ++i) l[i] *= rows[i].grow;
                    if (b > g.b0) {
                        wait_warp(bar(kO + ((n - 1) & 1)), ((n - 1) >> 1) & 1, abort, args.limit);
                        tc_fence_after_sync();
#pragma unroll 1
                        for (int q = 0; q < WEIGHTS * N / 16; ++q) {
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
                const uint32_t to = place + (n & 1) * kWeightBytes;
                uint32_t packed[WEIGHTS][N / 4] = {};
#pragma unroll
                for (int i = 0; i < N; i += SIDE) {
                    if (i >= live) break;
                    float p[SIDE];
#pragma unroll
                    for (int e = 0; e < SIDE; ++e) {
                        const float top = rows[i + e].top;
                        // (0 x inv_vs would not be 0 if an unseen key's scale is no number)
                        const bool seen = s[i + e] != -INFINITY;
                        p[e] = seen ? ex2_approx(s[i + e] - (top == -INFINITY ? 0.f : top)) : 0.f;
                        l[i + e] = seen ? fmaf(p[e], inv_vs, l[i + e]) : l[i + e];
                    }
                    uint32_t h[SIDE / 2];
#pragma unroll
                    for (int e = 0; e < SIDE / 2; ++e) h[e] = weight_pair(p[2 * e], p[2 * e + 1]);
#pragma unroll
                    for (int q = 0; q < WEIGHTS; ++q)
#pragma unroll
                        for (int e = 0; e < SIDE / 2; e += 2) {
                            packed[q][(i + 2 * e) / 4] = q + 1 < WEIGHTS ? e5m2_four(h[e], h[e + 1]) : e5m2_four_rounded(h[e], h[e + 1]);
                            h[e] = eight_times_rest(h[e]);
                            h[e + 1] = eight_times_rest(h[e + 1]);
                        }
                }
#pragma unroll
                for (int q = 0; q < WEIGHTS; ++q)
#pragma unroll
                    for (int i = 0; i < N; i += 16) {
                        if (i >= live) break;
                        sts128(to + ((static_cast<uint32_t>(q * N + i) / 16u ^ flip) << 4),
                               make_uint4(packed[q][i / 4], packed[q][i / 4 + 1], packed[q][i / 4 + 2], packed[q][i / 4 + 3]));
                    }
                if (first + kTile > keys) {
                    // what lies behind the sequence has weight 0, but 0 x NaN is not 0
                    const int nv = 2 * n + 1;
                    wait_warp(bar(kFull + nv % STAGES), (nv / STAGES) & 1, abort, args.limit);
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
            for (int i = 0; i < N; i += 4) {
                if (i >= live) break;
                float4 sum;
                sum.x = warp_sum(l[i]);
                sum.y = warp_sum(l[i + 1]);
                sum.z = warp_sum(l[i + 2]);
                sum.w = warp_sum(l[i + 3]);
                if (lane == 0) *reinterpret_cast<float4 *>(tops + (warp & 3) * N + i) = sum;
            }
            named_sync(1, 128);
            const bool whole = g.b0 == 0 && g.b1 == g.total, good = *abort == 0;
            float *to = piece_of(args, blockIdx.x, g.b0 == 0 ? 1 : 0);
            float o[N];
            tmem_ld_cols<N>(t_o + lanes, o);
            float step = 1.0f / 8.0f;
#pragma unroll
            for (int q = 1; q < WEIGHTS; ++q, step *= 1.0f / 8.0f) {
                float more[N];
                tmem_ld_cols<N>(t_o + q * N + lanes, more);
#pragma unroll
                for (int i = 0; i < N; ++i) o[i] = fmaf(more[i], step, o[i]);
            }
            tc_fence_before_sync();
            const auto sum_of = [&](int i) { return (tops[i] + tops[N + i]) + (tops[2 * N + i] + tops[3 * N + i]); };
            // thread r has channel r of every row, and the sums of row r
            if (good && whole) {
#pragma unroll
                for (int i = 0; i < N; i += 4) {
                    if (i >= live) break;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float sum = sum_of(i + e);
                        const int64_t at = rows[i + e].out;
                        if (at >= 0 && r < c.dim)
                            static_cast<T *>(a.out)[at * c.dim + r] = from_float<T>(sum == 0.f ? 0.f : __fdividef(o[i + e] * kSumDown, sum));
                    }
                }
                if (r < N && rows[r].out >= 0) {
                    const float sum = sum_of(r);
                    a.lse[rows[r].lse] = sum == 0.f ? -INFINITY : (rows[r].top + kSumUnit + log2f(sum)) * kLn2;
                }
            } else if (good) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    if (i >= live) break;
                    if (r < c.dim) to[2 * N + i * c.dim + r] = o[i];
                }
                if (r < N && r < live) {
                    to[r] = rows[r].top;
                    to[N + r] = sum_of(r);
                }
            }
            named_sync(1, 128);           // `tops` is free
            if (lane == 0) mbar_arrive(bar(kQFree + (segment & 1)));
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

template <typename T, int MODE>
cudaError_t launch(const CattnArgs &args, const CUtensorMap &mk, const CUtensorMap &mv, int ctas, cudaStream_t s)
{
    constexpr int PARTS = query_parts<T>();
    static std::atomic<uint64_t> done{0};
    const Kernel kernel = cached_few_kernel<T, MODE>;
    const cudaError_t e = allow_shared(reinterpret_cast<const void *>(kernel), kRoom, done);
    if (e != cudaSuccess) return e;
    return tc::launch_pdl(kernel, dim3(static_cast<unsigned>(ctas)), dim3(kThreads),
                          layout(kFewTile, PARTS, stages_of(kFewTile, PARTS)).total, s, mk, mv, args);
}

template <typename T>
cudaError_t launch_mode(const CattnArgs &a, const CUtensorMap &mk, const CUtensorMap &mv, int ctas, cudaStream_t s)
{
    const int mode = (a.p.a.cap > 0.f ? kCap : 0) | (a.p.a.slopes ? kBias : 0);
    if (mode == 0) return launch<T, 0>(a, mk, mv, ctas, s);
    if (mode == kCap) return launch<T, kCap>(a, mk, mv, ctas, s);
    if (mode == kBias) return launch<T, kBias>(a, mk, mv, ctas, s);
    return launch<T, kCap | kBias>(a, mk, mv, ctas, s);
}

}  // namespace

cudaError_t launch_cached_few(const CattnArgs &a, const CUtensorMap &mk, const CUtensorMap &mv, int ctas, cudaStream_t s)
{
    return a.p.a.format == GN_FORMAT_BF16 ? launch_mode<__nv_bfloat16>(a, mk, mv, ctas, s) : launch_mode<__half>(a, mk, mv, ctas, s);
}

}  // namespace cattn
}  // namespace gn
