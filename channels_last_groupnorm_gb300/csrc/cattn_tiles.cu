// cattn_tiles.cu -- attention over the paged cache for many rows: chunks of prompts.
//
// As the forward kernel of packed attention (pattn_forward.cu): a CTA has two halves of
// 128 rows, whose warps turn scores into weights by turns while the tensor core works
// for the other half.  Rows are a run of a sequence's new tokens times the query heads
// that share a key / value head, so that the pages are read once for all of them.  The
// cache's 8 bits make the difference:
//   S_t = Q_t K^T      the keys go into the tensor core as they are; a query is split into
//                      2 (bf16) or 3 (fp16) e4m3 numbers that add up to it, whose products go
//                      into the same accumulator.  e4m3 products take half the time of
//                      half-precision ones, so bf16 queries cost no more than before;
//   P_t = 2^(S_t c + log2 v - m)   c the key's scale, v the value's, both one number for every 8
//                      keys: v leaves the weights' sum again;
//   O_t += P_t V       in fp16: warps of their own widen the values, e4m3 is exact there.
//                      (Splitting the weights would cost the softmax warps, which
//                      bound this kernel, six operations more for every two.)
// One CTA per SM, with an equal part of all blocks (cattn_common.cuh).
// The softmax warps' instructions are what counts: pages of whole 32 tokens have a kernel of
// their own with one pair of scales for 32 keys, and the widening is spread over the SM's
// four schedulers (one warp for it all made the softmax warps beside it the last).
#include <algorithm>

#include "cattn_common.cuh"

namespace gn {
namespace cattn {
namespace {

constexpr int kThreads = 512;    // warps: 0 loads, 1 MMA, 2 the MMA's waits, 4-7 and 8-11 the halves' softmax, 12-15 widen values
constexpr int kKeyStages = 3;    // at most
constexpr int kSegments = 16;  // that are found at a time
constexpr int kScales = 4;       // blocks whose scales are in shared memory
constexpr float kLeastScale = 0x1p-100f, kLeastFactor = 0x1p-126f;
constexpr float kShift = 7.0f;   // fp16 weights, away from its subnormals (weight_shift of packed attention)
constexpr uint32_t kWide = 2 * kHalfBytes;    // a tile of values in fp16

// Registers: 512 threads are launched with 128 each; 256 x 192 + 256 x 64 is the same.
__device__ __forceinline__ void softmax_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 192;"); }
__device__ __forceinline__ void other_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 64;"); }

// The largest of three.
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// kP: per half the weights of a block's first and last 64 keys; kWideFull: the values widened
enum Bar { kQ = 0, kKFull = 2, kKEmpty = kKFull + kKeyStages, kVFull = kKEmpty + kKeyStages, kVEmpty = kVFull + 2,
           kWideFull = kVEmpty + 2, kWideEmpty = kWideFull + 2, kS = kWideEmpty + 2, kP = kS + 2, kO = kP + 4, kScale = kO + 2,
           kDrain = kScale + kScales, kBars };

struct Layout {
    uint32_t q, keys, values, wide, scales, bars, words, deal, work, total;
};

__host__ __device__ constexpr Layout layout(int parts)
{
    Layout l = {};
    l.q = 0;                                                       // [2][parts] tiles
    l.keys = 2 * static_cast<uint32_t>(parts) * kTileBytes;
    l.values = l.keys + (parts == 2 ? kKeyStages : 2) * kTileBytes;
    l.wide = l.values + 2 * kTileBytes;
    l.scales = l.wide + 2 * kWide;                                 // kScales x 16 groups of 8 keys
    l.bars = l.scales + kScales * 16 * sizeof(float4);
    l.words = l.bars + 8 * kBars;                                  // tensor-memory slot, abort
    l.deal = (l.words + 16 + 15) / 16 * 16;
    l.work = l.deal + sizeof(DealRoom);
    l.total = l.work + sizeof(WorkList<kSegments>);
    return l;
}

// One tile's values in fp16 ([2][128 tokens][64 channels], 128-byte swizzle) from their
// bytes; rows from `rows` on become zeros (0 x NaN is not 0).  Eight lanes at a time take
// four pieces of 16 channels of rows r and r ^ 5, which lie in all 32 banks, both where
// they are read and where they are written.
__device__ __forceinline__ void widen(uint32_t from, uint32_t to, int dim, int rows)
{
    // (each warp 32 rows)
    const int lane = threadIdx.x & 31, first = (threadIdx.x >> 5 & 3) * 4, q0 = lane & 3, flip = lane & 4 ? 5 : 0, base = lane >> 3;
    constexpr int kBatch = 4;       // loads that are under way together
    for (int part = 0; part * 64 < dim; ++part) {
        const int q = part * 4 + q0;
        uint4 v[kBatch];
        // rows 8 i + {0, 1, 2, 3} and, flipped, 8 i + {5, 4, 7, 6}
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int r = 8 * (first + i) + (base ^ flip);
            v[i] = lds128(from + r * 128u + ((q ^ (r & 7u)) << 4));
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int r = 8 * (first + i) + (base ^ flip);
            if (r >= rows) v[i] = make_uint4(0u, 0u, 0u, 0u);
            const uint32_t key = r & 7u, at = to + part * kHalfBytes + r * 128u;
            sts128(at + (((2u * q0) ^ key) << 4),
                   make_uint4(e4m3_half2(v[i].x), e4m3_half2(v[i].x >> 16), e4m3_half2(v[i].y), e4m3_half2(v[i].y >> 16)));
            sts128(at + (((2u * q0 + 1u) ^ key) << 4),
                   make_uint4(e4m3_half2(v[i].z), e4m3_half2(v[i].z >> 16), e4m3_half2(v[i].w), e4m3_half2(v[i].w >> 16)));
        }
    }
}

// A row's query (none: zeros) as row r of PARTS tiles; returns what its products are to be
// multiplied by.  (Loops, with the query read twice: this runs once a tile, and as straight
// code the fetching of its instructions took longer than a tile's first blocks.)
template <typename T, int PARTS>
__device__ __forceinline__ float split_query(const T *q, int dim, uint32_t tiles, int r)
{
    constexpr uint32_t kInf = IsBf16<T>::value ? 0x7f80u : 0x7c00u;
    const uint4 *from = reinterpret_cast<const uint4 *>(q);
    uint32_t most = 0;
#pragma unroll 8
    for (int i = 0; i < dim / 8; ++i) {
        const uint4 v = q ? __ldg(from + i) : make_uint4(0u, 0u, 0u, 0u);
        most = __vmaxu2(most, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
    }
    most = max(most & 0xffffu, most >> 16);
    // (infinities too: their products with keys of either sign are no numbers)
    const bool number = most < kInf;
    const int shift = number ? query_shift(Half2<T>::unpack(most).x) : 0;
    const float up = number ? power_of_two(shift) : NAN;
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
        uint32_t bytes[PARTS][4] = {};
        if (q && 16 * i < dim) {
            const uint4 a = __ldg(from + 2 * i), b = __ldg(from + 2 * i + 1);
            const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 x = Half2<T>::unpack(w[e]);
                uint32_t part[PARTS];
                split_e4m3<PARTS>(x.x * up, x.y * up, part);
#pragma unroll
                for (int p = 0; p < PARTS; ++p) bytes[p][e / 2] |= part[p] << (e % 2 * 16);
            }
        }
#pragma unroll
        for (int p = 0; p < PARTS; ++p)
            sts128(tiles + p * kTileBytes + r * 128u + ((i ^ (r & 7u)) << 4),
                   make_uint4(bytes[p][0], bytes[p][1], bytes[p][2], bytes[p][3]));
    }
    return power_of_two(-shift);
}

template <typename T, int MODE, int GROUP>
__global__ void __launch_bounds__(kThreads, 1)
    cached_tiles_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                        const __grid_constant__ CattnArgs args)
{
    constexpr int PARTS = IsBf16<T>::value ? 2 : 3, KEYS = PARTS == 2 ? kKeyStages : 2;
    constexpr Layout lay = layout(PARTS);
    extern __shared__ __align__(1024) uint8_t gbase[];
    const uint32_t base = smem_addr(gbase);
    const gn_cache &c = args.p.c;
    const gn_attn_cached_args &a = args.p.a;
    const auto bar = [&](int i) { return base + lay.bars + 8u * static_cast<uint32_t>(i); };
    volatile uint32_t *words = reinterpret_cast<volatile uint32_t *>(gbase + lay.words);
    volatile int *abort = reinterpret_cast<volatile int *>(words + 1);
    float4 *scales = reinterpret_cast<float4 *>(gbase + lay.scales);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kBars; ++i) mbar_init(bar(i), i < kQ + 2 || (i >= kP && i < kP + 4) || (i >= kWideFull && i < kWideFull + 2) || (i >= kVEmpty && i < kVEmpty + 2) ? 4 : 1);
        *abort = (*reinterpret_cast<volatile unsigned int *>(args.limit.status) != 0u) ? 1 : 0;
        mbar_init_fence();
        prefetch_tensormap(&map_k);
        prefetch_tensormap(&map_v);
    }
    if (warp == 1) {
        tmem_alloc(base + lay.words, 512);
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
    const uint32_t tmem = words[0];
    const bool skip = *abort != 0;

    Reader<kSegments> work(*reinterpret_cast<WorkList<kSegments> *>(gbase + lay.work));
    Segment g;
    const auto rows_of = [&](const Segment &s) {
        return min(args.tokens, s.s.end - s.s.begin - s.run * args.tokens) * args.heads;
    };
    if (warp >= 4 && warp < 12) {
        softmax_registers();
        // ---- softmax: one row per thread ----
        const int half = warp >= 8 ? 1 : 0, r = (warp & 3) * 32 + lane, row = half * kTile + r;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + 128 * half, to = tmem + lanes + 256 + 128 * half;
        gn_attn_packed_args bend = {};
        bend.scale = a.scale;
        bend.cap = a.cap;
        int n = 0, block = 0, mine = 0;        // blocks of this half, of the CTA, tiles of this half
        while (work.next(g)) {
            const int live = rows_of(g);
            if (half * kTile >= live) {        // (the whole half has no rows)
                block += g.b1 - g.b0;
                continue;
            }
            const int first_token = g.run * args.tokens, keys = keys_of(args, g.s, g.run);
            const auto place_of = [&](int i) { return g.s.first_place() + first_token + i / args.heads; };
            const auto end_of = [&](int place) { return a.causal ? min(max(place + 1, 0), g.s.held) : g.s.held; };
            const int place = place_of(min(row, live - 1)), end = end_of(place), all = end_of(place_of(half * kTile));
            const int head = g.hk * args.p.group + g.first_head + row % args.heads;
            const bool there = row < live && g.first_head + row % args.heads < args.p.group;
            const int64_t token = g.s.begin + first_token + row / args.heads;
            // the row's query in parts, 16 channels at a time (all are asked for at once)
            const float factor = split_query<T, PARTS>(there ? static_cast<const T *>(a.q) + token * a.q_token + head * a.q_head : nullptr,
                                                       c.dim, base + lay.q + half * PARTS * kTileBytes, r);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kQ + half));
            const float slope2 = (MODE & kBias) && a.slopes && there ? __ldg(a.slopes + head) * kLog2e : 0.f;
            const float by = MODE ? factor : factor * args.scale_log2;
            float m = -INFINITY, l = 0.f;
            for (int b = g.b0; b < g.b1; ++b, ++n, ++block) {
                const int j0 = b * kTile;
                const bool masked = j0 + kTile > all;
                wait_warp(bar(kScale + block % kScales), (block / kScales) & 1, abort, args.limit);
                const float4 *scale = scales + (block % kScales) * 16;
                wait_warp(bar(kS + half), n & 1, abort, args.limit);
                tc_fence_after_sync();
                float s[kTile];
                tmem_ld_all(ts, s);
                float bent = 1.0f;
                if (MODE) {
#pragma unroll
                    for (int q = 0; q < kTile / GROUP; ++q) {
                        const float f = by * scale[q * (GROUP / 8)].x;
                        const uint64_t f2 = pack2(f, f);
#pragma unroll
                        for (int k = GROUP * q; k < GROUP * (q + 1); k += 2) {
                            const float2 v = unpack2(mul2(pack2(s[k], s[k + 1]), f2));
                            s[k] = v.x;
                            s[k + 1] = v.y;
                        }
                    }
                    bent = bend_scores<MODE>(s, bend, args.scale_log2, slope2, place - j0);
                }
                if (masked) mask_scores(s, 0, static_cast<unsigned>(max(0, end - j0)));
                // What a group's scores are multiplied by and what is added: a group of which the row
                // sees nothing has weights of 0, whatever its scale is (it may be no number).  The factor
                // is above 0, as masked scores are -inf by now: keys of scale 0 (a page that there is not)
                // or a zero query's product with that of zero keys (2^-120 x 2^-100) would make them NaN.
                const auto factors = [&](int q, float &f, float &add, float &inv) {
                    const float4 kv = scale[q * (GROUP / 8)];
                    const bool any = j0 + GROUP * q < end;
                    f = any && !MODE ? max_nan(by * kv.x, kLeastFactor) : bent;
                    add = any ? kv.y : -INFINITY;
                    inv = any ? kv.z : 0.f;
                };
                float mx = -INFINITY;
#pragma unroll
                for (int q = 0; q < kTile / GROUP; ++q) {
                    float f, add, inv, top = s[GROUP * q], other = s[GROUP * q + 1];
                    factors(q, f, add, inv);
#pragma unroll
                    for (int k = 2; k < GROUP; k += 2) {
                        if (k % 4) top = max3(top, s[GROUP * q + k], s[GROUP * q + k + 1]);
                        else other = max3(other, s[GROUP * q + k], s[GROUP * q + k + 1]);
                    }
                    mx = fmaxf(mx, fmaf(fmaxf(top, other), f, add));
                }
                const bool grew = mx > m + (kShift + kRescaleLog2) || (b == g.b0 && mx > m);
                if (__any_sync(0xffffffffu, grew)) {
                    const float to_m = grew ? mx - kShift : m;
                    const float f = grew && m != -INFINITY ? ex2_approx(m - to_m) : 1.0f;
                    m = to_m;
                    l *= f;
                    if (b > g.b0) rescale_columns(to, f);
                }
                // the weights, 32 keys at a time; the first 64 are handed over early
                const float m_use = m == -INFINITY ? 0.f : m;
                uint64_t sum2 = 0;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 32 / GROUP; ++e) {
                        float f, add, inv;
                        factors(q * (32 / GROUP) + e, f, add, inv);
                        add -= m_use;
                        const uint64_t c2 = pack2(f, f), m2 = pack2(add, add);
                        uint64_t some = 0;
#pragma unroll
                        for (int k = 0; k < GROUP / 2; ++k) {
                            const int at = 32 * q + GROUP * e + 2 * k;
                            const float2 x = unpack2(fma2(pack2(s[at], s[at + 1]), c2, m2));
                            const float p0 = ex2_approx(x.x), p1 = ex2_approx(x.y);
                            some = k == 0 ? pack2(p0, p1) : add2(some, pack2(p0, p1));
                            pk[GROUP / 2 * e + k] = weight_pair(p0, p1);
                        }
                        sum2 = fma2(some, pack2(inv, inv), sum2);
                    }
                    tmem_st16(ts + 16 * q, pk);
                    if (q == 1) {
                        tmem_wait_st();
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(kP + 2 * half));
                    }
                }
                const float2 sums = unpack2(sum2);
                l += sums.x + sums.y;
                tmem_wait_st();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kP + 2 * half + 1));
            }
            wait_warp(bar(kO + half), mine & 1, abort, args.limit);
            ++mine;
            tc_fence_after_sync();
            const bool whole = g.b0 == 0 && g.b1 == g.total, good = *abort == 0;
            const float inv = l == 0.f ? 0.f : kSumDown / l;
            T *dst = static_cast<T *>(a.out) + (token * a.heads + head) * c.dim;
            float *piece = piece_of(args, blockIdx.x, g.b0 == 0 ? 1 : 0);
            float *dst_piece = piece + 2 * args.rows + static_cast<int64_t>(row) * c.dim;
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
                if (32 * q >= c.dim) break;
                float o[32];
                tmem_ld32(to + 32 * q, o);
                tmem_wait_ld();
                if (!there || !good) continue;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int ch = 32 * q + 8 * k;
                    if (ch >= c.dim) continue;
                    if (whole) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = l == 0.f ? 0u : Half2<T>::pack(o[8 * k + 2 * e] * inv, o[8 * k + 2 * e + 1] * inv);
                        *reinterpret_cast<uint4 *>(dst + ch) = make_uint4(w[0], w[1], w[2], w[3]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; e += 4)
                            *reinterpret_cast<float4 *>(dst_piece + ch + e) =
                                make_float4(o[8 * k + e], o[8 * k + e + 1], o[8 * k + e + 2], o[8 * k + e + 3]);
                    }
                }
            }
            if (there && good) {
                if (whole) {
                    a.lse[static_cast<int64_t>(head) * a.tokens + token] = l == 0.f ? -INFINITY : (m + kSumUnit + log2f(l)) * kLn2;
                } else {
                    piece[row] = m;
                    piece[args.rows + row] = l;
                }
            }
            tc_fence_before_sync();
        }
    } else {
        other_registers();
        if (warp == 0) {
            // ---- loads, and every 8 keys' scales by a lane of its own: asked for ahead of a
            // block's loads and stored behind them.  (Their slot was last read kScales blocks
            // ago, by a softmax whose products the values' stages have waited for.)
            const int step = args.chunk / 8;
            int block = 0, key_tiles = 0, value_tiles = 0;
            bool go = true;
            begin_work(args);
            Walk walk(args);
            walk.start(part.seq, part.offset, skip ? 0 : part.count, part.first);
            while (work.next(g, [&](WorkList<kSegments> &w) { fill_work(w, walk, part); })) {
                if (!go) continue;
                const int keys = keys_of(args, g.s, g.run);
                int key = g.b0 * kTile + lane * 8;
                bool mine = lane < 16 && key < keys;
                int page = mine ? page_for(args, g.seq, key) : 0;
                for (int b = g.b0; go && b < g.b1; ++b, ++block) {
                    const int key_now = key, page_now = page;
                    const bool now = mine, load = lane < 16 && lane % step == 0 && now;
                    float ks = 0.f, vs = 0.f;
                    if (now && page_now < c.pages) {
                        ks = __ldg(c.k_scales + static_cast<int64_t>(page_now) * c.kv_heads + g.hk);
                        vs = __ldg(c.v_scales + static_cast<int64_t>(page_now) * c.kv_heads + g.hk);
                    }
                    key += kTile;
                    mine = lane < 16 && key < keys && b + 1 < g.b1;
                    if (mine) page = page_for(args, g.seq, key);
                    go = block < KEYS || wait_warp(bar(kKEmpty + block % KEYS), (block / KEYS - 1) & 1, abort, args.limit);
                    if (!go) break;
                    load_pages(base + lay.keys + block % KEYS * kTileBytes, &map_k, args, key_now, page_now, g.hk, bar(kKFull + block % KEYS), load);
                    ++key_tiles;
                    go = block < 2 || wait_warp(bar(kVEmpty + block % 2), (block / 2 - 1) & 1, abort, args.limit);
                    if (!go) break;
                    load_pages(base + lay.values + block % 2 * kTileBytes, &map_v, args, key_now, page_now, g.hk, bar(kVFull + block % 2), load);
                    ++value_tiles;
                    vs = vs < kLeastScale ? kLeastScale : vs;
                    if (lane < 16) scales[(block % kScales) * 16 + lane] = make_float4(ks, log2f(vs), kSumDown / vs, 0.f);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kScale + block % kScales));
                }
            }
            // nothing is left in flight when the CTA ends, whatever became of the others
            for (int k = max(0, key_tiles - KEYS); k < key_tiles; ++k)
                tc::drain(bar(kKFull + k % KEYS), (k / KEYS) & 1, args.limit.timeout_ns);
            for (int k = max(0, value_tiles - 2); k < value_tiles; ++k)
                tc::drain(bar(kVFull + k % 2), (k / 2) & 1, args.limit.timeout_ns);
            __syncwarp();
        } else if (warp >= 12) {
            // ---- values to fp16 ----
            int block = 0;
            while (work.next(g)) {
                const int keys = keys_of(args, g.s, g.run);
                for (int b = g.b0; b < g.b1; ++b, ++block) {
                    wait_warp(bar(kVFull + block % 2), (block / 2) & 1, abort, args.limit);
                    if (block >= 2) wait_warp(bar(kWideEmpty + block % 2), (block / 2 - 1) & 1, abort, args.limit);
                    widen(base + lay.values + block % 2 * kTileBytes, base + lay.wide + block % 2 * kWide, c.dim, keys - b * kTile);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(bar(kWideFull + block % 2));
                        mbar_arrive(bar(kVEmpty + block % 2));
                    }
                }
            }
        } else if (warp == 3) {
            while (work.next(g)) {}
        } else {
            // ---- MMA: per block and half the weighted values of the block before, then
            // the scores of this one ----
            const bool waits = warp == 2;
            const int steps = (c.dim + 31) / 32;
            const uint32_t is = instruction_e4m3(kTile, false), io = instruction<__half>((c.dim + 15) / 16 * 16, true);
            int block = 0, tiles = 0, n[2] = {0, 0}, q_full[2] = {0, 0};
            for (; work.next(g); ++tiles) {
                const int halves = rows_of(g) > kTile ? 2 : 1, blocks = g.b1 - g.b0;
                for (int b = 0; b <= blocks; ++b) {
                    const int nv = block + b - 1, nk = block + b;
                    const uint32_t v_tile = base + lay.wide + (nv & 1) * kWide;
                    if (waits) {
                        if (b > 0) wait_warp(bar(kWideFull + (nv & 1)), (nv >> 1) & 1, abort, args.limit);
                        if (b < blocks) wait_warp(bar(kKFull + nk % KEYS), (nk / KEYS) & 1, abort, args.limit);
                    }
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (t >= halves) break;
                        if (b > 0) {
#pragma unroll
                            for (int part_of_keys = 0; part_of_keys < 2; ++part_of_keys) {
                                if (waits) wait_warp(bar(kP + 2 * t + part_of_keys), (n[t] + b - 1) & 1, abort, args.limit);
                                hand_over();
                                if (waits) continue;
                                tc_fence_after_sync();
                                mma_channels(tmem + 256 + 128 * t, tmem + 128 * t + 32 * part_of_keys, v_tile, part_of_keys, io,
                                             b > 1 || part_of_keys);
                            }
                            if (!waits && b == blocks) commit(bar(kO + t));
                        }
                        if (b < blocks) {
                            if (waits && b == 0) wait_warp(bar(kQ + t), q_full[t] & 1, abort, args.limit);
                            if (b == 0) hand_over();
                            if (waits) continue;
                            if (b == 0) tc_fence_after_sync();
                            if (elect_one()) {
#pragma unroll
                                for (int p = 0; p < PARTS; ++p) {
                                    const uint64_t dq = sw128_kmajor_desc(base + lay.q + (t * PARTS + p) * kTileBytes);
                                    const uint64_t dk = sw128_kmajor_desc(base + lay.keys + nk % KEYS * kTileBytes);
#pragma unroll
                                    for (int k = 0; k < 4; ++k) {
                                        if (k >= steps) break;
                                        umma_e4m3(tmem + 128 * t, dq + 2 * k, dk + 2 * k, is, p > 0 || k > 0);
                                    }
                                }
                            }
                            __syncwarp();
                            commit(bar(kS + t));
                        }
                    }
                    hand_over();
                    if (!waits) {
                        if (b > 0) commit(bar(kWideEmpty + (nv & 1)));
                        if (b < blocks) commit(bar(kKEmpty + nk % KEYS));
                    }
                }
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    if (t < halves) {
                        n[t] += blocks;
                        ++q_full[t];
                    }
                block += blocks;
            }
            if (!waits && block > 0) {
                commit(bar(kDrain));
                tc::drain(bar(kDrain), 0, args.limit.timeout_ns);
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

template <typename T, int MODE, int GROUP>
cudaError_t launch_group(const CattnArgs &args, const CUtensorMap &mk, const CUtensorMap &mv, int ctas, cudaStream_t s)
{
    constexpr uint32_t bytes = layout(IsBf16<T>::value ? 2 : 3).total;
    static_assert(bytes <= 227 * 1024, "a CTA's shared memory");
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_shared(reinterpret_cast<const void *>(cached_tiles_kernel<T, MODE, GROUP>), bytes, done);
    if (e != cudaSuccess) return e;
    return tc::launch_pdl(cached_tiles_kernel<T, MODE, GROUP>, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), bytes, s, mk, mv,
                          args);
}

template <typename T, int MODE>
cudaError_t launch(const CattnArgs &a, const CUtensorMap &mk, const CUtensorMap &mv, int ctas, cudaStream_t s)
{
    return a.chunk >= 32 ? launch_group<T, MODE, 32>(a, mk, mv, ctas, s) : launch_group<T, MODE, 8>(a, mk, mv, ctas, s);
}

template <typename T>
cudaError_t launch_mode(const CattnArgs &a, const CUtensorMap &mk, const CUtensorMap &mv, int ctas, cudaStream_t s)
{
    // (a scale that is not positive needs more than a factor at the end: a bias with slopes of 0)
    int mode = (a.p.a.cap > 0.f ? kCap : 0) | (a.p.a.slopes ? kBias : 0);
    if (mode == 0 && !(a.p.a.scale > 0.f)) mode = kBias;
    if (mode == 0) return launch<T, 0>(a, mk, mv, ctas, s);
    if (mode == kCap) return launch<T, kCap>(a, mk, mv, ctas, s);
    if (mode == kBias) return launch<T, kBias>(a, mk, mv, ctas, s);
    return launch<T, kCap | kBias>(a, mk, mv, ctas, s);
}

}  // namespace

cudaError_t launch_cached_tiles(const CattnArgs &a, const CUtensorMap &mk, const CUtensorMap &mv, int ctas, cudaStream_t s)
{
    return a.p.a.format == GN_FORMAT_BF16 ? launch_mode<__nv_bfloat16>(a, mk, mv, ctas, s) : launch_mode<__half>(a, mk, mv, ctas, s);
}

}  // namespace cattn
}  // namespace gn
