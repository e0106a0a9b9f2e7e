// cattn_common.cuh -- what the kernels of attention over the paged cache share: how
// the work is dealt out, and where pieces of a tile go that several CTAs share.
//
// A tile is a run of a sequence's new tokens times some of the query heads that share
// a key / value head; its keys are cut into blocks of 128.  All (tile, block) pairs of
// a call, in the order of sequences, heads, runs and blocks, are dealt to the CTAs in
// equal consecutive parts, whatever the sequences' lengths are (only the device
// knows them); a tile counts as some blocks more than it has (`extra`), for its start
// and end, and one of no more blocks than that is not split: it belongs to the CTA whose part
// holds its first unit (two prompts of 512 tokens, 32 heads on 8: 128 tiles of up to 4 blocks,
// 38 us replayed with nearly every tile in pieces, 32 so).  A CTA's part is a list of segments, one for each tile that it meets; a
// tile that several CTAs share leaves unnormalised pieces in the workspace, which
// a second kernel joins in the order of the keys.
#pragma once

#include <cstdint>

#include "cache_common.cuh"
#include "pattn_tiles.cuh"

namespace gn {
namespace cattn {

using namespace pattn;
using cache::Sequence;

// Rows of a tile in the kernel for few of them and in the one for many.
constexpr int kFewTile = 16, kManyRows = 2 * kTile;

// Sums of weights, which are taken without the values' scales, are in units of 2^20: 2^30 keys whose
// values have the least scale (2^-100: zeros) add up to 2^(30 + 100) and more.
constexpr float kSumDown = 0x1p-20f, kSumUnit = 20.0f;

struct CattnArgs {
    CachedAttn p;
    WaitLimit limit;
    float scale_log2;
    int least, most;              // tokens of the sequences that this kernel looks after
    int tokens, heads, chunks;    // of a tile: its tokens, its query heads; chunks of heads per key / value head
    int rows;                     // room for rows in a tile's piece
    int chunk;                    // keys that one load brings: they lie in one page
    int extra;                    // blocks that a tile's start and end count as
    struct Shared *shared;        // [CTAs]
    float *pieces;                // [CTAs][2][rows][2 + dim]: maxima, sums, outputs
};

// A tile that this CTA began and others go on with: how many pieces it is in (0: there is no
// such tile; the first is this CTA's, the others those of the CTAs behind it) and where its
// results go.
struct __align__(32) Shared {
    int pieces, token, rows, head, heads;     // rows with head < heads of the tile's are real
    int pad[3];
};

// A CTA's piece: slot 0 of a tile that it did not begin, slot 1 of one that it did.
__device__ __forceinline__ float *piece_of(const CattnArgs &a, int64_t cta, int slot)
{
    return a.pieces + (cta * 2 + slot) * static_cast<int64_t>(a.rows) * (2 + a.p.c.dim);
}

// What is to be done for one tile: blocks [b0, b1) of its `total`.
struct Segment {
    int seq, hk, first_head, run;     // first_head within the group
    int b0, b1, total;
    Sequence s;
};

// The keys that the last token of a run sees, and the run's blocks (one at least:
// rows that see nothing are written too).
__host__ __device__ __forceinline__ int keys_of(const CattnArgs &a, const Sequence &s, int run)
{
    if (!a.p.a.causal) return s.held;
    return min(max(s.first_place() + min(s.end - s.begin, (run + 1) * a.tokens), 0), s.held);
}

__host__ __device__ __forceinline__ int blocks_of(const CattnArgs &a, const Sequence &s, int run)
{
    return max(1, (keys_of(a, s, run) + kTile - 1) / kTile);
}

__host__ __device__ __forceinline__ int first_sequence(const CattnArgs &a) { return a.p.c.cu ? -1 : 0; }
__host__ __device__ __forceinline__ int sequence_count(const CattnArgs &a) { return a.p.c.sequences + (a.p.c.cu ? 2 : 0); }

// (Units of work: a tile's first `extra` are its start and end, the others its blocks.)
struct Walk {
    const CattnArgs &a;
    int64_t left, per_head, at, tile_end;    // units to go; among all: the next one, and the current tile's end
    int seq, head, run, unit, runs;
    Sequence s;

    __host__ __device__ __forceinline__ explicit Walk(const CattnArgs &args) : a(args) {}

    __host__ __device__ __forceinline__ void load(int n)
    {
        seq = n;
        s = cache::sequence_of(a.p.c, a.p.a.tokens, n);
        const int count = s.end - s.begin;
        runs = count < a.least || count > a.most ? 0 : (count + a.tokens - 1) / a.tokens;
        per_head = 0;
#pragma unroll 1
        for (int r = 0; r < runs; ++r) per_head += a.extra + blocks_of(a, s, r);
    }
    __host__ __device__ __forceinline__ int heads() const { return a.p.c.kv_heads * a.chunks; }
    __host__ __device__ __forceinline__ int64_t units() const { return per_head * heads(); }

    // begins `offset` units into sequence n
    __host__ __device__ __forceinline__ void start(int n, int64_t offset, int64_t count, int64_t first)
    {
        left = count;
        at = first;
        if (count <= 0) return;
        load(n);
#pragma unroll 1
        for (head = 0; offset >= per_head; ++head) offset -= per_head;
#pragma unroll 1
        for (run = 0; run < runs - 1; ++run) {
            const int b = a.extra + blocks_of(a, s, run);
            if (offset < b) break;
            offset -= b;
        }
        unit = static_cast<int>(offset);
        const int total = blocks_of(a, s, run);
        if (unit > 0 && total <= a.extra) spend(a.extra + total - unit);      // another CTA's
    }
    // `count` units are done with, which end the tile or the part
    __host__ __device__ __forceinline__ void spend(int count)
    {
        at += count;
        left -= count;
        unit = 0;
        if (left > 0 && ++run == runs) {
            run = 0;
            if (++head == heads()) {
                head = 0;
                const int last = first_sequence(a) + sequence_count(a);
                int n = seq + 1;
#pragma unroll 1
                for (load(n); runs == 0 && n + 1 < last; load(n)) ++n;
                if (runs == 0) left = 0;
            }
        }
    }
    // the next tile of which the part has blocks
    __host__ __device__ __forceinline__ bool next(Segment &g)
    {
#pragma unroll 1
        while (left > 0) {
            g.seq = seq;
            g.s = s;
            g.hk = head / a.chunks;
            g.first_head = (head - g.hk * a.chunks) * a.heads;
            g.run = run;
            g.total = blocks_of(a, s, run);
            const int all = a.extra + g.total;
            const int take = g.total <= a.extra || left > all - unit ? all - unit : static_cast<int>(left);
            g.b0 = max(unit - a.extra, 0);
            g.b1 = max(unit + take - a.extra, 0);
            tile_end = at + all - unit;
            spend(take);
            if (g.b0 < g.b1) return true;
        }
        return false;
    }
};

// This CTA's part of the work: `count` units from unit `first` of `all`, which lies
// `offset` into sequence `seq`.
struct Part {
    int64_t offset, count, first, all;
    int seq, ctas;                // the CTAs that have work
};

// Where part n of `all` units begins.  (By a fraction of 32 bits: it only has to grow with n
// and be the same wherever it is asked for, and a division of 64 bits is a long stretch of
// instructions.  The fraction is a little high, so that whole parts come out whole.)
__host__ __device__ __forceinline__ int64_t part_begin(int64_t all, int ctas, int n)
{
    if (n >= ctas) return all;
#ifdef __CUDA_ARCH__
    const float share = static_cast<float>(n) * __frcp_rn(static_cast<float>(ctas));
#else
    const float share = static_cast<float>(n) * (1.0f / static_cast<float>(ctas));
#endif
    const uint64_t fraction = static_cast<uint64_t>(share * 4294967296.0f) + (n > 0 ? 1024u : 0u);
#ifdef __CUDA_ARCH__
    return static_cast<int64_t>(__umul64hi(static_cast<uint64_t>(all), fraction << 32));
#else
    return static_cast<int64_t>(static_cast<unsigned __int128>(all) * fraction >> 32);
#endif
}

// The part that holds a unit.
__host__ __device__ __forceinline__ int part_of(int64_t all, int ctas, int64_t unit)
{
    int n = static_cast<int>(static_cast<float>(unit) / static_cast<float>(all) * static_cast<float>(ctas));
    n = min(max(n, 0), ctas - 1);
#pragma unroll 1
    while (n > 0 && part_begin(all, ctas, n) > unit) --n;
#pragma unroll 1
    while (n + 1 < ctas && part_begin(all, ctas, n + 1) <= unit) ++n;
    return n;
}

struct DealRoom {
    int64_t sums[32];
    Part part;
};

// For the whole CTA (whole warps).
__device__ __forceinline__ Part deal(const CattnArgs &a, DealRoom &room, int ctas)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int count = sequence_count(a), each = (count + blockDim.x - 1) / blockDim.x;
    const int n0 = first_sequence(a) + threadIdx.x * each, n1 = min(n0 + each, first_sequence(a) + count);
    Walk w(a);
    int64_t own = 0;
#pragma unroll 1
    for (int n = n0; n < n1; ++n) {
        w.load(n);
        own += w.units();
    }
    int64_t before = own;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int64_t v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
    }
    if (lane == 31) room.sums[warp] = before;
    if (threadIdx.x == 0) room.part.count = 0;
    __syncthreads();
    int64_t all = 0;
    before -= own;
#pragma unroll 1
    for (int i = 0; i < warps; ++i) {
        if (i < warp) before += room.sums[i];
        all += room.sums[i];
    }
    const int busy = static_cast<int>(all < ctas ? (all > 0 ? all : 1) : ctas);
    if (static_cast<int>(blockIdx.x) < busy && all > 0) {
        const int64_t u0 = part_begin(all, busy, blockIdx.x), u1 = part_begin(all, busy, blockIdx.x + 1);
        if (u0 < u1 && u0 >= before && u0 < before + own) {
            int n = n0;
#pragma unroll 1
            for (w.load(n); before + w.units() <= u0 && n + 1 < n1; w.load(n)) {
                before += w.units();
                ++n;
            }
            room.part = {u0 - before, u1 - u0, u0, all, n, busy};
        }
    }
    __syncthreads();
    return room.part;
}

// A CTA's segments, found by one thread and read by all roles, K at a time.  (Each role
// walking by itself would be five copies of the walk, which pushed what the roles loop over
// out of the instruction cache.)
template <int K>
struct WorkList {
    Segment list[K];
    int count, more;
};

// Every role of the CTA calls next() until it says no, whatever becomes of the others: the
// list is refilled between two barriers of all threads.  fill(list) is the loader's.
template <int K>
struct Reader {
    WorkList<K> &work;
    int at = 0, count = 0, more = 1;

    __device__ __forceinline__ explicit Reader(WorkList<K> &w) : work(w) {}

    template <typename F>
    __device__ __forceinline__ bool next(Segment &g, F &&fill)
    {
        if (at == count) {
            if (!more) return false;
            named_sync(0, blockDim.x);
            fill(work);
            named_sync(0, blockDim.x);
            count = work.count;
            more = work.more;
            at = 0;
            if (count == 0) return false;
        }
        g = work.list[at++];
        return true;
    }
    __device__ __forceinline__ bool next(Segment &g)
    {
        return next(g, [](WorkList<K> &) {});
    }
};

// Of CTA `cta`, which also says in `shared` which tile of its own is to be joined (one at the
// most, its last; the list that it is in need not be the last one that is asked for, so
// `shared` says none ahead of the first list, and is only written where there is one).
template <int K>
__host__ __device__ __forceinline__ void list_work(WorkList<K> &w, Walk &walk, const Part &part, int cta, Shared &shared)
{
    const CattnArgs &a = walk.a;
    int n = 0;
#pragma unroll 1
    for (; n < K && walk.next(w.list[n]); ++n) {
        const Segment &g = w.list[n];
        if (g.b0 != 0 || g.b1 == g.total) continue;
        const int first_token = g.run * a.tokens;
        Shared s = {};
        s.pieces = part_of(part.all, part.ctas, walk.tile_end - 1) + 1 - cta;
        s.token = g.s.begin + first_token;
        s.rows = min(a.tokens, g.s.end - g.s.begin - first_token) * a.heads;
        s.head = g.hk * a.p.group + g.first_head;
        s.heads = a.p.group - g.first_head;
        shared = s;
    }
    w.count = n;
    w.more = n == K && walk.left > 0;
}

// (the loader's)
__device__ __forceinline__ void begin_work(const CattnArgs &a)
{
    if ((threadIdx.x & 31) == 0) a.shared[blockIdx.x] = {};
}

template <int K>
__device__ __forceinline__ void fill_work(WorkList<K> &w, Walk &walk, const Part &part)
{
    if ((threadIdx.x & 31) == 0) list_work(w, walk, part, static_cast<int>(blockIdx.x), walk.a.shared[blockIdx.x]);
    __syncwarp();
}

cudaError_t launch_cached_few(const CattnArgs &a, const CUtensorMap &mk, const CUtensorMap &mv, int ctas, cudaStream_t s);
cudaError_t launch_cached_tiles(const CattnArgs &a, const CUtensorMap &mk, const CUtensorMap &mv, int ctas, cudaStream_t s);

// Two weights in fp16, past 65504 as that (NaN: NaN).  A weight is bounded by how far its score may
// be above the row's maximum, but scores of 2^26 and more (a bias far from its query) have steps of
// 8 and more: infinities there, times values of either sign and times 0 in the join, would be NaN.
__device__ __forceinline__ uint32_t weight_pair(float a, float b)
{
    uint32_t r;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// ---- operands in 8 bits ------------------------------------------------------------
// Instruction descriptor: fp32 accumulator, M = 128, e4m3 operands, both K-major but
// for a_mn: the A operand is MN-major.
__device__ __forceinline__ uint32_t instruction_e4m3(int n, bool a_mn)
{
    return (1u << 4) | (a_mn ? 1u << 15 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(kTile >> 4) << 24);
}

__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// A tile of 128 tokens in 8 bits: rows of 128 bytes (channels past the head's width
// come as zeros), 128-byte swizzle.
constexpr uint32_t kTileBytes = kTile * 128;

// One tile's loads by a warp: a lane with `go` brings `chunk` keys from `key` on, which lie
// in `page` (its own), on one barrier.
__device__ __forceinline__ void load_pages(uint32_t dst, const void *map, const CattnArgs &a, int key, int page, int hk, uint32_t bar, bool go)
{
    const unsigned loads = __ballot_sync(0xffffffffu, go);
    if ((threadIdx.x & 31) == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(__popc(loads)) * static_cast<uint32_t>(a.chunk) * 128u);
    __syncwarp();
    if (go) tma_load_4d(dst + static_cast<uint32_t>(key % kTile) * 128u, map, 0, key % a.p.c.page_size, hk, page, bar);
    __syncwarp();
}

// The page for lane n's chunk of a block (pages past the pool: zeros), if the chunk has a key.
__device__ __forceinline__ int page_for(const CattnArgs &a, int seq, int key)
{
    const int page = cache::page_of(a.p.c, seq, key / a.p.c.page_size);
    return page < 0 ? static_cast<int>(a.p.c.pages) : page;
}

__device__ __forceinline__ void zero_tile_row(uint32_t tile, int r)
{
#pragma unroll
    for (int c = 0; c < 8; ++c) sts128(tile + static_cast<uint32_t>(r) * 128u + c * 16u, make_uint4(0u, 0u, 0u, 0u));
}

// Two channels of a query, scaled to 2^7 .. 2^8 for its largest, as PARTS pairs of e4m3
// numbers that add up to them (by way of fp16, which holds either half format's bits).
template <int PARTS>
__device__ __forceinline__ void split_e4m3(float a, float b, uint32_t (&w)[PARTS])
{
    uint32_t h = Half2<__half>::pack(a, b);
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
        w[p] = e4m3_pair_half(h);
        if (p + 1 < PARTS) {
            const uint32_t near = e4m3_half2(w[p]);
            const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&h), *reinterpret_cast<const __half2 *>(&near));
            h = *reinterpret_cast<const uint32_t *>(&d);
        }
    }
}

// The power of two that takes `most` to [2^7, 2^8) (within 2^120).
__device__ __forceinline__ int query_shift(float most)
{
    const int e = static_cast<int>(__float_as_uint(most) >> 23) - 127;
    return min(7 - e, 120);
}

__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

}  // namespace cattn
}  // namespace gn
