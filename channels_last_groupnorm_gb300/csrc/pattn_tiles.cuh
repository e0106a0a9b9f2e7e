// pattn_tiles.cuh -- what the tensor-core kernels of packed attention share:
// the shared-memory tiles and their descriptors, the MMA loops, the bounded
// waits, and the tensor maps.
//
// A tile is 128 tokens of one head: one or two halves of 64 channels, each
// [128][64] half-precision elements in rows of 128 bytes (128-byte swizzle, as
// the tensor-map loads write them; channels past the head's width and tokens
// past the end come as zeros).  The same tile serves as a K-major operand
// (channels are the contraction) and as an MN-major one (tokens are).
#pragma once

#include <cuda.h>

#include <atomic>
#include <cstdint>

#include "gn_ptx.cuh"
#include "pattn_common.cuh"
#include "tc_common.cuh"
#include "tc_ptx.cuh"

namespace gn {

namespace pattn {

constexpr int kTile = 128;
constexpr uint32_t kHalfBytes = kTile * 64 * 2;   // one half of a tile

struct TileArgs {
    PackedAttn p;
    float scale_log2;
    WaitLimit limit;
    int tiles;             // tile groups along the token axis that the CTAs own
    int parts;             // dK and dV: CTAs that share a group's query heads
};

__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int *abort, const WaitLimit &l)
{
    return tc::wait(bar, parity, abort, l.timeout_ns, l.status, l.host_status);
}

// The same for a whole warp, with one answer.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int *abort, const WaitLimit &l)
{
    return __all_sync(0xffffffffu, wait(bar, parity, abort, l));
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void *map, int c0, int c1, int c2, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}

// One tile: `halves` loads on one barrier (the caller has armed it).
__device__ __forceinline__ void load_tile(uint32_t dst, const void *map, int halves, int head, int token, uint32_t bar)
{
    for (int n = 0; n < halves; ++n) tma_load_3d(dst + n * kHalfBytes, map, n * 64, head, token, bar);
}

// Registers between a kernel's warp groups of four: the first has the loads and
// the MMA issue, the others the softmax (384 threads are launched with 168 each:
// 128 x 72 + 256 x 216 = 384 x 168).
__device__ __forceinline__ void few_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 72;"); }
__device__ __forceinline__ void many_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 216;"); }

// Matrix descriptor of a tile read MN-major (the 64 channels of a row are
// contiguous along M or N, tokens along the contraction), 128-byte swizzle:
// 16 KB from one group of 64 channels to the next (leading offset), 1 KB from 8
// tokens to the next 8 (stride offset); a contraction step of 16 tokens
// advances the start by 2 KB.
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t smem)
{
    uint64_t d = static_cast<uint64_t>((smem & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(kHalfBytes >> 4) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}

// Instruction descriptor: fp32 accumulator, M = 128, both operands of type T;
// b_mn: the shared-memory B operand is MN-major.
template <typename T> struct IsBf16 { static constexpr bool value = false; };
template <> struct IsBf16<__nv_bfloat16> { static constexpr bool value = true; };

template <typename T>
__device__ __forceinline__ uint32_t instruction(int n, bool b_mn)
{
    const uint32_t fmt = IsBf16<T>::value ? 1u : 0u;
    return (1u << 4) | (fmt << 7) | (fmt << 10) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(kTile >> 4) << 24);
}

// D[tmem] (+)= A[tmem] * B[smem]: A is 128 rows, one per lane, two elements per column.
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// The products are issued by one warp, the waits ahead of them are done by
// another: an mbarrier wait by a thread with products in flight only returns
// when they are done (2 x 4096 tokens, 19 heads, D = 128: 252 us forward with
// both in one warp, 216 us so).  Both warps run the same loop; the waiter waits, then both meet
// at a named barrier, then the issuer goes on.  A wait that runs out sets the
// abort flag, after which the waiter's waits return at once and the issuer runs
// on over whatever is there: wrong values of a call that is reported as failed,
// never a wrong address, and never a longer wait.
constexpr uint32_t kHandBarrier = 2;

__device__ __forceinline__ void hand_over() { named_sync(kHandBarrier, 64); }

// One lane of the warp, the same one every time.  The whole warp runs the loop
// and elects the issuer around each group of products: inside a branch on the
// lane number the compiler has to take the operands for divergent.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}

// Arrival on `bar` (an mbarrier) once every product issued so far is done.
__device__ __forceinline__ void commit(uint32_t bar)
{
    if (elect_one()) umma_commit(bar);
    __syncwarp();
}

// The issuing thread's own instructions would take longer than the products
// (64 cycles a step) if it built a descriptor for each: the steps only add to
// the descriptors' address field, and are unrolled.

// D = A B^T over the channels of two tiles (128 x 128, `steps` of 16 channels);
// a_half, b_half: bytes from an operand's first 64 channels to its others.
__device__ __forceinline__ void mma_tokens(uint32_t d, uint32_t a, uint32_t b, int steps, uint32_t idesc,
                                           uint32_t a_half = kHalfBytes, uint32_t b_half = kHalfBytes)
{
    const uint64_t da = sw128_kmajor_desc(a), db = sw128_kmajor_desc(b);
    if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (k >= steps) break;
            umma_f16(d, da + (k >> 2) * (a_half >> 4) + (k & 3) * 2, db + (k >> 2) * (b_half >> 4) + (k & 3) * 2, idesc,
                     k > 0);
        }
    }
    __syncwarp();
}

// D (+)= A B over 64 of a tile's tokens (half 0 or 1): A in tensor memory, 32 columns.
__device__ __forceinline__ void mma_channels(uint32_t d, uint32_t a_tmem, uint32_t b, int half, uint32_t idesc,
                                             bool accumulate)
{
    const uint64_t db = sw128_mnmajor_desc(b) + half * 4 * (2048u >> 4);
    if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 4; ++k) umma_ts(d, a_tmem + 8u * k, db + k * (2048u >> 4), idesc, accumulate || k > 0);
    }
    __syncwarp();
}

// What a kernel is built for: scores capped, biased by distance.
constexpr int kCap = 1, kBias = 2;

// ---- the cap's tanh, for N scores in place -------------------------------------------
// v <- tanh(v k).  Scores are mostly small against their cap: up to 1/2 by x + x^3
// p(x^2), two scores per instruction and no special-function unit; beyond, by 1 - 2 /
// (1 + e^2|x|) with two of its instructions each.  p is the polynomial of degree
// three whose largest relative error is least there, 2^-26 (Remez' exchange on
// tanh(x) / x in 40 digits; the coefficients' sum in fp32 is within 1.3 2^-24).
// A score's value depends on itself alone, never on its neighbours, which may be
// ones that nobody sees: the warp leaves the second formula out where no score
// wants it, and otherwise takes either for each (NaN passes through both).  Choosing
// one for the whole warp or for a thread's scores would let unseen ones have a say,
// or want them cleared first.  (4360 tokens, 16 heads on 4, D = 64, prefix mask,
// scores of deviation 2: cap 50 and 30 80 us forward, cap 2 120 us; the series of
// tanh up to 1/4 79, 158 and 120; a choice per thread 95, 136 and 113.)
template <int N>
__device__ __forceinline__ void tanh_all(float (&v)[N], float k)
{
    constexpr float kSmall = 0.5f;
    const uint64_t k2 = pack2(k, k);
    const uint64_t c0 = pack2(-0.33333144f, -0.33333144f), c1 = pack2(0.13325879f, 0.13325879f);
    const uint64_t c2 = pack2(-0.053045496f, -0.053045496f), c3 = pack2(0.017241493f, 0.017241493f);
    const auto small = [&](uint64_t x) {
        const uint64_t y = mul2(x, x), p = fma2(fma2(fma2(c3, y, c2), y, c1), y, c0);
        return unpack2(fma2(mul2(x, y), p, x));
    };
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) top = fmaxf(top, fabsf(v[i]));
    if (__all_sync(0xffffffffu, top * fabsf(k) <= kSmall)) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float2 r = small(mul2(pack2(v[i], v[i + 1]), k2));
            v[i] = r.x;
            v[i + 1] = r.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float2 x = unpack2(mul2(pack2(v[i], v[i + 1]), k2)), r = small(pack2(x.x, x.y));
            v[i] = fabsf(v[i]) * fabsf(k) <= kSmall ? r.x : tanh_fast(x.x);
            v[i + 1] = fabsf(v[i + 1]) * fabsf(k) <= kSmall ? r.y : tanh_fast(x.y);
        }
    }
}

// D (+)= A^T B over the 128 tokens of a tile A (channels are the lanes), B the
// weights of some rows, [2][rows][64 tokens], `half` bytes apart.
__device__ __forceinline__ void mma_values(uint32_t d, uint32_t a, uint32_t b, uint32_t half, uint32_t idesc, bool accumulate)
{
    const uint64_t da = sw128_mnmajor_desc(a), db = sw128_kmajor_desc(b);
    if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            umma_f16(d, da + k * (2048u >> 4), db + (k >> 2) * (half >> 4) + (k & 3) * 2, idesc, accumulate || k > 0);
    }
    __syncwarp();
}

__device__ __forceinline__ void sts_u16(uint32_t addr, uint32_t v)
{
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(static_cast<unsigned short>(v)) : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32])
{
    uint32_t u[32];
    tmem_ld_32x32b_x32(taddr, u);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(u[i]);
}

// N columns of the thread's lane, loads issued together.
template <int N>
__device__ __forceinline__ void tmem_ld_all(uint32_t taddr, float (&v)[N])
{
#pragma unroll
    for (int q = 0; q < N / 32; ++q) {
        uint32_t u[32];
        tmem_ld_32x32b_x32(taddr + 32 * q, u);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[32 * q + i] = __uint_as_float(u[i]);
    }
    tmem_wait_ld();
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *v)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
          "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// s[k] <- by s[k] - slope2 |at + DIR k| for N neighbouring tokens of the other
// side.  Where all of them lie on one side for the whole warp, the distance is
// linear in k: two operations for two scores instead of three for one.
template <int DIR, int N>
__device__ __forceinline__ void take_distance(float (&s)[N], float by, float slope2, int at)
{
    const int end = at + DIR * (N - 1);
    const bool ahead = __all_sync(0xffffffffu, min(at, end) >= 0), behind = __all_sync(0xffffffffu, max(at, end) <= 0);
    const float p = static_cast<float>(at);
    if (ahead || behind) {
        const float by_one = ahead ? -slope2 : slope2;    // per unit of at + DIR k
        const uint64_t by2 = pack2(by, by), t2 = pack2(by_one, by_one), b2 = pack2(by_one * p, by_one * p);
#pragma unroll
        for (int k = 0; k < N; k += 2) {
            const float2 v = unpack2(fma2(pack2(s[k], s[k + 1]), by2,
                                          fma2(t2, pack2(static_cast<float>(DIR * k), static_cast<float>(DIR * (k + 1))), b2)));
            s[k] = v.x;
            s[k + 1] = v.y;
        }
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k) s[k] = fmaf(-slope2, fabsf(p + static_cast<float>(DIR * k)), s[k] * by);
    }
}

// ---- scores of one query against N neighbouring keys -----------------------------------
// In place, to what times the returned factor is in units of log2 (capped and
// biased).  at: the query's position relative to the first key.  Without a cap or
// a bias (and with a positive scale: see score_mode) the raw scores only want
// their factor.
template <int MODE, int N>
__device__ __forceinline__ float bend_scores(float (&s)[N], const gn_attn_packed_args &a, float scale_log2, float slope2,
                                             int at)
{
    float by = scale_log2;
    if (MODE & kCap) {
        tanh_all(s, a.scale / a.cap);
        by = a.cap * kLog2e;
    }
    if (!(MODE & kBias)) return by;
    take_distance<-1>(s, by, slope2, at);
    return 1.0f;
}

template <int N>
__device__ __forceinline__ void mask_scores(float (&s)[N], int lo, unsigned len)
{
#pragma unroll
    for (int k = 0; k < N; ++k) s[k] = static_cast<unsigned>(k - lo) < len ? s[k] : -INFINITY;
}

template <int N>
__device__ __forceinline__ float top_score(const float (&s)[N])
{
    float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
    for (int k = 4; k < N; ++k) top[k & 3] = fmaxf(top[k & 3], s[k]);
    return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
}

// Multiplies 128 accumulator columns of the thread's lane by f.
__device__ __forceinline__ void rescale_columns(uint32_t taddr, float f)
{
#pragma unroll 1
    for (int q = 0; q < 8; ++q) {
        uint32_t u[16];
        tmem_ld16(taddr + 16 * q, u);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 16; ++k) u[k] = __float_as_uint(__uint_as_float(u[k]) * f);
        tmem_st16(taddr + 16 * q, u);
    }
}

// The running maximum only moves when a score is more than 2^8 above it; fp16
// weights are kept 2^7 higher than bf16 ones, away from fp16's subnormals (the
// largest is then 2^15, under its 65504).
constexpr float kRescaleLog2 = 8.0f;
template <typename T> constexpr float weight_shift() { return IsBf16<T>::value ? 0.f : 7.f; }

// Weights 2^(c s - m) of 32 scores: packed for the tensor core, their sums added up.
template <typename T>
__device__ __forceinline__ void weigh_32(const float *s, uint64_t c2, uint64_t m2, uint64_t (&sum2)[2], uint32_t (&pk)[16])
{
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const float2 x = unpack2(fma2(pack2(s[2 * k], s[2 * k + 1]), c2, m2));
        const float p0 = ex2_approx(x.x), p1 = ex2_approx(x.y);
        sum2[k & 1] = add2(sum2[k & 1], pack2(p0, p1));
        pk[k] = Half2<T>::pack(p0, p1);
    }
}

// The forward kernels' MODE of a call (a scale that is not positive needs more
// than a factor at the end: a bias with slopes of 0).  The modes have kernels of
// their own: the cap's tanh, never taken, cost a biased call of 16384 tokens, 8 heads,
// D = 96 29 us of 522.
inline int score_mode(const gn_attn_packed_args &a)
{
    const int mode = (a.cap > 0.f ? kCap : 0) | (a.slopes ? kBias : 0);
    return mode == 0 && !(a.scale > 0.f) ? kBias : mode;
}

// A float at the same place of the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ float peer_float(uint32_t addr, int rank)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(addr, rank)) : "memory");
    return v;
}

// Row r of a tile holds an infinity or a NaN.
template <typename T>
__device__ __forceinline__ bool row_not_finite(uint32_t tile, int r, int halves)
{
    constexpr uint32_t kExp = IsBf16<T>::value ? 0x7f80u : 0x7c00u;
    uint32_t most = 0;
    for (int h = 0; h < halves; ++h) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const uint4 v = lds128(tile + h * kHalfBytes + static_cast<uint32_t>(r) * 128u + c * 16u);
            most = __vmaxu2(most, v.x & 0x7fff7fffu);
            most = __vmaxu2(most, v.y & 0x7fff7fffu);
            most = __vmaxu2(most, v.z & 0x7fff7fffu);
            most = __vmaxu2(most, v.w & 0x7fff7fffu);
        }
    }
    return (most & 0xffffu) >= kExp || (most >> 16) >= kExp;
}

__device__ __forceinline__ void zero_row(uint32_t tile, int r, int halves)
{
    for (int h = 0; h < halves; ++h)
        for (int c = 0; c < 8; ++c)
            sts128(tile + h * kHalfBytes + static_cast<uint32_t>(r) * 128u + c * 16u, make_uint4(0u, 0u, 0u, 0u));
}

// Whether a warp finds an infinity or a NaN in one head's rows of tokens [lo, hi).
template <typename T>
static __device__ __noinline__ bool any_not_finite(const void *base, int64_t token, int64_t head, int lo, int hi, int dim)
{
    constexpr uint32_t kExp = IsBf16<T>::value ? 0x7f80u : 0x7c00u;
    const int lane = threadIdx.x & 31;
    for (int j0 = lo; j0 < hi; j0 += 32) {
        uint32_t most = 0;
        if (j0 + lane < hi) {
            const uint4 *row = reinterpret_cast<const uint4 *>(static_cast<const T *>(base) + (j0 + lane) * token + head);
            for (int c = 0; c < dim / 8; ++c) {
                const uint4 v = __ldg(row + c);
                most = __vmaxu2(most, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                               __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
            }
        }
        if (__any_sync(0xffffffffu, (most & 0xffffu) >= kExp || (most >> 16) >= kExp)) return true;
    }
    return false;
}

// A whole tile's look at its rows (one per thread) ahead of a product whose
// weights are zero for some of them: 0 x NaN is not 0.  A row with an infinity
// or a NaN is cleared; if its token lies in [lo, hi), where something in the
// CTA may see it, it is also noted in bad[0..1] (first and last such token).
// What sees one of those is computed again, one by one, at the end: of all that
// see a token between the first and the last, each looks for one that it sees
// itself (any_not_finite), since the ones around it may be others' alone.
template <typename T>
__device__ __forceinline__ void clear_not_finite(uint32_t tile, int r, int token, int lo, int hi, int halves, int *bad)
{
    if (row_not_finite<T>(tile, r, halves)) {
        zero_row(tile, r, halves);
        if (token >= lo && token < hi) {
            atomicMin(bad, token);
            atomicMax(bad + 1, token);
        }
    }
    fence_proxy_async_smem();
}

// One query's output computed by one warp (four channels per lane) without ever
// touching a key that it does not see.  (Its lse has no part in the values: the
// tile's stands.)
template <typename T>
static __device__ __noinline__ void row_forward(const gn_attn_packed_args &a, int group, int i, int h)
{
    const int lane = threadIdx.x & 31, hk = h / group;
    const Span s = query_span(a, i);
    const float slope = a.slopes ? a.slopes[h] : 0.f;
    const float4 q = load4<T>(a.q, i * a.q_token + h * a.q_head, lane, a.dim);
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = s.lo; j < s.hi; ++j) {
        const float4 k = load4<T>(a.k, j * a.k_token + hk * a.k_head, lane, a.dim);
        const float4 v = load4<T>(a.v, j * a.v_token + hk * a.v_head, lane, a.dim);
        float slack;
        const float t = score_log2(a, slope, warp_sum(dot4(q, k)), s.pos, j, slack);
        if (t > m) {
            const float f = m == -INFINITY ? 0.f : ex2_approx(m - t);
            l *= f;
            o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
            m = t;
        }
        const float w = t == -INFINITY ? 0.f : ex2_approx(t - m);
        l += w;
        axpy4(o, w, v);
        if (l != 0.f && all_nan(o, lane, a.dim)) break;
    }
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    store4<T>(a.out, (static_cast<int64_t>(i) * a.heads + h) * a.dim, lane, a.dim,
              l == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
}

// Document of `token` for a whole warp: with up to 32 documents their ends
// come in one load and are handed round, otherwise every lane searches.
__device__ __forceinline__ int doc_of_warp(const int32_t *ends, int docs, int token, int lane)
{
    if (docs > 32) return doc_of(ends, docs, token);
    const int first = __ldg(ends), end = __ldg(ends + 1 + min(lane, docs - 1));
    int d = 0;
    for (int n = 0; n < docs - 1; ++n) d += __shfl_sync(0xffffffffu, end, n) <= token;
    const int last = __shfl_sync(0xffffffffu, end, d);
    return token >= first && token < last ? d : -1;
}

__device__ __forceinline__ Span query_span_warp(const gn_attn_packed_args &a, int i, int lane)
{
    const int d = a.cu_q ? doc_of_warp(a.cu_q, a.docs, i, lane) : 0;
    if (d < 0) return Span{0, 0, 0};
    return query_span_in(a, doc_bounds(a, d), i);
}

// A barrier of `count` threads that also tells whether any of them passed true.
__device__ __forceinline__ bool bar_any(uint32_t id, uint32_t count, bool pred)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "barrier.cta.red.or.pred p, %2, %3, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(pred ? 1u : 0u), "r"(id), "r"(count)
        : "memory");
    return r != 0;
}

// Lets `kernel` run in clusters of more than eight CTAs, once per device.
inline cudaError_t allow_clusters(const void *kernel, std::atomic<uint64_t> &done)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const uint64_t bit = 1ull << (dev & 63);
    if (e != cudaSuccess || (dev < 64 && (done.load() & bit))) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e == cudaSuccess) done.fetch_or(bit);
    return e;
}

// Tensor map over [tokens][heads][dim] with boxes of 64 channels x box_heads x
// box_tokens.
inline bool encode_heads(CUtensorMap *map, const void *base, bool bf16, int64_t tokens, int64_t token_stride, int heads,
                         int64_t head_stride, int dim, int box_heads = 1, int box_tokens = kTile)
{
    const tc::EncodeTiledFn fn = tc::encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(heads),
                                static_cast<cuuint64_t>(tokens)};
    // an axis of one has no stride of its own
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(heads > 1 ? head_stride : dim) * 2,
                                   static_cast<cuuint64_t>(tokens > 1 ? token_stride : static_cast<int64_t>(heads) * dim) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_tokens)};
    const cuuint32_t step[3] = {1, 1, 1};
    return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
              const_cast<void *>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace pattn
}  // namespace gn
