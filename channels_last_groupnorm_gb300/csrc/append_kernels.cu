// append_kernels.cu -- sm_103a kernel that appends new tokens to a paged cache in
// 8 bits: the keys are turned by rotary positions on the way, keys and values
// become e4m3 with a scale for each page and head, and the query heads are turned.
//
//   a page's scale: the least power of two 2^e with 448 2^e >= the largest
//   magnitude, e >= -100 (a power of two loses nothing: e4m3's precision is
//   relative), NaN if a magnitude is not finite.  A page that is filled further has
//   scale max(old, needed); where that is larger, what it holds is rounded again.
//
// A unit is what the call adds to one page: its tokens' angles are formed once, in
// shared memory, for all heads, and teams of warps (of a few other CTAs too where there
// are few units) take heads of q, k and v by turns.  A team is one warp for a few tokens,
// up to the whole CTA for a large page: a head's tokens one after the other in one warp are a
// chain of waits (8004 tokens in pages of 128: 66 us with single warps).  A key or value
// head is gone over twice, for the largest magnitude and for the bytes; the second time
// its rows come from L1 or L2.
//
// Bound by memory: q, k and v are read once, q and a byte per channel are written.
// The angles are formed in turns with 64-bit whole numbers: position times the
// turns of a unit in units of 2^-64, whose overflow is the whole turns that do not
// matter.  (In fp64, which this GPU does at 1/64 of fp32's rate, they would take as
// long as everything else.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cstdint>

#include "block_internal.h"
#include "block_math.cuh"
#include "cache_common.cuh"
#include "gn_ptx.cuh"
#include "tc_common.cuh"

namespace gn {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kLeastExponent = -100;

// The turns of a pair at a position, in [-1/2, 1/2), in units of 2^-64.
__device__ __forceinline__ bool turns_of(const Append &p, int64_t token, uint64_t unit, int axis, int64_t &turns)
{
    const int64_t at = token * p.a.axes + axis;
    uint64_t whole;
    if (p.a.position_format == GN_POSITIONS_INT32) {
        whole = static_cast<uint64_t>(static_cast<int64_t>(static_cast<const int32_t *>(p.a.positions)[at])) * unit;
    } else if (p.a.position_format == GN_POSITIONS_INT64) {
        whole = static_cast<uint64_t>(static_cast<const int64_t *>(p.a.positions)[at]) * unit;
    } else {
        const float v = static_cast<const float *>(p.a.positions)[at];
        if (!(fabsf(v) < 9.0e18f)) return false;              // no place
        const float low = truncf(v);
        const uint64_t rest = __umul64hi(static_cast<uint64_t>(fabsf(v - low) * 4294967296.0f) << 32, unit);
        whole = static_cast<uint64_t>(static_cast<int64_t>(low)) * unit + (v < 0.f ? 0 - rest : rest);
    }
    turns = static_cast<int64_t>(whole);
    return true;
}

// Cosine and sine: of the turns' first 24 bits, which fp32 holds, and to first order of
// the rest (which would cost as much precision as everything else together).
__device__ __forceinline__ float2 angle_of(const Append &p, int64_t token, uint64_t unit, int axis)
{
    int64_t turns;
    if (!turns_of(p, token, unit, axis, turns)) return make_float2(NAN, NAN);
    const float near = static_cast<float>(static_cast<int>(turns >> 40)) * 0x1p-24f;
    const float left = static_cast<float>(static_cast<uint32_t>(turns >> 8)) * (6.2831853f * 0x1p-56f);
    float s, c;
    sincospif(2.0f * near, &s, &c);
    return make_float2(fmaf(-left, s, c), fmaf(left, c, s));
}

// The least power of two of which 448 times is at least `most`, or NaN.
__device__ __forceinline__ float scale_for(float most)
{
    if (!(most < INFINITY)) return NAN;
    const uint32_t b = __float_as_uint(most);
    // most = m 2^x: 448 = 1.75 2^8
    const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float(static_cast<uint32_t>(max(e, kLeastExponent) + 127) << 23);
}

// One unit: `count` packed tokens from `token`, at slots `slot` on of page `page`
// (-1: not stored).
struct Unit {
    int token, count, slot, page;
};

// Eight neighbouring channels of a token's head.
template <typename T>
struct Eight {
    float f[8];
    __device__ __forceinline__ void load(const T *p)
    {
        if constexpr (sizeof(T) == 4) {
            const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
            f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
        } else {
            const uint4 v = *reinterpret_cast<const uint4 *>(p);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 u = Half2<T>::unpack(w[e]);
                f[2 * e] = u.x;
                f[2 * e + 1] = u.y;
            }
        }
    }
    __device__ __forceinline__ void store(T *p) const
    {
        if constexpr (sizeof(T) == 4) {
            reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
            reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
        } else {
            *reinterpret_cast<uint4 *>(p) = make_uint4(Half2<T>::pack(f[0], f[1]), Half2<T>::pack(f[2], f[3]),
                                                       Half2<T>::pack(f[4], f[5]), Half2<T>::pack(f[6], f[7]));
        }
    }
    __device__ __forceinline__ uint2 bytes(float by) const
    {
        return make_uint2(e4m3_four(f[0] * by, f[1] * by, f[2] * by, f[3] * by),
                          e4m3_four(f[4] * by, f[5] * by, f[6] * by, f[7] * by));
    }
};

__device__ __forceinline__ void turn_pair(float &a, float &b, float2 w)
{
    const float x = fmaf(a, w.x, -(b * w.y));
    b = fmaf(a, w.y, b * w.x);
    a = x;
}

// Which 8-channel pieces (cA, cB) lane unit u of a head takes: neighbours paired,
// or nothing turned: 16 channels; halves paired: 8 of each half, then the rest.
struct Pieces {
    int a, b;
};

__device__ __forceinline__ Pieces pieces_of(int u, int pairs, bool halves)
{
    if (halves && 8 * u < pairs) return {8 * u, pairs + 8 * u};
    return {16 * u, 16 * u + 8};
}

// A token's angles in shared memory: a lane takes eight pairs, two at a time, and lanes of
// neighbouring eights lie side by side each time (pair by pair they would meet in the same banks,
// 16 at once: 8555 tokens of 24 + 24 heads took 118 us instead of 84).
struct Angles {
    int eights;                   // of pairs, the last of which may be part empty
    __host__ __device__ __forceinline__ explicit Angles(int pairs) : eights((pairs + 7) / 8) {}
    __host__ __device__ __forceinline__ int row() const { return 8 * eights; }
    __device__ __forceinline__ int at(int pair) const { return ((pair & 7) >> 1) * 2 * eights + (pair >> 3) * 2 + (pair & 1); }
    // the eight pairs of lane unit u
    __device__ __forceinline__ void get(const float2 *row, int u, float2 (&w)[8]) const
    {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float4 v = *reinterpret_cast<const float4 *>(row + j * 2 * eights + 2 * u);
            w[2 * j] = make_float2(v.x, v.y);
            w[2 * j + 1] = make_float2(v.z, v.w);
        }
    }
};

template <typename T>
__device__ __forceinline__ void turn_pieces(Eight<T> &x, Eight<T> &y, const float2 *row, int u, Pieces at, int pairs, bool halves)
{
    if (8 * u >= pairs) return;       // (with either pairing lane unit u has pairs 8 u .. 8 u + 7)
    float2 w[8];
    Angles(pairs).get(row, u, w);
    if (halves) {
#pragma unroll
        for (int e = 0; e < 8; ++e) turn_pair(x.f[e], y.f[e], w[e]);
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) turn_pair(x.f[2 * e], x.f[2 * e + 1], w[e]);
    if (at.b < 2 * pairs)
#pragma unroll
        for (int e = 0; e < 4; ++e) turn_pair(y.f[2 * e], y.f[2 * e + 1], w[4 + e]);
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// What a warp does with one head of a unit: in pieces of eight channels (VEC), or
// channel by channel where pieces are not aligned or a turn's halves are no whole pieces.
template <typename T, bool VEC>
struct Head {
    const Append &p;
    const Unit &u;
    const float2 *angle;          // [tokens][Angles::row()]
    int lane, member, team;       // this warp among those that share the head
    float (*tops)[kWarps];        // two rows of the CTA's, taken by turns
    int turn = 0;

    // fn(token of the unit, where its two pieces are, the pieces turned) for each of the
    // head's rows from `in` on, lanes side by side
    template <typename F>
    __device__ __forceinline__ void each(const T *in, int64_t stride, bool turned, F &&fn) const
    {
        const int dim = p.c.dim, pairs = turned ? p.pairs : 0;
        const bool halves = turned && p.pairs > 0 && !p.a.interleaved;
        if constexpr (VEC) {
            const int units = dim / 16, rows = 32 / units, n = lane / units, w = lane - n * units;
            const Pieces at = pieces_of(w, pairs, halves);
            if (n >= rows) return;
#pragma unroll 4
            for (int i = n + rows * member; i < u.count; i += rows * team) {
                const T *row = in + (u.token + i) * stride;
                Eight<T> x, y;
                x.load(row + at.a);
                y.load(row + at.b);
                turn_pieces(x, y, angle + i * Angles(pairs).row(), w, at, pairs, halves);
                fn(i, at, x, y);
            }
        } else {
            // single channels: pairs first, then the rest two at a time
            const int half = dim / 2;
            for (int n = lane + 32 * member; n < u.count * half; n += 32 * team) {
                const int i = n / half, k = n - i * half;
                const T *row = in + (u.token + i) * stride;
                Pieces at = {2 * k, 2 * k + 1};
                if (halves && k < pairs) at = {k, pairs + k};
                float x = to_float(row[at.a]), y = to_float(row[at.b]);
                if (k < pairs) turn_pair(x, y, angle[i * Angles(pairs).row() + Angles(pairs).at(k)]);
                fn(i, at, x, y);
            }
        }
    }

    __device__ __forceinline__ void query(const T *in, int64_t stride, T *out, int64_t out_stride) const
    {
        each(in, stride, true, [&](int i, Pieces at, const auto &x, const auto &y) {
            T *row = out + (u.token + i) * out_stride;
            if constexpr (VEC) {
                x.store(row + at.a);
                y.store(row + at.b);
            } else {
                row[at.a] = from_float<T>(x);
                row[at.b] = from_float<T>(y);
            }
        });
    }

    // The largest magnitude of the head's rows as they are, from their bits: of numbers
    // without a sign the larger has the larger bits, and NaN the largest.
    __device__ __forceinline__ float largest(const T *in, int64_t stride) const
    {
        const int units = p.c.dim / 16, rows = 32 / units, n = lane / units, w = lane - n * units;
        uint32_t most = 0;
        if (n < rows)
#pragma unroll 4
            for (int i = n + rows * member; i < u.count; i += rows * team) {
                const uint4 *at = reinterpret_cast<const uint4 *>(in + (u.token + i) * stride + 16 * w);
#pragma unroll
                for (int e = 0; e < static_cast<int>(sizeof(T)); ++e) {
                    const uint4 v = __ldg(at + e);
                    if (sizeof(T) == 2)
                        most = __vmaxu2(most, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                                       __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
                    else
                        most = max(most, max(max(v.x & 0x7fffffffu, v.y & 0x7fffffffu), max(v.z & 0x7fffffffu, v.w & 0x7fffffffu)));
                }
            }
        if constexpr (sizeof(T) == 4)
            return __uint_as_float(most);
        else
            return Half2<T>::unpack(max(most & 0xffffu, most >> 16)).x;
    }

    // The largest of the team's values (NaN if any is); what the team has read before is read.
    __device__ __forceinline__ float team_max(float v)
    {
        v = warp_max(v);
        if (team == 1) {
            __syncwarp();
            return v;
        }
        const int first = (threadIdx.x >> 5) - member;
        float *row = tops[turn];
        turn ^= 1;
        if (lane == 0) row[first + member] = v;
        named_sync(1 + first, 32 * team);
        v = row[first];
        for (int i = 1; i < team; ++i) v = max_nan(v, row[first + i]);
        return v;
    }

    __device__ __forceinline__ void keep(const T *in, int64_t stride, bool turned, uint8_t *page, int64_t page_stride,
                                         float *scale)
    {
        if (u.page < 0) return;
        float most = 0.f;
        if (VEC && !turned)
            most = largest(in, stride);
        else
            each(in, stride, turned, [&](int, Pieces, const auto &x, const auto &y) {
            if constexpr (VEC) {
#pragma unroll
                for (int e = 0; e < 8; ++e) most = max_nan3(most, x.f[e], y.f[e]);
            } else {
                most = max_nan3(most, x, y);
            }
        });
        const float old = u.slot > 0 ? *scale : 0.f;
        float now = scale_for(team_max(most));
        if (u.slot > 0) {
            now = max_nan(old, now);
            if (now > old) {
                const float by = old / now;
                for (int n = lane + 32 * member; n < u.slot * (p.c.dim / 16); n += 32 * team) {
                    const int i = n / (p.c.dim / 16), w = n - i * (p.c.dim / 16);
                    uint4 *at = reinterpret_cast<uint4 *>(page + i * page_stride + 16 * w);
                    const uint4 v = *at;
                    uint32_t b[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 lo = e4m3_values(b[e]), hi = e4m3_values(b[e] >> 16);
                        b[e] = e4m3_four(lo.x * by, lo.y * by, hi.x * by, hi.y * by);
                    }
                    *at = make_uint4(b[0], b[1], b[2], b[3]);
                }
            }
        }
        if (lane == 0 && member == 0) *scale = now;
        const bool number = now == now;
        const float by = number ? 1.0f / now : 0.f;
        each(in, stride, turned, [&](int i, Pieces at, const auto &x, const auto &y) {
            uint8_t *row = page + (u.slot + i) * page_stride;
            if constexpr (VEC) {
                const uint2 zero = make_uint2(0u, 0u);
                const uint2 a = number ? x.bytes(by) : zero, b = number ? y.bytes(by) : zero;
                if (at.b == at.a + 8) {
                    *reinterpret_cast<uint4 *>(row + at.a) = make_uint4(a.x, a.y, b.x, b.y);
                } else {
                    *reinterpret_cast<uint2 *>(row + at.a) = a;
                    *reinterpret_cast<uint2 *>(row + at.b) = b;
                }
            } else {
                const uint32_t b = number ? e4m3_pair(x * by, y * by) : 0u;
                row[at.a] = static_cast<uint8_t>(b);
                row[at.b] = static_cast<uint8_t>(b >> 8);
            }
        });
    }
};

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ Append p, int team)
{
    extern __shared__ __align__(16) float2 angle[];
    __shared__ float tops[2][kWarps];
    __shared__ uint64_t units[kRopeMaxPairs];
    __shared__ unsigned char axes[kRopeMaxPairs];
    tc::griddep_wait();
    if (threadIdx.x == 0) tc::griddep_launch_dependents();
    const gn_cache &c = p.c;
    const gn_append_args &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the unit of this block
    int n, piece;
    if (c.cu) {
        n = cache::sequence_of_piece(c, a.tokens, blockIdx.x, c.page_size, 2, lane);
        piece = static_cast<int>(blockIdx.x - cache::first_piece(c, a.tokens, n, c.page_size, 2));
    } else {
        const int each = static_cast<int>(a.tokens / c.sequences), pieces = (each + c.page_size - 2) / c.page_size + 1;
        n = blockIdx.x / pieces;
        piece = blockIdx.x - n * pieces;
    }
    const cache::Sequence s = cache::sequence_of(c, a.tokens, n);
    const int place = s.first_place(), size = c.page_size;
    const int page0 = place >= 0 ? place / size : -((size - 1 - place) / size);
    const int low = max(place, (page0 + piece) * size), high = min(s.length, (page0 + piece + 1) * size);
    if (piece < 0 || low >= high) return;
    Unit u;
    u.token = s.begin + (low - place);
    u.count = high - low;
    u.slot = low - (page0 + piece) * size;
    u.page = cache::page_of(c, n, page0 + piece);
    // (the pairs' turns by way of shared memory: parameters are read one address at a time)
    for (int k = threadIdx.x; k < p.pairs; k += kThreads) {
        units[k] = p.turns[k];
        axes[k] = p.axis[k];
    }
    __syncthreads();
#pragma unroll 2
    for (int i = threadIdx.x; i < u.count * p.pairs; i += kThreads) {
        const int t = i / p.pairs, k = i - t * p.pairs;
        angle[t * Angles(p.pairs).row() + Angles(p.pairs).at(k)] = angle_of(p, u.token + t, units[k], axes[k]);
    }
    __syncthreads();
    Head<T, VEC> head = {p, u, angle, lane, warp % team, team, tops};
    const int heads = a.heads + 2 * c.kv_heads, teams = kWarps / team;
    // keys and values first: they take longer
    for (int i = blockIdx.y * teams + warp / team; i < heads; i += gridDim.y * teams) {
        if (i < 2 * c.kv_heads) {
            const bool key = i < c.kv_heads;
            const int h = key ? i : i - c.kv_heads;
            const int64_t page = max(u.page, 0);
            if (key)
                head.keep(static_cast<const T *>(a.k) + h * a.k_head, a.k_token, true,
                          static_cast<uint8_t *>(c.k_pages) + page * c.k_page + h * c.k_head, c.k_token,
                          c.k_scales + page * c.kv_heads + h);
            else
                head.keep(static_cast<const T *>(a.v) + h * a.v_head, a.v_token, false,
                          static_cast<uint8_t *>(c.v_pages) + page * c.v_page + h * c.v_head, c.v_token,
                          c.v_scales + page * c.kv_heads + h);
        } else {
            const int h = i - 2 * c.kv_heads;
            head.query(static_cast<const T *>(a.q) + h * a.q_head, a.q_token, static_cast<T *>(a.q_out) + h * a.q_out_head,
                       a.q_out_token);
        }
    }
}

template <typename T>
cudaError_t append(const Append &p, int sm_count, cudaStream_t s)
{
    const gn_cache &c = p.c;
    const gn_append_args &a = p.a;
    constexpr int EPV = 16 / sizeof(T);
    bool vec = a.interleaved ? p.pairs % 4 == 0 : p.pairs % 8 == 0;
    const auto row_ok = [&](const void *ptr, int64_t token, int64_t head) {
        return !ptr || (reinterpret_cast<uintptr_t>(ptr) % 16 == 0 && token % EPV == 0 && head % EPV == 0);
    };
    vec = vec && row_ok(a.q, a.q_token, a.q_head) && row_ok(a.q_out, a.q_out_token, a.q_out_head) &&
          row_ok(a.k, a.k_token, a.k_head) && row_ok(a.v, a.v_token, a.v_head);
    const int64_t each = a.tokens / c.sequences;
    const int64_t units = c.cu ? a.tokens / c.page_size + 2 * (static_cast<int64_t>(c.sequences) + 2)
                               : c.sequences * ((each + c.page_size - 2) / c.page_size + 1);
    // about the units that hold tokens; enough CTAs for every SM to have a few
    const int64_t busy = c.cu ? a.tokens / c.page_size + c.sequences : units;
    const int heads = a.heads + 2 * c.kv_heads;
    const int most = static_cast<int>(std::min<int64_t>(c.page_size, c.cu ? a.tokens : each));
    // Teams: until there are some 48 warps of work for an SM, with 8 tokens a warp at least
    // (145 pages of 64 tokens, 72 heads: 83 us with single warps, 102 with four; 70 pages of 128
    // tokens, 18 heads: 56 us with single warps, 36 with eight).
    const int64_t tokens = std::min<int64_t>(most, a.tokens / c.sequences);
    int team = 1;
    while (team < kWarps && 16 * team <= tokens && busy * heads * team < 48 * sm_count) team *= 2;
    const int teams = kWarps / team;
    const int64_t split = std::max<int64_t>(1, std::min<int64_t>((heads + teams - 1) / teams, 3 * sm_count / busy));
    const size_t smem = sizeof(float2) * static_cast<size_t>(most) * static_cast<size_t>(Angles(p.pairs).row());
    const auto kernel = vec ? append_kernel<T, true> : append_kernel<T, false>;
    static std::atomic<uint64_t> done[2];
    // (pages of up to 256 tokens, 64 pairs: 128 KB)
    cudaError_t e = smem > 40 * 1024 ? allow_shared(reinterpret_cast<const void *>(kernel), 128 * 1024, done[vec]) : cudaSuccess;
    if (e != cudaSuccess) return e;
    return tc::launch_pdl(kernel, dim3(static_cast<unsigned>(units), static_cast<unsigned>(split)), dim3(kThreads), smem, s, p, team);
}

}  // namespace

cudaError_t launch_cache_append(const Append &p, int sm_count, cudaStream_t s)
{
    if (p.a.format == GN_FORMAT_BF16) return append<__nv_bfloat16>(p, sm_count, s);
    if (p.a.format == GN_FORMAT_FP16) return append<__half>(p, sm_count, s);
    return append<float>(p, sm_count, s);
}

}  // namespace gn
