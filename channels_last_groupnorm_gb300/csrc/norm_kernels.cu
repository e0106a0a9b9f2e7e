// norm_kernels.cu -- sm_103a kernels of layer norm over the last axis and its
// backward pass.
//
//   forward   mean = sum(x) / C, rstd = 1 / sqrt(sum((x - mean)^2) / C + eps),
//             y = (x - mean) rstd w + b
//   backward  with h = (x - mean) rstd and g = dy w,
//             dx = rstd (g - sum(g) / C - h sum(g h) / C),
//             dw = sum over rows of dy h,  db = sum over rows of dy
//
// Both are bound by memory (forward x in, y out; backward x, dy in, dx out).
// A row is held in the registers of `tpr` threads (NV slots each of EPV
// consecutive elements), so that x (and dy) are read once, the variance is
// the second pass over registers about the exact mean, and nothing is
// recomputed.  A thread keeps its columns for every row that it meets: in the
// backward pass it adds up its part of dw and db in registers.  All sums are
// fp32; y and dx are rounded once to the type of x, dw and db once to the type
// of the weight.
//
// Two ways to the rows:
//  * streamed: one CTA per SM, rows brought by bulk copies into a ring of
//    shared memory that a warp of its own keeps full, so that up to 200 KB per
//    SM are in flight whatever the arithmetic does.  When every CTA meets several
//    batches of rows.  Rows that begin at any element come as the 16-byte blocks
//    that hold them and are shifted into place on their way to the registers.
//  * direct: plain loads, many CTAs.  For few rows, where the ring would not
//    fill, and for rows too long for the ring.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "block_internal.h"
#include "block_math.cuh"
#include "gn_ptx.cuh"
#include "tc_common.cuh"

namespace gn {
namespace {

// A word of two half-precision values (fp32 rows have no use for it).
template <typename T> __device__ __forceinline__ float2 unpack_word(uint32_t v) { return Half2<T>::unpack(v); }
template <> __device__ __forceinline__ float2 unpack_word<float>(uint32_t) { return make_float2(0.f, 0.f); }
template <typename T> __device__ __forceinline__ uint32_t pack_word(float a, float b) { return Half2<T>::pack(a, b); }
template <> __device__ __forceinline__ uint32_t pack_word<float>(float, float) { return 0u; }

template <typename T, int N>
__device__ __forceinline__ void load_as(const T *p, float (&f)[N])
{
    // (a parameter vector has only its element's alignment)
#pragma unroll
    for (int e = 0; e < N; ++e) f[e] = to_float(p[e]);
}

// N consecutive elements of the weight or the bias, in its own format.
template <int N>
__device__ __forceinline__ void load_params(const void *p, int format, int c, float (&f)[N])
{
    if (format == GN_FORMAT_FP32) {
        const float *q = static_cast<const float *>(p) + c;
        if (N % 4 == 0 && reinterpret_cast<uintptr_t>(q) % 16 == 0) {
#pragma unroll
            for (int e = 0; e < N / 4; ++e) {
                const float4 v = reinterpret_cast<const float4 *>(q)[e];
                f[4 * e] = v.x;
                f[(4 * e + 1) % N] = v.y;
                f[(4 * e + 2) % N] = v.z;
                f[(4 * e + 3) % N] = v.w;
            }
        } else {
            load_as(q, f);
        }
    } else if (format == GN_FORMAT_BF16) {
        load_as(static_cast<const __nv_bfloat16 *>(p) + c, f);
    } else {
        load_as(static_cast<const __half *>(p) + c, f);
    }
}

__device__ __forceinline__ void store_param(void *p, int format, int c, float v)
{
    if (format == GN_FORMAT_FP32)
        static_cast<float *>(p)[c] = v;
    else if (format == GN_FORMAT_BF16)
        static_cast<__nv_bfloat16 *>(p)[c] = __float2bfloat16_rn(v);
    else
        static_cast<__half *>(p)[c] = __float2half_rn(v);
}

// Element offset of row n (rows are counted in 32 bits where they are in two levels).
__device__ __forceinline__ int64_t row_offset(const RowsAt &at, int64_t inner, int64_t rows, int64_t n)
{
    if (inner >= rows) return n * at.stride;
    const uint32_t a = static_cast<uint32_t>(n) / static_cast<uint32_t>(inner);
    return a * at.outer + (n - a * inner) * at.stride;
}

// The threads of one row: tpr of them (a power of two up to 32, or whole
// warps), group g of the CTA's.
struct Group {
    int tpr, g, lane;                // lane: this thread's place in its group
    float (*scratch)[32][2];         // two buffers of the group, taken in turn
    int turn;
};

// Sums of N values over a group.  Within a warp by shuffles; over several
// warps through the group's scratch, whose two buffers make one barrier per
// reduction enough.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], Group &gr)
{
    if (gr.tpr < 32) {
        for (int o = gr.tpr >> 1; o > 0; o >>= 1)
#pragma unroll
            for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
        return;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
    if (gr.tpr == 32) return;
    const int warp = gr.lane >> 5, lane = threadIdx.x & 31, warps = gr.tpr >> 5;
    float(*s)[2] = gr.scratch[gr.turn];
    gr.turn ^= 1;
    if (lane == 0)
#pragma unroll
        for (int n = 0; n < N; ++n) s[warp][n] = v[n];
    named_sync(1 + gr.g, gr.tpr);
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = lane < warps ? s[lane][n] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
}

struct Shifted {};

// A thread's elements of a row, NV slots of EPV: slot k begins at element (lane +
// k tpr) EPV; zeros past the end.  They stay in the row's own type (half the
// registers, converted twice) and are handed out two at a time.
template <typename T, int EPV, int NV>
struct Row {
    static constexpr int kPairs = NV * EPV / 2;
    static constexpr int kWords = EPV == 1 ? 1 : 4;
    uint32_t raw[NV][kWords];

    __device__ __forceinline__ Row(const T *row, const Group &gr, int cols)
    {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (gr.lane + k * gr.tpr) * EPV;
            if (EPV == 1) {
                raw[k][0] = __float_as_uint(c < cols ? to_float(row[c]) : 0.f);
            } else {
                const uint4 v = c < cols ? *reinterpret_cast<const uint4 *>(row + c) : make_uint4(0u, 0u, 0u, 0u);
                raw[k][0] = v.x;
                raw[k][1 % kWords] = v.y;
                raw[k][2 % kWords] = v.z;
                raw[k][3 % kWords] = v.w;
            }
        }
    }
    // From shared memory where the row begins at any element: a slot's 16 bytes
    // come out of the two aligned blocks that hold them.  (16 bytes past the row's
    // last block are read and dropped; what lies past its end is zero.)
    __device__ __forceinline__ Row(const uint8_t *row, const Group &gr, int cols, Shifted)
    {
        const uint32_t at = smem_addr(row) & 15u;
        const uint8_t *base = row - at;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (gr.lane + k * gr.tpr) * EPV;
            uint32_t w[8] = {};
            if (c < cols) {
                const uint4 a = *reinterpret_cast<const uint4 *>(base + c * sizeof(T));
                const uint4 b = *reinterpret_cast<const uint4 *>(base + c * sizeof(T) + 16);
                w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
            }
#pragma unroll
            for (int i = 0; i < 6; ++i) w[i] = at & 8u ? w[i + 2] : w[i];
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = at & 4u ? w[i + 1] : w[i];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (sizeof(T) == 2 && (at & 2u)) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
                const int left = (cols - c) * static_cast<int>(sizeof(T)) - 4 * i;    // bytes of the row from this word on
                raw[k][i % kWords] = left >= 4 ? w[i] : left == 2 ? w[i] & 0xffffu : 0u;
            }
        }
    }
    // elements 2 j and 2 j + 1
    __device__ __forceinline__ uint64_t pair(int j) const
    {
        if (EPV == 1) return pack2(__uint_as_float(raw[2 * j][0]), __uint_as_float(raw[2 * j + 1][0]));
        if (sizeof(T) == 4)
            return pack2(__uint_as_float(raw[j / 2][(j % 2) * 2 % kWords]), __uint_as_float(raw[j / 2][((j % 2) * 2 + 1) % kWords]));
        const float2 v = unpack_word<T>(raw[j / 4 % NV][j % 4 % kWords]);
        return pack2(v.x, v.y);
    }
};

// The thread's part of the weight (ones without) or the bias (zeros), in pairs:
// held in registers, or asked for at every row (where the registers are full).
template <int EPV, int NV, bool kHeld = (NV * EPV <= 16), bool kTail = false>
struct Own {
    const void *p;
    int format, cols;
    float fill;
    uint64_t v[kHeld ? NV * EPV / 2 : 1];

    __device__ __forceinline__ void fetch(const Group &gr, int k, float (&f)[EPV]) const
    {
        const int c = (gr.lane + k * gr.tpr) * EPV;
        if (p && (kTail ? c + EPV : c + 1) <= cols) {
            load_params<EPV>(p, format, c, f);
        } else if (kTail && p && c < cols) {
#pragma unroll
            for (int e = 0; e < EPV; ++e) {
                float one[1] = {fill};
                if (c + e < cols) load_params<1>(p, format, c + e, one);
                f[e] = one[0];
            }
        } else {
#pragma unroll
            for (int e = 0; e < EPV; ++e) f[e] = fill;
        }
    }
    // the pairs of slot k (EPV > 1) or of slots k and k + 1
    __device__ __forceinline__ void fetch_pairs(const Group &gr, int k, uint64_t (&f)[EPV == 1 ? 1 : EPV / 2]) const
    {
        float one[EPV], two[EPV];
        fetch(gr, k, one);
        if (EPV == 1) {
            fetch(gr, k + 1, two);
            f[0] = pack2(one[0], two[0]);
        } else {
#pragma unroll
            for (int e = 0; e < EPV / 2; ++e) f[e % (EPV == 1 ? 1 : EPV / 2)] = pack2(one[2 * e % EPV], one[(2 * e + 1) % EPV]);
        }
    }
    __device__ __forceinline__ Own(const void *ptr, int fmt, const Group &gr, int n, float other)
        : p(ptr), format(fmt), cols(n), fill(other)
    {
        if (!kHeld) return;
        constexpr int kStep = EPV == 1 ? 2 : 1, kEach = EPV == 1 ? 1 : EPV / 2;
#pragma unroll
        for (int k = 0; k < NV; k += kStep) {
            uint64_t f[kEach];
            fetch_pairs(gr, k, f);
#pragma unroll
            for (int e = 0; e < kEach; ++e) v[kHeld ? k / kStep * kEach + e : 0] = f[e];
        }
    }
    // the pairs of group k of slots (one slot, or two of one element)
    __device__ __forceinline__ void get(const Group &gr, int k, uint64_t (&f)[EPV == 1 ? 1 : EPV / 2]) const
    {
        constexpr int kEach = EPV == 1 ? 1 : EPV / 2;
        if (kHeld) {
#pragma unroll
            for (int e = 0; e < kEach; ++e) f[e] = v[kHeld ? k * kEach + e : 0];
        } else {
            fetch_pairs(gr, EPV == 1 ? 2 * k : k, f);
        }
    }
};

// Writes the pairs of group k of slots, rounded once.
template <typename T, int EPV>
__device__ __forceinline__ void store_pairs(T *row, const Group &gr, int k, int cols, const uint64_t (&f)[EPV == 1 ? 1 : EPV / 2])
{
    if (EPV == 1) {
        const float2 v = unpack2(f[0]);
        const int c = gr.lane + 2 * k * gr.tpr;
        if (c < cols) row[c] = from_float<T>(v.x);
        if (c + gr.tpr < cols) row[c + gr.tpr] = from_float<T>(v.y);
        return;
    }
    const int c = (gr.lane + k * gr.tpr) * EPV;
    if (c >= cols) return;
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (sizeof(T) == 4) {
            const float2 v = unpack2(f[e / 2 % (EPV == 1 ? 1 : EPV / 2)]);
            w[e] = __float_as_uint(e % 2 ? v.y : v.x);
        } else {
            const float2 v = unpack2(f[e % (EPV == 1 ? 1 : EPV / 2)]);
            w[e] = pack_word<T>(v.x, v.y);
        }
    }
    *reinterpret_cast<uint4 *>(row + c) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Where a row's results go: straight to memory,
template <typename T, int EPV>
struct Straight {
    static constexpr bool kTail = false;
    __device__ __forceinline__ void put(T *row, const Group &gr, int k, int cols, const uint64_t (&f)[EPV == 1 ? 1 : EPV / 2])
    {
        store_pairs<T, EPV>(row, gr, k, cols, f);
    }
    __device__ __forceinline__ void done(T *, const Group &, int, bool) {}
};

// or, for a row that begins at any element, through a copy in shared memory that
// lies to 16 bytes as the row does: whole blocks of it leave as vectors, and the
// blocks that it shares with its neighbours element by element.
template <typename T, int EPV>
struct Staged {
    static constexpr bool kTail = true;   // (a slot may reach over the row's end)
    uint8_t *buffer;                      // the group's
    __device__ __forceinline__ void put(T *row, const Group &gr, int k, int cols, const uint64_t (&f)[EPV == 1 ? 1 : EPV / 2])
    {
        const int c = (gr.lane + k * gr.tpr) * EPV;
        if (c >= cols) return;
        uint8_t *to = buffer + (reinterpret_cast<uintptr_t>(row) & 15u) + c * sizeof(T);
        if (c + EPV > cols) {
            T *one = reinterpret_cast<T *>(to);
#pragma unroll
            for (int e = 0; e < EPV; ++e)
                if (c + e < cols) {
                    const float2 v = unpack2(f[e / 2]);
                    one[e] = from_float<T>(e % 2 ? v.y : v.x);
                }
            return;
        }
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 v = unpack2(f[sizeof(T) == 4 ? e / 2 : e % (EPV / 2)]);
            w[e] = sizeof(T) == 4 ? __float_as_uint(e % 2 ? v.y : v.x) : pack_word<T>(v.x, v.y);
        }
        if (sizeof(T) == 2 && (reinterpret_cast<uintptr_t>(row) & 2u)) {
            *reinterpret_cast<uint16_t *>(to) = static_cast<uint16_t>(w[0]);
#pragma unroll
            for (int e = 0; e < 3; ++e) *reinterpret_cast<uint32_t *>(to + 2 + 4 * e) = __funnelshift_r(w[e], w[e + 1], 16);
            *reinterpret_cast<uint16_t *>(to + 14) = static_cast<uint16_t>(w[3] >> 16);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) *reinterpret_cast<uint32_t *>(to + 4 * e) = w[e];
        }
    }
    // (all threads of the group; the next row's sums come before its next put)
    __device__ __forceinline__ void done(T *row, const Group &gr, int cols, bool live)
    {
        if (gr.tpr > 32)
            named_sync(1 + gr.g, gr.tpr);
        else
            __syncwarp();
        if (live) {
            const int at = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15u), end = at + cols * static_cast<int>(sizeof(T));
            uint8_t *base = reinterpret_cast<uint8_t *>(row) - at;
            const int first = at ? 1 : 0, last = end / 16;
            for (int i = first + gr.lane; i < last; i += gr.tpr)
                reinterpret_cast<uint4 *>(base)[i] = reinterpret_cast<const uint4 *>(buffer)[i];
            const int head = min(16 * first, end), tail = max(16 * last, head);
            for (int i = at + gr.lane * static_cast<int>(sizeof(T)); i < head; i += gr.tpr * static_cast<int>(sizeof(T)))
                *reinterpret_cast<T *>(base + i) = *reinterpret_cast<const T *>(buffer + i);
            for (int i = tail + gr.lane * static_cast<int>(sizeof(T)); i < end; i += gr.tpr * static_cast<int>(sizeof(T)))
                *reinterpret_cast<T *>(base + i) = *reinterpret_cast<const T *>(buffer + i);
        }
        if (gr.tpr <= 32) __syncwarp();
    }
};

// One row from registers: statistics out, y out.
template <typename T, int EPV, int NV, typename Params, typename Out>
__device__ __forceinline__ void norm_row(const NormArgs &a, const Row<T, EPV, NV> &x, const Params &w, const Params &b,
                                         Group &gr, int64_t row, bool live, Out out)
{
    constexpr int kEach = EPV == 1 ? 1 : EPV / 2, kGroups = Row<T, EPV, NV>::kPairs / kEach;
    const float inv = 1.0f / static_cast<float>(a.cols);
    uint64_t s2 = 0;
#pragma unroll
    for (int j = 0; j < Row<T, EPV, NV>::kPairs; ++j) s2 = add2(s2, x.pair(j));
    float s[1] = {unpack2(s2).x + unpack2(s2).y};
    row_sum(s, gr);
    const float mean = s[0] * inv;
    const uint64_t minus = pack2(-mean, -mean);
    uint64_t q2 = 0;
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
        // what lies past the row's end adds nothing
        const int c = EPV == 1 ? gr.lane + 2 * k * gr.tpr : (gr.lane + k * gr.tpr) * EPV;
        if (c >= a.cols) break;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            uint64_t d = add2(x.pair(k * kEach + e), minus);
            if (EPV == 1 && c + gr.tpr >= a.cols) d = pack2(unpack2(d).x, 0.f);
            if (Out::kTail && c + EPV > a.cols)
                d = pack2(c + 2 * e < a.cols ? unpack2(d).x : 0.f, c + 2 * e + 1 < a.cols ? unpack2(d).y : 0.f);
            q2 = fma2(d, d, q2);
        }
    }
    float q[1] = {unpack2(q2).x + unpack2(q2).y};
    row_sum(q, gr);
    const float rstd = rsqrtf(fmaf(q[0], inv, a.eps));   // (two steps of fp32 at most)
    T *y = static_cast<T *>(a.y) + (live ? row_offset(a.y_at, a.inner, a.rows, row) : 0);
    if (live) {
        if (gr.lane == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
        const uint64_t r2 = pack2(rstd, rstd);
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
            uint64_t f[kEach], bk[kEach];
            w.get(gr, k, f);
            b.get(gr, k, bk);
#pragma unroll
            for (int e = 0; e < kEach; ++e) f[e] = fma2(mul2(add2(x.pair(k * kEach + e), minus), r2), f[e], bk[e]);
            out.put(y, gr, k, a.cols, f);
        }
    }
    out.done(y, gr, a.cols, live);
}

// One row of the backward pass from registers: dx out, column sums on.  (Past
// the row's end dy is zero and adds nothing; so is all of it for a row that is
// not there.)
template <typename T, int EPV, int NV, typename Params, typename After, typename Out>
__device__ __forceinline__ void norm_grad_row(const NormGradArgs &a, const Row<T, EPV, NV> &x, const Row<T, EPV, NV> &dy,
                                              const Params &w, uint64_t (&sw)[NV * EPV / 2], uint64_t (&sb)[NV * EPV / 2],
                                              float mean, float rstd, Group &gr, int64_t row, bool live, const After &after, Out out)
{
    constexpr int kEach = EPV == 1 ? 1 : EPV / 2, kGroups = Row<T, EPV, NV>::kPairs / kEach;
    const float inv = 1.0f / static_cast<float>(a.cols);
    const uint64_t minus = pack2(-mean, -mean), r2 = pack2(rstd, rstd);
    uint64_t s0 = 0, s1 = 0;
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
        uint64_t wk[kEach];
        w.get(gr, k, wk);
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int j = k * kEach + e;
            const uint64_t h = mul2(add2(x.pair(j), minus), r2), d = dy.pair(j), g = mul2(d, wk[e]);
            sw[j] = fma2(d, h, sw[j]);
            sb[j] = add2(sb[j], d);
            s0 = add2(s0, g);
            s1 = fma2(g, h, s1);
        }
    }
    float s[2] = {unpack2(s0).x + unpack2(s0).y, unpack2(s1).x + unpack2(s1).y};
    row_sum(s, gr);
    after();                              // (every thread of the row holds its elements in registers)
    T *dx = static_cast<T *>(a.dx) + (live ? row_offset(a.dx_at, a.inner, a.rows, row) : 0);
    if (live) {
        const float m0 = -s[0] * inv, m1 = -s[1] * inv;
        const uint64_t m02 = pack2(m0, m0), m12 = pack2(m1, m1);
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
            uint64_t f[kEach];
            w.get(gr, k, f);
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const int j = k * kEach + e;
                const uint64_t h = mul2(add2(x.pair(j), minus), r2);
                f[e] = mul2(r2, fma2(h, m12, fma2(dy.pair(j), f[e], m02)));
            }
            out.put(dx, gr, k, a.cols, f);
        }
    }
    out.done(dx, gr, a.cols, live);
}

// A CTA's column sums into its row of partial sums.  Groups that share a warp
// are added up by shuffles; then every group (or warp) puts its sums down in
// `columns` ([groups or warps][2 cols]) and all threads add them up, column by
// column, in a fixed order.  One group of several warps needs neither.
template <int EPV, int NV>
__device__ __forceinline__ void write_partial(const NormGradArgs &a, uint64_t (&sw)[NV * EPV / 2],
                                              uint64_t (&sb)[NV * EPV / 2], const Group &gr, int workers, float *columns)
{
    float *out = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
    const int parts = gr.tpr < 32 ? workers / 32 : workers / gr.tpr;
    if (static_cast<int>(threadIdx.x) < workers) {
        for (int o = gr.tpr; o < 32; o <<= 1)
#pragma unroll
            for (int j = 0; j < NV * EPV / 2; ++j) {
                sw[j] = add2(sw[j], __shfl_xor_sync(0xffffffffu, sw[j], o));
                sb[j] = add2(sb[j], __shfl_xor_sync(0xffffffffu, sb[j], o));
            }
        const int part = gr.tpr < 32 ? threadIdx.x >> 5 : gr.g;
        float *to = parts > 1 ? columns + static_cast<int64_t>(part) * 2 * a.cols : out;
        if (gr.tpr >= 32 || (static_cast<int>(threadIdx.x) & 31) < gr.tpr) {
#pragma unroll
            for (int j = 0; j < NV * EPV / 2; ++j) {
                const float2 v = unpack2(sw[j]), u = unpack2(sb[j]);
                // (columns of the pair's two elements)
                const int c0 = EPV == 1 ? gr.lane + 2 * j * gr.tpr : (gr.lane + 2 * j / EPV * gr.tpr) * EPV + 2 * j % EPV;
                const int c1 = EPV == 1 ? c0 + gr.tpr : c0 + 1;
                if (c0 < a.cols) {
                    to[c0] = v.x;
                    to[a.cols + c0] = u.x;
                }
                if (c1 < a.cols) {
                    to[c1] = v.y;
                    to[a.cols + c1] = u.y;
                }
            }
        }
    }
    if (parts == 1) return;
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * a.cols; c += blockDim.x) {
        float v = columns[c];
        for (int p = 1; p < parts; ++p) v += columns[p * 2 * a.cols + c];
        out[c] = v;
    }
}

// ---------------------------------------------------------------------------
// direct
// ---------------------------------------------------------------------------
// (rows up to kNormMaxCols: 2048 slots of 8 or 4096 of 4 take 4 a thread, single
// elements 16; THREADS bounds the CTA, and so the registers a thread may have.
// The longest rows' backward pass asks for one CTA per SM: left to itself the
// compiler gives its 1024 threads 32 registers and spills: 2300 x 12002 fp32 347
// us, and 201 with the 64 that there are.)
constexpr int kDirectGroups = 8;               // groups of several warps in a CTA

template <typename T, int EPV, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_direct_kernel(const NormArgs a, int tpr)
{
    __shared__ float scratch[kDirectGroups][2][32][2];
    tc::griddep_wait();
    if (threadIdx.x == 0) tc::griddep_launch_dependents();
    const int per = blockDim.x / tpr;
    Group gr = {tpr, static_cast<int>(threadIdx.x) / tpr, static_cast<int>(threadIdx.x) % tpr, nullptr, 0};
    if (tpr > 32) gr.scratch = scratch[gr.g];
    const Own<EPV, NV> w(a.weight, a.weight_format, gr, a.cols, 1.f), b(a.bias, a.weight_format, gr, a.cols, 0.f);
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * per; r0 < a.rows; r0 += static_cast<int64_t>(gridDim.x) * per) {
        const int64_t row = r0 + threadIdx.x / tpr;
        const bool live = row < a.rows;   // whole warps stay for the shuffles (with zeros)
        const Row<T, EPV, NV> x(static_cast<const T *>(a.x) + row_offset(a.x_at, a.inner, a.rows, live ? row : r0), gr, live ? a.cols : 0);
        norm_row(a, x, w, b, gr, row, live, Straight<T, EPV>());
    }
}

template <typename T, int EPV, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS, NV == 16 && THREADS == 1024 ? 1 : 0) norm_grad_direct_kernel(const NormGradArgs a, int tpr)
{
    extern __shared__ __align__(128) uint8_t smem[];    // with a weight and several groups: their column sums
    __shared__ float scratch[kDirectGroups][2][32][2];
    tc::griddep_wait();
    if (threadIdx.x == 0) tc::griddep_launch_dependents();
    const int per = blockDim.x / tpr;
    Group gr = {tpr, static_cast<int>(threadIdx.x) / tpr, static_cast<int>(threadIdx.x) % tpr, nullptr, 0};
    if (tpr > 32) gr.scratch = scratch[gr.g];
    uint64_t sw[NV * EPV / 2] = {}, sb[NV * EPV / 2] = {};
    const Own<EPV, NV> w(a.weight, a.weight_format, gr, a.cols, 1.f);
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * per; r0 < a.rows; r0 += static_cast<int64_t>(gridDim.x) * per) {
        const int64_t row = r0 + threadIdx.x / tpr;
        const bool live = row < a.rows;
        const int64_t at = live ? row : r0;
        const int cols = live ? a.cols : 0;   // (a row that is not there is zeros, not row r0, which may be overwritten meanwhile)
        const Row<T, EPV, NV> x(static_cast<const T *>(a.x) + row_offset(a.x_at, a.inner, a.rows, at), gr, cols);
        const Row<T, EPV, NV> dy(static_cast<const T *>(a.dy) + row_offset(a.dy_at, a.inner, a.rows, at), gr, cols);
        norm_grad_row(a, x, dy, w, sw, sb, live ? a.mean[at] : 0.f, live ? a.rstd[at] : 0.f, gr, row, live, [] {}, Straight<T, EPV>());
    }
    if (!a.weight) return;
    write_partial<EPV, NV>(a, sw, sb, gr, blockDim.x, reinterpret_cast<float *>(smem));
}

// ---------------------------------------------------------------------------
// streamed
// ---------------------------------------------------------------------------
// The ring holds about kRingWant, at least three stages, and at most kRingMost
// (with a copy of the weight in the backward pass); what it leaves is L1.
constexpr uint32_t kRingWant = 112 * 1024, kRingMost = 208 * 1024;
constexpr int kMaxStages = 24;
constexpr int kStreamThreads = 384;           // of the row groups; 128 registers each

// The ring: `tensors` x `per` rows of row_bytes a stage; a batch is the next
// `per` rows, one for each group of threads.
struct Stream {
    int tpr, per, stages;
    uint32_t row_bytes, slot_bytes, stage_bytes;    // slot_bytes: of one row in the ring
    WaitLimit limit;
};

// Rows that are not whole 16-byte vectors, or do not begin at one, are brought
// with the 16-byte blocks that they begin and end in (what belongs to their
// neighbours is dropped), and lie in the ring to 16 bytes as they do in memory.
// A block that reaches out of the tensor, at its first and last row, is not
// touched: its elements are copied one by one.
struct Piece {
    uintptr_t a0, b0, b1, head, tail, end;          // bulk copy [b0, b1); elements [begin, head) and [tail, end)
};

__device__ __forceinline__ Piece piece_of(const char *src, int64_t bytes, const char *low, const char *high)
{
    Piece p;
    const uintptr_t s = reinterpret_cast<uintptr_t>(src);
    p.end = s + bytes;
    p.a0 = s & ~static_cast<uintptr_t>(15);
    const uintptr_t a1 = (p.end + 15) & ~static_cast<uintptr_t>(15);
    p.b0 = p.a0 < reinterpret_cast<uintptr_t>(low) && p.a0 < s ? p.a0 + 16 : p.a0;
    p.b1 = a1 > reinterpret_cast<uintptr_t>(high) && a1 > p.end ? a1 - 16 : a1;
    if (p.b1 < p.b0) p.b1 = p.b0;
    p.head = p.b0 > p.a0 ? min(p.b0, p.end) : s;
    p.tail = max(max(p.b1, p.head), s);
    return p;
}

template <typename T>
__device__ __forceinline__ void piece_ends(const Piece &p, const char *src, uint8_t *to)
{
    const uintptr_t s = reinterpret_cast<uintptr_t>(src);
    if (p.head <= s && p.tail >= p.end) return;
    for (uintptr_t i = s; i < p.head; i += sizeof(T)) *reinterpret_cast<T *>(to + (i - p.a0)) = *reinterpret_cast<const T *>(i);
    for (uintptr_t i = p.tail; i < p.end; i += sizeof(T)) *reinterpret_cast<T *>(to + (i - p.a0)) = *reinterpret_cast<const T *>(i);
    fence_proxy_async_smem();                       // (a later copy comes to the same place)
}

__device__ __forceinline__ void piece_load(const Piece &p, uint8_t *to, uint32_t full)
{
    if (p.b1 > p.b0)
        bulk_load(smem_addr(to) + static_cast<uint32_t>(p.b0 - p.a0), reinterpret_cast<const void *>(p.b0),
                  static_cast<uint32_t>(p.b1 - p.b0), full);
}

// One past the last byte of a tensor's last row.
__device__ __forceinline__ const char *rows_end(const char *src, const RowsAt &at, int64_t inner, int64_t rows, int size, uint32_t row_bytes)
{
    return src + row_offset(at, inner, rows, rows - 1) * size + row_bytes;
}

// Where row r0 + g of a batch lies in the ring.
__device__ __forceinline__ const uint8_t *row_in_ring(const Stream &s, const uint8_t *slots, const void *src, const RowsAt &at,
                                                      int64_t inner, int64_t rows, int size, int64_t r0, int g)
{
    const uintptr_t base = reinterpret_cast<uintptr_t>(src);
    if (inner >= rows && at.stride * size == s.row_bytes)
        return slots + ((base + r0 * s.row_bytes) & 15u) + g * s.row_bytes;
    return slots + g * s.slot_bytes + ((base + row_offset(at, inner, rows, min(r0 + g, rows - 1)) * size) & 15u);
}

// Brings a CTA's batches of N tensors' rows.  One warp; a copy per tensor where
// its rows lie end to end.
template <int N>
__device__ __forceinline__ void stream_rows(const Stream &s, const char *const (&src)[N], const RowsAt (&at)[N],
                                            int64_t inner, int size, int64_t rows, uint32_t ring, uint32_t full, uint32_t empty, volatile int *abort)
{
    const int lane = threadIdx.x & 31;
    int n = 0;
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * s.per; r0 < rows;
         r0 += static_cast<int64_t>(gridDim.x) * s.per, ++n) {
        const int st = n % s.stages;
        const int have = static_cast<int>(min(static_cast<int64_t>(s.per), rows - r0));
        bool go = true;
        if (n >= s.stages)
            go = tc::wait(empty + 8 * st, (n / s.stages - 1) & 1, abort, s.limit.timeout_ns, s.limit.status, s.limit.host_status);
        if (!__all_sync(0xffffffffu, go)) break;
        if (lane == 0) mbar_arrive_expect_tx(full + 8 * st, N * have * s.row_bytes);
        __syncwarp();
#pragma unroll
        for (int t = 0; t < N; ++t) {
            const uint32_t dst = ring + st * s.stage_bytes + t * s.per * s.row_bytes;
            if (inner >= rows && at[t].stride * size == s.row_bytes) {
                if (lane == 0) bulk_load(dst, src[t] + r0 * s.row_bytes, have * s.row_bytes, full + 8 * st);
            } else {
                for (int r = lane; r < have; r += 32)
                    bulk_load(dst + r * s.row_bytes, src[t] + row_offset(at[t], inner, rows, r0 + r) * size, s.row_bytes,
                              full + 8 * st);
            }
        }
    }
    // what is still in flight lands before the CTA ends
    for (int k = max(0, n - s.stages); k < n; ++k) tc::drain(full + 8 * (k % s.stages), (k / s.stages) & 1, s.limit.timeout_ns);
}

// The same for rows that begin at any element.
template <typename T, int N>
__device__ __forceinline__ void stream_odd_rows(const Stream &s, const char *const (&src)[N], const RowsAt (&at)[N], int64_t inner,
                                                int64_t rows, uint8_t *ring, uint32_t full, uint32_t empty, volatile int *abort)
{
    const int lane = threadIdx.x & 31;
    int n = 0;
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * s.per; r0 < rows;
         r0 += static_cast<int64_t>(gridDim.x) * s.per, ++n) {
        const int st = n % s.stages;
        const int have = static_cast<int>(min(static_cast<int64_t>(s.per), rows - r0));
        bool go = true;
        if (n >= s.stages)
            go = tc::wait(empty + 8 * st, (n / s.stages - 1) & 1, abort, s.limit.timeout_ns, s.limit.status, s.limit.host_status);
        if (!__all_sync(0xffffffffu, go)) break;
        // the bytes of the copies and the tensor's ends first, then the copies
        uint32_t bytes = 0;
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
#pragma unroll
            for (int t = 0; t < N; ++t) {
                uint8_t *to = ring + st * s.stage_bytes + t * s.per * s.slot_bytes;
                const bool whole = inner >= rows && at[t].stride * static_cast<int64_t>(sizeof(T)) == s.row_bytes;
                const char *high = rows_end(src[t], at[t], inner, rows, sizeof(T), s.row_bytes);
                for (int r = lane; r < (whole ? 1 : have); r += 32) {
                    const char *from = src[t] + (whole ? r0 * s.row_bytes : row_offset(at[t], inner, rows, r0 + r) * static_cast<int64_t>(sizeof(T)));
                    const Piece p = piece_of(from, whole ? static_cast<int64_t>(have) * s.row_bytes : s.row_bytes, src[t], high);
                    if (pass == 0) {
                        piece_ends<T>(p, from, to + r * s.slot_bytes);
                        bytes += static_cast<uint32_t>(p.b1 - p.b0);
                    } else {
                        piece_load(p, to + r * s.slot_bytes, full + 8 * st);
                    }
                }
            }
            if (pass == 0) {
                bytes = __reduce_add_sync(0xffffffffu, bytes);
                __syncwarp();                       // every lane's elements are in the ring ahead of the arrival
                if (lane == 0) mbar_arrive_expect_tx(full + 8 * st, bytes);
                __syncwarp();                       // and the arrival is ahead of the copies
            }
        }
    }
    for (int k = max(0, n - s.stages); k < n; ++k) tc::drain(full + 8 * (k % s.stages), (k / s.stages) & 1, s.limit.timeout_ns);
}

struct StreamShared {
    float scratch[6][2][32][2];           // per group of several warps
    uint64_t full[kMaxStages], empty[kMaxStages];
    int abort;
};

// The setup both kernels share; the ring begins after the fixed part.
__device__ __forceinline__ void stream_setup(StreamShared &sh, const Stream &s, int workers)
{
    if (threadIdx.x == 0) {
        for (int i = 0; i < s.stages; ++i) {
            mbar_init(smem_addr(&sh.full[i]), 1);
            mbar_init(smem_addr(&sh.empty[i]), workers / 32);
        }
        sh.abort = (*reinterpret_cast<volatile unsigned int *>(s.limit.status) != 0u) ? 1 : 0;
        mbar_init_fence();
    }
    tc::griddep_wait();
    if (threadIdx.x == 0) tc::griddep_launch_dependents();
}

// (a wait that runs out is reported and answered with whatever the stage
// holds: every thread goes on, so that none is left at a barrier)
__device__ __forceinline__ void stream_wait(StreamShared &sh, const Stream &s, int st, int parity)
{
    tc::wait(smem_addr(&sh.full[st]), parity, &sh.abort, s.limit.timeout_ns, s.limit.status, s.limit.host_status);
}

__device__ __forceinline__ void stream_release(StreamShared &sh, int st)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(smem_addr(&sh.empty[st]));
}

template <typename T, int EPV, int NV, bool ODD>
__device__ __forceinline__ Row<T, EPV, NV> ring_row(const Stream &s, const uint8_t *slots, const void *src, const RowsAt &at, int64_t inner,
                                                    int64_t rows, int64_t r0, const Group &gr, int cols)
{
    if (ODD) return Row<T, EPV, NV>(row_in_ring(s, slots, src, at, inner, rows, sizeof(T), r0, gr.g), gr, cols, Shifted());
    return Row<T, EPV, NV>(reinterpret_cast<const T *>(slots + gr.g * s.slot_bytes), gr, cols);
}

template <typename T, int NV, bool ODD>
__global__ void __launch_bounds__(kStreamThreads + 32, 1)
    norm_stream_kernel(const __grid_constant__ NormArgs a, const __grid_constant__ Stream s)
{
    constexpr int EPV = 16 / sizeof(T);
    extern __shared__ __align__(128) uint8_t smem[];
    StreamShared &sh = *reinterpret_cast<StreamShared *>(smem);
    uint8_t *ring = smem + (sizeof(StreamShared) + 127) / 128 * 128;
    const int workers = s.per * s.tpr;
    stream_setup(sh, s, workers);
    __syncthreads();
    const bool skip = sh.abort != 0;
    if (static_cast<int>(threadIdx.x) >= workers) {
        const char *const src[1] = {static_cast<const char *>(a.x)};
        const RowsAt at[1] = {a.x_at};
        if (!skip) {
            if (ODD)
                stream_odd_rows<T, 1>(s, src, at, a.inner, a.rows, ring, smem_addr(sh.full), smem_addr(sh.empty), &sh.abort);
            else
                stream_rows<1>(s, src, at, a.inner, sizeof(T), a.rows, smem_addr(ring), smem_addr(sh.full), smem_addr(sh.empty), &sh.abort);
        }
        return;
    }
    if (skip) return;
    Group gr = {s.tpr, static_cast<int>(threadIdx.x) / s.tpr, static_cast<int>(threadIdx.x) % s.tpr, nullptr, 0};
    if (s.tpr > 32) gr.scratch = sh.scratch[gr.g];
    const Own<EPV, NV, true, ODD> w(a.weight, a.weight_format, gr, a.cols, 1.f), b(a.bias, a.weight_format, gr, a.cols, 0.f);
    int st = 0, parity = 0;
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * s.per; r0 < a.rows; r0 += static_cast<int64_t>(gridDim.x) * s.per) {
        const int64_t row = r0 + gr.g;
        stream_wait(sh, s, st, parity);
        const Row<T, EPV, NV> x = ring_row<T, EPV, NV, ODD>(s, ring + st * s.stage_bytes, a.x, a.x_at, a.inner, a.rows, r0, gr,
                                                            row < a.rows ? a.cols : 0);
        stream_release(sh, st);
        if (++st == s.stages) {
            st = 0;
            parity ^= 1;
        }
        if (ODD)
            norm_row(a, x, w, b, gr, row, row < a.rows, Staged<T, EPV>{ring + s.stages * s.stage_bytes + gr.g * s.slot_bytes});
        else
            norm_row(a, x, w, b, gr, row, row < a.rows, Straight<T, EPV>());
    }
}

template <typename T, bool ODD>
__global__ void __launch_bounds__(kStreamThreads + 32, 1)
    norm_grad_stream_kernel(const __grid_constant__ NormGradArgs a, const __grid_constant__ Stream s)
{
    constexpr int EPV = 16 / sizeof(T), NV = 2;
    extern __shared__ __align__(128) uint8_t smem[];
    StreamShared &sh = *reinterpret_cast<StreamShared *>(smem);
    float *weight = reinterpret_cast<float *>(smem + (sizeof(StreamShared) + 127) / 128 * 128);
    uint8_t *ring = reinterpret_cast<uint8_t *>(weight) + (a.weight ? (4 * a.cols + 127) / 128 * 128 : 0);
    const int padded = (a.cols + EPV - 1) / EPV * EPV;
    uint8_t *const staging = ring + s.stages * s.stage_bytes;
    const int workers = s.per * s.tpr;
    stream_setup(sh, s, workers);
    if (a.weight)
        for (int c = threadIdx.x; c < padded; c += blockDim.x) {
            float one[1] = {0.f};
            if (c < a.cols) load_params<1>(a.weight, a.weight_format, c, one);
            weight[c] = one[0];
        }
    __syncthreads();
    const bool skip = sh.abort != 0;
    Group gr = {s.tpr, static_cast<int>(threadIdx.x) / s.tpr, static_cast<int>(threadIdx.x) % s.tpr, nullptr, 0};
    uint64_t sw[NV * EPV / 2] = {}, sb[NV * EPV / 2] = {};
    if (static_cast<int>(threadIdx.x) >= workers) {
        const char *const src[2] = {static_cast<const char *>(a.x), static_cast<const char *>(a.dy)};
        const RowsAt at[2] = {a.x_at, a.dy_at};
        if (!skip) {
            if (ODD)
                stream_odd_rows<T, 2>(s, src, at, a.inner, a.rows, ring, smem_addr(sh.full), smem_addr(sh.empty), &sh.abort);
            else
                stream_rows<2>(s, src, at, a.inner, sizeof(T), a.rows, smem_addr(ring), smem_addr(sh.full), smem_addr(sh.empty), &sh.abort);
        }
    } else if (!skip) {
        if (s.tpr > 32) gr.scratch = sh.scratch[gr.g];
        const Own<EPV, NV, false> w(a.weight ? weight : nullptr, GN_FORMAT_FP32, gr, padded, 1.f);
        const int64_t step = static_cast<int64_t>(gridDim.x) * s.per;
        int64_t row = static_cast<int64_t>(blockIdx.x) * s.per + gr.g;
        // (the statistics are asked for a batch ahead)
        float mean = row < a.rows ? __ldg(a.mean + row) : 0.f, rstd = row < a.rows ? __ldg(a.rstd + row) : 0.f;
        int st = 0, parity = 0;
        for (int64_t r0 = row - gr.g; r0 < a.rows; r0 += step, row += step) {
            const float mean_now = mean, rstd_now = rstd;
            if (row + step < a.rows) {
                mean = __ldg(a.mean + row + step);
                rstd = __ldg(a.rstd + row + step);
            }
            stream_wait(sh, s, st, parity);
            const uint8_t *at = ring + st * s.stage_bytes;
            const int cols = row < a.rows ? a.cols : 0;
            const Row<T, EPV, NV> x = ring_row<T, EPV, NV, ODD>(s, at, a.x, a.x_at, a.inner, a.rows, r0, gr, cols);
            const Row<T, EPV, NV> dy = ring_row<T, EPV, NV, ODD>(s, at + s.per * s.slot_bytes, a.dy, a.dy_at, a.inner, a.rows, r0, gr, cols);
            stream_release(sh, st);
            if (++st == s.stages) {
                st = 0;
                parity ^= 1;
            }
            if (ODD)
                norm_grad_row(a, x, dy, w, sw, sb, mean_now, rstd_now, gr, row, row < a.rows, [] {},
                              Staged<T, EPV>{staging + gr.g * s.slot_bytes});
            else
                norm_grad_row(a, x, dy, w, sw, sb, mean_now, rstd_now, gr, row, row < a.rows, [] {}, Straight<T, EPV>());
        }
    }
    if (!a.weight) return;
    __syncthreads();                      // every copy has landed, every row is done: the ring is free
    write_partial<EPV, NV>(a, sw, sb, gr, workers, reinterpret_cast<float *>(ring));
}

// The same for a row that 384 threads with two slots do not hold: four slots a
// thread, one row per batch, and no loader warp.  The barrier of a row's sums
// says that its stage has been read, and thread 0 then fills the stage again.
// With a loader warp the CTA's 13 warps are given registers as 16, 128 a thread,
// and the column sums spill beside a ring that leaves little L1; 12 warps may
// have 168 (bf16, weight in fp32, with the kernel that adds the columns up: 4608 x
// 12288 173 us with a loader warp, 120 us so, 4608 x 8192 118 and 99 us; fp32,
// which does not spill either way, 4608 x 4096 57 and 58 us).  768 threads with
// two slots spill as well (181 us).
template <typename T, bool ODD>
__global__ void __launch_bounds__(kStreamThreads, 1)
    norm_grad_wide_kernel(const __grid_constant__ NormGradArgs a, const __grid_constant__ Stream s)
{
    constexpr int EPV = 16 / sizeof(T), NV = 4;
    extern __shared__ __align__(128) uint8_t smem[];
    StreamShared &sh = *reinterpret_cast<StreamShared *>(smem);
    float *weight = reinterpret_cast<float *>(smem + (sizeof(StreamShared) + 127) / 128 * 128);
    uint8_t *ring = reinterpret_cast<uint8_t *>(weight) + (a.weight ? (4 * a.cols + 127) / 128 * 128 : 0);
    const int padded = (a.cols + EPV - 1) / EPV * EPV;
    stream_setup(sh, s, s.tpr);
    if (a.weight)
        for (int c = threadIdx.x; c < padded; c += blockDim.x) {
            float one[1] = {0.f};
            if (c < a.cols) load_params<1>(a.weight, a.weight_format, c, one);
            weight[c] = one[0];
        }
    __syncthreads();
    const bool skip = sh.abort != 0;
    Group gr = {s.tpr, 0, static_cast<int>(threadIdx.x), sh.scratch[0], 0};
    uint64_t sw[NV * EPV / 2] = {}, sb[NV * EPV / 2] = {};
    if (!skip) {
        int issued = 0, fill = 0;             // copies begun, and the stage of the next (thread 0)
        int64_t next = blockIdx.x;
        const auto load = [&] {
            if (next >= a.rows) return;
            const uint32_t full = smem_addr(&sh.full[fill]);
            uint8_t *const to = ring + fill * s.stage_bytes;
            const char *const x0 = static_cast<const char *>(a.x), *const dy0 = static_cast<const char *>(a.dy);
            const char *const xr = x0 + row_offset(a.x_at, a.inner, a.rows, next) * static_cast<int64_t>(sizeof(T));
            const char *const dyr = dy0 + row_offset(a.dy_at, a.inner, a.rows, next) * static_cast<int64_t>(sizeof(T));
            if (ODD) {
                const Piece px = piece_of(xr, s.row_bytes, x0, rows_end(x0, a.x_at, a.inner, a.rows, sizeof(T), s.row_bytes));
                const Piece pd = piece_of(dyr, s.row_bytes, dy0, rows_end(dy0, a.dy_at, a.inner, a.rows, sizeof(T), s.row_bytes));
                piece_ends<T>(px, xr, to);
                piece_ends<T>(pd, dyr, to + s.slot_bytes);
                mbar_arrive_expect_tx(full, static_cast<uint32_t>(px.b1 - px.b0 + pd.b1 - pd.b0));
                piece_load(px, to, full);
                piece_load(pd, to + s.slot_bytes, full);
            } else {
                mbar_arrive_expect_tx(full, 2 * s.row_bytes);
                bulk_load(smem_addr(to), xr, s.row_bytes, full);
                bulk_load(smem_addr(to) + s.slot_bytes, dyr, s.row_bytes, full);
            }
            next += gridDim.x;
            ++issued;
            if (++fill == s.stages) fill = 0;
        };
        if (threadIdx.x == 0)
            for (int i = 0; i < s.stages; ++i) load();
        const Own<EPV, NV, false> w(a.weight ? weight : nullptr, GN_FORMAT_FP32, gr, padded, 1.f);
        int64_t row = blockIdx.x;
        // (the statistics are asked for a row ahead)
        float mean = row < a.rows ? __ldg(a.mean + row) : 0.f, rstd = row < a.rows ? __ldg(a.rstd + row) : 0.f;
        int st = 0, parity = 0;
        bool good = true;
        for (; row < a.rows; row += gridDim.x) {
            const float mean_now = mean, rstd_now = rstd;
            if (row + gridDim.x < a.rows) {
                mean = __ldg(a.mean + row + gridDim.x);
                rstd = __ldg(a.rstd + row + gridDim.x);
            }
            // (after a wait that ran out nothing more is asked for)
            good = tc::wait(smem_addr(&sh.full[st]), parity, &sh.abort, s.limit.timeout_ns, s.limit.status, s.limit.host_status) && good;
            const uint8_t *at = ring + st * s.stage_bytes;
            const Row<T, EPV, NV> x = ring_row<T, EPV, NV, ODD>(s, at, a.x, a.x_at, a.inner, a.rows, row, gr, a.cols);
            const Row<T, EPV, NV> dy = ring_row<T, EPV, NV, ODD>(s, at + s.slot_bytes, a.dy, a.dy_at, a.inner, a.rows, row, gr, a.cols);
            if (++st == s.stages) {
                st = 0;
                parity ^= 1;
            }
            const auto refill = [&] {
                if (threadIdx.x == 0 && good) load();
            };
            if (ODD)
                norm_grad_row(a, x, dy, w, sw, sb, mean_now, rstd_now, gr, row, true, refill,
                              Staged<T, EPV>{ring + s.stages * s.stage_bytes});
            else
                norm_grad_row(a, x, dy, w, sw, sb, mean_now, rstd_now, gr, row, true, refill, Straight<T, EPV>());
        }
        // what is still in flight lands before the CTA ends
        if (threadIdx.x == 0 && !good)
            for (int k = max(0, issued - s.stages); k < issued; ++k)
                tc::drain(smem_addr(&sh.full[k % s.stages]), (k / s.stages) & 1, s.limit.timeout_ns);
    }
    if (!a.weight) return;
    write_partial<EPV, NV>(a, sw, sb, gr, s.tpr, nullptr);    // (one row at a time: nothing to add up)
}

// dw and db from the CTAs' partial sums: a warp's lanes take 32 neighbouring
// columns, the eight warps every eighth partial each, added up in a fixed order.
__global__ void __launch_bounds__(256) norm_columns_kernel(const NormGradArgs a, int blocks)
{
    __shared__ float part[8][32];
    tc::griddep_wait();
    if (threadIdx.x == 0) tc::griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x * 32 + lane;
    float v = 0.f;
    if (c < 2 * a.cols)
#pragma unroll 8
        for (int b = warp; b < blocks; b += 8) v += a.partial[static_cast<int64_t>(b) * 2 * a.cols + c];
    part[warp][lane] = v;
    __syncthreads();
    if (warp != 0 || c >= 2 * a.cols) return;
#pragma unroll
    for (int w = 1; w < 8; ++w) v += part[w][lane];
    if (c < a.cols)
        store_param(a.dweight, a.weight_format, c, v);
    else
        store_param(a.dbias, a.weight_format, c - a.cols, v);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// Threads per row for `slots` of a row, nv each.
int threads_per_row(int slots, int nv)
{
    const int need = (slots + nv - 1) / nv;
    if (need > 32) return (need + 31) / 32 * 32;
    int t = 1;
    while (t < need) t *= 2;
    return t;
}

bool vectors_ok(int cols, int epv, const void *const *ptrs, int n, const int64_t *strides)
{
    if (cols % epv) return false;
    for (int i = 0; i < n; ++i)
        if (reinterpret_cast<uintptr_t>(ptrs[i]) % 16 || strides[2 * i] % epv || strides[2 * i + 1] % epv) return false;
    return true;
}

// The streamed form's shape, or stages = 0 where it does not pay: it wants at
// least three stages of ring, and at least four batches of rows for every SM.
// A thread has two slots of a row as long as that takes at most all threads;
// the forward pass, which has no column sums to keep, four of a row longer than
// a warp's two.  With one slot (24 warps on a row of 6144) the reductions'
// instructions took longer than the row's memory does (62 us forward for 4608 x
// 6144); with four the backward pass has a kernel of its own.
Stream stream_shape(int64_t rows, int cols, int size, bool vec, int tensors, size_t fixed, int sm_count, int *nv)
{
    Stream s = {};
    const int slots = (cols * size + 15) / 16;
    *nv = slots <= (tensors == 1 ? 64 : 2 * kStreamThreads) ? 2 : 4;
    s.tpr = threads_per_row(slots, *nv);
    s.per = std::max(1, kStreamThreads / s.tpr);
    s.row_bytes = static_cast<uint32_t>(cols * size);
    // (a row that begins at any element: its blocks, and one more that is read)
    s.slot_bytes = vec ? s.row_bytes : (s.row_bytes + 15) / 16 * 16 + 32;
    s.stage_bytes = static_cast<uint32_t>(tensors * s.per) * s.slot_bytes;
    if (!vec) fixed += s.per * s.slot_bytes;
    s.stages = static_cast<int>(std::min<size_t>(kMaxStages, std::max<size_t>(3, kRingWant / s.stage_bytes)));
    if (!vec && s.stages == 3 && 3 * static_cast<size_t>(s.stage_bytes) + fixed > kRingMost) s.stages = 2;
    if (s.tpr > kStreamThreads || s.stages * static_cast<size_t>(s.stage_bytes) + fixed > kRingMost ||
        rows < static_cast<int64_t>(4) * sm_count * s.per)
        s.stages = 0;
    return s;
}

constexpr size_t kStreamFixed = (sizeof(StreamShared) + 127) / 128 * 128;
constexpr size_t kStreamBytes = kStreamFixed + kRingMost;

size_t weight_copy(const NormGradArgs &a) { return a.weight ? (4u * static_cast<size_t>(a.cols) + 127) / 128 * 128 : 0; }

// Floats that `threads` of a CTA put down in write_partial.
size_t columns_bytes(const NormGradArgs &a, int tpr, int threads)
{
    const size_t parts = static_cast<size_t>(tpr < 32 ? threads / 32 : threads / tpr);
    return a.weight && parts > 1 ? parts * 8u * static_cast<size_t>(a.cols) : 0;
}

// Bytes of the results' rows in shared memory.
size_t staging_bytes(const Stream &s) { return s.slot_bytes == s.row_bytes ? 0 : static_cast<size_t>(s.per) * s.slot_bytes; }

template <typename T, int NV, bool ODD>
cudaError_t forward_stream(const NormArgs &a, const Stream &s, int sm_count, cudaStream_t st)
{
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_shared(reinterpret_cast<const void *>(norm_stream_kernel<T, NV, ODD>), kStreamBytes, done);
    if (e != cudaSuccess) return e;
    return tc::launch_pdl(norm_stream_kernel<T, NV, ODD>, dim3(static_cast<unsigned>(sm_count)), dim3(s.per * s.tpr + 32),
                          kStreamFixed + s.stages * s.stage_bytes + staging_bytes(s), st, a, s);
}

template <typename T, bool ODD>
cudaError_t backward_stream(const NormGradArgs &a, const Stream &s, int sm_count, cudaStream_t st)
{
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_shared(reinterpret_cast<const void *>(norm_grad_stream_kernel<T, ODD>), kStreamBytes, done);
    if (e != cudaSuccess) return e;
    // (384 threads with two slots of 16 bytes: the column sums take at most 48 KB)
    const size_t ring = std::max<size_t>(s.stages * s.stage_bytes + staging_bytes(s), columns_bytes(a, s.tpr, s.per * s.tpr));
    return tc::launch_pdl(norm_grad_stream_kernel<T, ODD>, dim3(static_cast<unsigned>(sm_count)), dim3(s.per * s.tpr + 32),
                          kStreamFixed + weight_copy(a) + ring, st, a, s);
}

template <typename T, bool ODD>
cudaError_t backward_wide(const NormGradArgs &a, const Stream &s, int sm_count, cudaStream_t st)
{
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_shared(reinterpret_cast<const void *>(norm_grad_wide_kernel<T, ODD>), kStreamBytes, done);
    if (e != cudaSuccess) return e;
    return tc::launch_pdl(norm_grad_wide_kernel<T, ODD>, dim3(static_cast<unsigned>(sm_count)), dim3(s.tpr),
                          kStreamFixed + weight_copy(a) + s.stages * s.stage_bytes + staging_bytes(s), st, a, s);
}

// The direct form: up to nv slots a thread, a row's threads one CTA or, for
// short rows, a part of one of 256 threads.
struct Direct {
    int nv, tpr, threads;
};

Direct direct_shape(int slots, bool vec, int64_t rows, int sm_count)
{
    Direct d;
    if (vec) {
        // few slots: one each, so that a short row is spread over a warp
        d.nv = slots <= 1024 ? 1 : 4;
    } else {
        // Single elements: four a thread while the rows do not fill the SMs, then 8
        // or 16, which leave a row to a warp or a few and several rows to a CTA
        // (forward and backward, fp32 and weight: 12000 x 131 21 + 43 us with four,
        // 13 + 24 with 8; 6600 x 4001 106 + 136 with four, 54 + 83 with 16).  Rows of
        // up to 1024 fill them later (3001 x 1003 18 + 24 with four, 18 + 31 with 16;
        // 4800 x 515 20 + 26 and 18 + 28; 9000 x 515 29 + 36 and 22 + 36).
        const int few = (slots > 256 && slots <= 1024 ? 32 : 4) * sm_count;
        d.nv = slots <= 128 || (slots <= 4096 && rows <= few) ? 4 : slots <= 256 ? 8 : 16;
    }
    d.tpr = threads_per_row(slots, d.nv);
    d.threads = d.tpr <= 32 ? 256 : vec ? d.tpr : d.tpr * std::max(1, 256 / d.tpr);
    return d;
}

template <typename T>
cudaError_t forward(const NormArgs &a, int sm_count, const WaitLimit &limit, cudaStream_t s)
{
    constexpr int EPV = 16 / sizeof(T);
    const void *ptrs[] = {a.x, a.y};
    const int64_t strides[] = {a.x_at.outer, a.x_at.stride, a.y_at.outer, a.y_at.stride};
    const bool vec = vectors_ok(a.cols, EPV, ptrs, 2, strides);
    int nv;
    Stream st = stream_shape(a.rows, a.cols, sizeof(T), vec, 1, 0, sm_count, &nv);
    st.limit = limit;
    if (st.stages && vec) return nv == 2 ? forward_stream<T, 2, false>(a, st, sm_count, s) : forward_stream<T, 4, false>(a, st, sm_count, s);
    // (Rows that begin at any element: half types are streamed, 4608 x 6143 bf16 73
    // us straight and 54 so; fp32 elements are wide enough for plain loads, 4608 x
    // 6143 77 us streamed and 67 straight.)
    if constexpr (sizeof(T) == 2) {
        if (st.stages) return nv == 2 ? forward_stream<T, 2, true>(a, st, sm_count, s) : forward_stream<T, 4, true>(a, st, sm_count, s);
    }
    const Direct d = direct_shape(vec ? a.cols / EPV : a.cols, vec, a.rows, sm_count);
    const int64_t per = d.threads / d.tpr;
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>((a.rows + per - 1) / per, 8 * sm_count)));
    if (vec && d.nv == 1) return tc::launch_pdl(norm_direct_kernel<T, EPV, 1, 1024>, grid, dim3(d.threads), 0, s, a, d.tpr);
    if (vec) return tc::launch_pdl(norm_direct_kernel<T, EPV, 4, EPV == 8 ? 512 : 1024>, grid, dim3(d.threads), 0, s, a, d.tpr);
    if (d.nv == 4) return tc::launch_pdl(norm_direct_kernel<T, 1, 4, 1024>, grid, dim3(d.threads), 0, s, a, d.tpr);
    if (d.nv == 8) return tc::launch_pdl(norm_direct_kernel<T, 1, 8, 256>, grid, dim3(d.threads), 0, s, a, d.tpr);
    return tc::launch_pdl(norm_direct_kernel<T, 1, 16, 1024>, grid, dim3(d.threads), 0, s, a, d.tpr);
}

template <typename T>
cudaError_t backward(const NormGradArgs &a, int sm_count, const WaitLimit &limit, cudaStream_t s, int *blocks)
{
    constexpr int EPV = 16 / sizeof(T);
    const void *ptrs[] = {a.x, a.dy, a.dx};
    const int64_t strides[] = {a.x_at.outer, a.x_at.stride, a.dy_at.outer, a.dy_at.stride, a.dx_at.outer, a.dx_at.stride};
    const bool vec = vectors_ok(a.cols, EPV, ptrs, 3, strides);
    int nv;
    Stream st = stream_shape(a.rows, a.cols, sizeof(T), vec, 2, weight_copy(a), sm_count, &nv);
    st.limit = limit;
    // (Rows that begin at any element: half types are streamed, 4608 x 6143 bf16 323
    // us straight and 90 so; fp32 where a row takes more than 256 threads straight,
    // 4608 x 6143 112 us straight and 104 so, 6600 x 4001 83 and 118.)
    if (st.stages && (vec || sizeof(T) == 2 || a.cols > 4096)) {
        *blocks = sm_count;
        if (vec) return nv == 2 ? backward_stream<T, false>(a, st, sm_count, s) : backward_wide<T, false>(a, st, sm_count, s);
        if constexpr (sizeof(T) == 2) {
            if (nv == 2) return backward_stream<T, true>(a, st, sm_count, s);
        }
        return backward_wide<T, true>(a, st, sm_count, s);
    }
    const Direct d = direct_shape(vec ? a.cols / EPV : a.cols, vec, a.rows, sm_count);
    const int64_t per = d.threads / d.tpr;
    *blocks = static_cast<int>(std::min<int64_t>((a.rows + per - 1) / per, layer_norm_blocks(a.rows, a.cols, sm_count)));
    const dim3 grid(static_cast<unsigned>(*blocks));
    // (several groups for rows of up to 128 threads: 32 KB at most)
    const size_t smem = columns_bytes(a, d.tpr, d.threads);
    if (vec && d.nv == 1) return tc::launch_pdl(norm_grad_direct_kernel<T, EPV, 1, 1024>, grid, dim3(d.threads), smem, s, a, d.tpr);
    if (vec) return tc::launch_pdl(norm_grad_direct_kernel<T, EPV, 4, EPV == 8 ? 512 : 1024>, grid, dim3(d.threads), smem, s, a, d.tpr);
    if (d.nv == 4) return tc::launch_pdl(norm_grad_direct_kernel<T, 1, 4, 1024>, grid, dim3(d.threads), smem, s, a, d.tpr);
    if (d.nv == 8) return tc::launch_pdl(norm_grad_direct_kernel<T, 1, 8, 256>, grid, dim3(d.threads), smem, s, a, d.tpr);
    if (d.threads <= 512) return tc::launch_pdl(norm_grad_direct_kernel<T, 1, 16, 512>, grid, dim3(d.threads), smem, s, a, d.tpr);
    return tc::launch_pdl(norm_grad_direct_kernel<T, 1, 16, 1024>, grid, dim3(d.threads), smem, s, a, d.tpr);
}

}  // namespace

int layer_norm_blocks(int64_t rows, int, int sm_count)
{
    return static_cast<int>(std::min<int64_t>(rows, 4 * sm_count));
}

cudaError_t launch_layer_norm(const NormArgs &a, int sm_count, const WaitLimit &limit, cudaStream_t s)
{
    if (a.format == GN_FORMAT_BF16) return forward<__nv_bfloat16>(a, sm_count, limit, s);
    if (a.format == GN_FORMAT_FP16) return forward<__half>(a, sm_count, limit, s);
    return forward<float>(a, sm_count, limit, s);
}

cudaError_t launch_layer_norm_backward(const NormGradArgs &a, int sm_count, const WaitLimit &limit, cudaStream_t s,
                                       int *launches)
{
    cudaError_t e;
    int blocks = 0;
    if (a.format == GN_FORMAT_BF16)
        e = backward<__nv_bfloat16>(a, sm_count, limit, s, &blocks);
    else if (a.format == GN_FORMAT_FP16)
        e = backward<__half>(a, sm_count, limit, s, &blocks);
    else
        e = backward<float>(a, sm_count, limit, s, &blocks);
    if (e != cudaSuccess) return e;
    *launches = 1;
    if (!a.weight) return e;
    e = tc::launch_pdl(norm_columns_kernel, dim3((2 * a.cols + 31) / 32), dim3(256), 0, s, a, blocks);
    if (e == cudaSuccess) *launches = 2;
    return e;
}

}  // namespace gn
