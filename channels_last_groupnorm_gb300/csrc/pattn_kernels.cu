// pattn_kernels.cu -- attention of packed documents on sm_103a.
//
// Query i of a document sees a run [lo_i, hi_i) of the document's keys: all of
// them, or (causal) those up to its own position and those of the document's
// prefix.  With t_ij = scale q_i . k_j, capped (t <- cap tanh(t / cap)) and
// biased (t <- t - slope |pos_i - j|):
//   lse_i = log sum_j exp(t_ij),  p_ij = exp(t_ij - lse_i),  out_i = sum_j p_ij v_j
//   delta_i = dout_i . out_i,     ds_ij = p_ij (dout_i . v_j - delta_i) (1 - tanh^2)
//   dq_i = scale sum_j ds_ij k_j, dk_j = scale sum_i ds_ij q_i, dv_j = sum_i p_ij dout_i
// with dk and dv summed over the query heads that share a key / value head.
// A query that sees no key has out = 0, lse = -inf and adds nothing to any
// gradient.  Keys outside a query's run are never read for it.
#include <algorithm>

#include "gn_ptx.cuh"
#include "pattn_common.cuh"
#include "tc_common.cuh"
#include "tc_ptx.cuh"

namespace gn {
namespace {

using namespace pattn;

// ---------------------------------------------------------------------------
// Rows: one query token and HC of the query heads of one key / value head per
// cluster, the keys split between the cluster's CTAs and their warps.
// ---------------------------------------------------------------------------
constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;

// Sums N values over groups of L neighbouring lanes, halving the values at
// each step while there are several: afterwards a lane holds the sums with
// numbers (its place in the group) * N / L + 0, 1, ...
template <int N, int L>
__device__ __forceinline__ void spread_sum(float (&v)[N], int lane)
{
    int n = N;
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) {
        if (n > 1) {
            n >>= 1;
            const bool up = (lane & o) != 0;
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                if (i < n) {
                    const float send = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
                }
            }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
        }
    }
}

// LPK lanes read one key (8 channels each), so a warp takes 32 / LPK keys per
// step and UN steps at a time.
template <typename T, int LPK, int HC, int UN>
__global__ void __launch_bounds__(kRowThreads) attn_rows_kernel(const PackedAttn p, int chunks, int splits)
{
    constexpr int KPS = 32 / LPK, KPI = KPS * UN;   // keys per step and per iteration of a warp
    constexpr int NV = UN * HC;                     // (head, step) scores per lane group
    constexpr int PER = NV > LPK ? NV / LPK : 1;    // of which a lane ends up with this many
    __shared__ float so[kRowWarps][HC][128];
    __shared__ float sm[kRowWarps][HC], sl[kRowWarps][HC];
    __shared__ float co[HC][128];
    __shared__ float cm[HC], cl[HC];
    tc::griddep_wait();
    if (threadIdx.x == 0) tc::griddep_launch_dependents();
    const gn_attn_packed_args &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int i = static_cast<int>(blockIdx.x / splits), split = static_cast<int>(blockIdx.x % splits);
    const int hk = blockIdx.y / chunks, h0 = hk * p.group + (blockIdx.y % chunks) * HC;
    const int heads = min(HC, (hk + 1) * p.group - h0);
    const int place = lane % LPK, sub = lane / LPK, c0 = place * 8;
    const bool wide = c0 < a.dim;
    const Span span = query_span(a, i);
    const int len = span.hi - span.lo, share = (len + splits - 1) / splits;
    const int lo = min(span.hi, span.lo + split * share), hi = min(span.hi, lo + share);

    float q[HC][8];
#pragma unroll
    for (int h = 0; h < HC; ++h) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (wide && h < heads)
            v = *reinterpret_cast<const uint4 *>(static_cast<const T *>(a.q) + i * a.q_token + (h0 + h) * a.q_head + c0);
        unpack8<T>(v, q[h]);
    }
    float o[HC][8] = {};
    float m[HC];
    float l[PER] = {};
#pragma unroll
    for (int h = 0; h < HC; ++h) m[h] = -INFINITY;
    // the first of this lane's scores: number = head * UN + step (with fewer
    // scores than lanes, SHARED neighbouring lanes hold the same one)
    constexpr int SHARED = NV < LPK ? LPK / NV : 1;
    const int mine = place * PER / SHARED;
    const T *kbase = static_cast<const T *>(a.k) + hk * a.k_head + c0;
    const T *vbase = static_cast<const T *>(a.v) + hk * a.v_head + c0;

    for (int j0 = lo + warp * KPI; j0 < hi; j0 += kRowWarps * KPI) {
        uint4 kv[UN], vv[UN];
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const int j = j0 + u * KPS + sub;
            const bool in = wide && j < hi;
            kv[u] = in ? __ldg(reinterpret_cast<const uint4 *>(kbase + j * a.k_token)) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const int j = j0 + u * KPS + sub;
            const bool in = wide && j < hi;
            vv[u] = in ? __ldg(reinterpret_cast<const uint4 *>(vbase + j * a.v_token)) : make_uint4(0u, 0u, 0u, 0u);
        }
        float s[NV];
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            float k[8];
            unpack8<T>(kv[u], k);
#pragma unroll
            for (int h = 0; h < HC; ++h) {
                float d = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) d = fmaf(q[h][e], k[e], d);
                s[h * UN + u] = d;
            }
        }
        spread_sum<NV, LPK>(s, lane);
        bool grew = false;
#pragma unroll
        for (int n = 0; n < PER; ++n) {
            const int h = (mine + n) / UN, j = j0 + ((mine + n) % UN) * KPS + sub;
            float slack;
            const float slope = a.slopes && h < heads ? __ldg(a.slopes + h0 + h) : 0.f;
            s[n] = j < hi ? score_log2(a, slope, s[n], span.pos, j, slack) : -INFINITY;
            float mh = m[0];
#pragma unroll
            for (int g = 1; g < HC; ++g) mh = h == g ? m[g] : mh;
            // the running maximum only moves when a score is more than 2^8
            // above it: the weights stay below 2^8 and nothing is lost in fp32
            grew = grew || s[n] > mh + 8.0f || s[n] != s[n];
        }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
            for (int h = 0; h < HC; ++h) {
                float top = -INFINITY;
#pragma unroll
                for (int n = 0; n < PER; ++n)
                    if ((mine + n) / UN == h) top = fmaxf(top, s[n]);
#pragma unroll
                for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                top = fmaxf(top, m[h]);
                const float f = m[h] == -INFINITY ? 0.f : ex2_approx(m[h] - top);
#pragma unroll
                for (int n = 0; n < PER; ++n)
                    if ((mine + n) / UN == h) l[n] *= f;
#pragma unroll
                for (int e = 0; e < 8; ++e) o[h][e] *= f;
                m[h] = top;
            }
        }
#pragma unroll
        for (int n = 0; n < PER; ++n) {
            const int h = (mine + n) / UN;
            float mh = m[0];
#pragma unroll
            for (int g = 1; g < HC; ++g) mh = h == g ? m[g] : mh;
            s[n] = s[n] == -INFINITY ? 0.f : ex2_approx(s[n] - mh);
            l[n] += s[n];
        }
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            float v[8];
            unpack8<T>(vv[u], v);
#pragma unroll
            for (int h = 0; h < HC; ++h) {
                const int number = h * UN + u;
                const int from = sub * LPK + number / PER * SHARED;
                const float w = __shfl_sync(0xffffffffu, s[number % PER], from);
#pragma unroll
                for (int e = 0; e < 8; ++e) o[h][e] = fmaf(w, v[e], o[h][e]);
            }
        }
    }
    // the warp's lane groups, the CTA's warps, then the cluster's CTAs
#pragma unroll
    for (int h = 0; h < HC; ++h) {
        float lh = 0.f;
#pragma unroll
        for (int n = 0; n < PER; ++n)
            if ((mine + n) / UN == h && place % SHARED == 0) lh += l[n];
        lh = warp_sum(lh);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
#pragma unroll
            for (int x = LPK; x < 32; x <<= 1) o[h][e] += __shfl_xor_sync(0xffffffffu, o[h][e], x);
        }
        if (sub == 0 && wide)
#pragma unroll
            for (int e = 0; e < 8; ++e) so[warp][h][c0 + e] = o[h][e];
        if (lane == 0) {
            sm[warp][h] = m[h];
            sl[warp][h] = lh;
        }
    }
    __syncthreads();
    for (int n = threadIdx.x; n < HC * a.dim; n += kRowThreads) {
        const int h = n / a.dim, c = n - h * a.dim;
        float top = -INFINITY, sum = 0.f, out = 0.f;
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) top = fmaxf(top, sm[w][h]);
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) {
            if (sm[w][h] == -INFINITY && sl[w][h] == 0.f) continue;   // saw nothing (so[] is zero)
            const float f = ex2_approx(sm[w][h] - top);
            sum = fmaf(f, sl[w][h], sum);
            out = fmaf(f, so[w][h][c], out);
        }
        co[h][c] = out;
        if (c == 0) {
            cm[h] = top;
            cl[h] = sum;
        }
    }
    if (splits > 1)
        cluster_sync_all();
    else
        __syncthreads();
    const uint32_t acm = smem_addr(cm), acl = smem_addr(cl), aco = smem_addr(co);
    const auto peer = [](uint32_t addr, int rank) {
        float v;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(addr, rank)) : "memory");
        return v;
    };
    for (int n = split * kRowThreads + threadIdx.x; n < heads * a.dim; n += splits * kRowThreads) {
        const int h = n / a.dim, c = n - h * a.dim;
        float top, sum, out;
        if (splits == 1) {
            top = cm[h];
            sum = cl[h];
            out = co[h][c];
        } else {
            top = -INFINITY;
            sum = out = 0.f;
            for (int r = 0; r < splits; ++r) top = fmaxf(top, peer(acm + 4u * h, r));
            for (int r = 0; r < splits; ++r) {
                const float mr = peer(acm + 4u * h, r), lr = peer(acl + 4u * h, r);
                if (mr == -INFINITY && lr == 0.f) continue;
                const float f = ex2_approx(mr - top);
                sum = fmaf(f, lr, sum);
                out = fmaf(f, peer(aco + 4u * (128u * h + c), r), out);
            }
        }
        const bool empty = sum == 0.f;   // no key, or scores of -inf only
        const float v = empty ? 0.f : out / sum;
        T *dst = static_cast<T *>(a.out) + (static_cast<int64_t>(i) * a.heads + h0 + h) * a.dim + c;
        *dst = static_cast<T>(v);
        if (c == 0 && a.lse)
            a.lse[static_cast<int64_t>(h0 + h) * a.tokens_q + i] = empty ? -INFINITY : (top + log2f(sum)) * kLn2;
    }
    if (splits > 1) cluster_sync_all();   // a CTA's sums stay until every peer has read them
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
template <typename T, int LPK, int HC, int UN>
cudaError_t launch_rows(const PackedAttn &p, int splits, cudaStream_t s)
{
    const int chunks = (p.group + HC - 1) / HC;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = static_cast<unsigned>(splits);
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.a.tokens_q * splits), static_cast<unsigned>(p.a.kv_heads * chunks));
    cfg.blockDim = dim3(kRowThreads);
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = splits > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, attn_rows_kernel<T, LPK, HC, UN>, p, chunks, splits);
}

template <typename T, int LPK>
cudaError_t launch_rows_heads(const PackedAttn &p, int splits, cudaStream_t s)
{
    if (p.group == 1) return launch_rows<T, LPK, 1, 8>(p, splits, s);
    if (p.group == 2) return launch_rows<T, LPK, 2, 4>(p, splits, s);
    return launch_rows<T, LPK, 4, 4>(p, splits, s);
}

template <typename T>
cudaError_t rows_forward(const PackedAttn &p, int sm_count, cudaStream_t s)
{
    // splits: enough CTAs to fill the GPU, as long as each has 256 keys of an
    // average document to read
    const int chunks = (p.group + 3) / 4;
    const int64_t keys = p.a.tokens_k / std::max(1, p.a.docs);
    int splits = 1;
    while (splits < 8 && p.a.tokens_q * p.a.kv_heads * chunks * splits < 4 * sm_count && keys / (2 * splits) >= 256)
        splits *= 2;
    return p.a.dim <= 64 ? launch_rows_heads<T, 8>(p, splits, s) : launch_rows_heads<T, 16>(p, splits, s);
}

}  // namespace

cudaError_t launch_packed_attn(const PackedAttn &p, int sm_count, const WaitLimit &limit, cudaStream_t s, int *launches)
{
    cudaError_t e;
    if (p.a.tokens_k > 0 && p.a.tokens_q > static_cast<int64_t>(4) * p.a.docs)
        e = launch_packed_attn_tiles(p, limit, s);
    else
        e = p.a.format == GN_FORMAT_BF16 ? rows_forward<__nv_bfloat16>(p, sm_count, s)
                                                       : rows_forward<__half>(p, sm_count, s);
    if (e == cudaSuccess) ++*launches;
    return e;
}

}  // namespace gn
