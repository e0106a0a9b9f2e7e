// cattn_kernels.cu -- attention of new tokens over the paged cache: one warp for
// each query and head, key by key.
#include <algorithm>
#include <cmath>

#include "cache_common.cuh"
#include "pattn_common.cuh"
#include "tc_common.cuh"

namespace gn {
namespace {

using namespace pattn;

template <typename T>
__global__ void __launch_bounds__(256) cached_rows_kernel(const __grid_constant__ CachedAttn p)
{
    tc::griddep_wait();
    if (threadIdx.x == 0) tc::griddep_launch_dependents();
    const gn_cache &c = p.c;
    const gn_attn_cached_args &a = p.a;
    const int lane = threadIdx.x & 31;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * 8;
    for (int64_t n = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); n < a.tokens * a.heads; n += warps) {
        const int64_t i = n / a.heads;
        const int h = static_cast<int>(n - i * a.heads), hk = h / p.group;
        const int doc = c.cu ? doc_of(c.cu, c.sequences, static_cast<int>(i)) : static_cast<int>(i / (a.tokens / c.sequences));
        float m = -INFINITY, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        if (doc >= 0) {
            const cache::Sequence s = cache::sequence_of(c, a.tokens, doc);
            const int pos = s.first_place() + static_cast<int>(i) - s.begin;
            const int end = a.causal ? min(s.length, pos + 1) : s.length;
            const float4 q = load4<T>(a.q, i * a.q_token + h * a.q_head, lane, c.dim);
            const float slope = a.slopes ? __ldg(a.slopes + h) : 0.f;
            for (int j = 0; j < end; ++j) {
                const int page = cache::page_of(c, doc, j / c.page_size), slot = j % c.page_size;
                float4 k = make_float4(0.f, 0.f, 0.f, 0.f), v = k;
                if (page >= 0 && 4 * lane < c.dim) {
                    const uint32_t kb = *reinterpret_cast<const uint32_t *>(static_cast<const uint8_t *>(c.k_pages) + page * c.k_page + slot * c.k_token + hk * c.k_head + 4 * lane);
                    const uint32_t vb = *reinterpret_cast<const uint32_t *>(static_cast<const uint8_t *>(c.v_pages) + page * c.v_page + slot * c.v_token + hk * c.v_head + 4 * lane);
                    const float ks = __ldg(c.k_scales + static_cast<int64_t>(page) * c.kv_heads + hk);
                    const float vs = __ldg(c.v_scales + static_cast<int64_t>(page) * c.kv_heads + hk);
                    const float2 k0 = e4m3_values(kb), k1 = e4m3_values(kb >> 16), v0 = e4m3_values(vb), v1 = e4m3_values(vb >> 16);
                    k = make_float4(k0.x * ks, k0.y * ks, k1.x * ks, k1.y * ks);
                    v = make_float4(v0.x * vs, v0.y * vs, v1.x * vs, v1.y * vs);
                }
                float t = warp_sum(dot4(q, k)) * a.scale;
                if (a.cap > 0.f) t = a.cap * tanh_full(t / a.cap);
                t = (t - slope * fabsf(static_cast<float>(pos - j))) * kLog2e;
                if (t > m) {
                    const float f = m == -INFINITY ? 0.f : ex2_approx(m - t);
                    l *= f;
                    o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
                    m = t;
                }
                const float w = t == -INFINITY ? 0.f : ex2_approx(t - m);
                l += w;
                axpy4(o, w, v);
            }
        }
        const float inv = l == 0.f ? 0.f : 1.0f / l;
        store4<T>(a.out, (i * a.heads + h) * c.dim, lane, c.dim, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
        if (lane == 0) a.lse[h * a.tokens + i] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    }
}

}  // namespace

size_t cached_attn_workspace_bytes(int64_t, int, int, int, int, int) { return 256; }

cudaError_t launch_cached_attn(const CachedAttn &p, int sm_count, const WaitLimit &, cudaStream_t s, int *launches)
{
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>((p.a.tokens * p.a.heads + 7) / 8, 8 * sm_count)));
    const auto kernel = p.a.format == GN_FORMAT_BF16 ? cached_rows_kernel<__nv_bfloat16> : cached_rows_kernel<__half>;
    const cudaError_t e = tc::launch_pdl(kernel, grid, dim3(256), 0, s, p);
    if (e == cudaSuccess) ++*launches;
    return e;
}

}  // namespace gn
