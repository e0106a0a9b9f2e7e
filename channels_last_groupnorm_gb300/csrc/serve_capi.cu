// serve_capi.cu -- the extern "C" entries (declared in include/gnsilu.h) of RMS norm
// and of the paged cache in 8 bits.  Argument validation here; the kernels are in
// rms_kernels.cu, append_kernels.cu and cattn_*.cu.
#include <cmath>
#include <cstdint>
#include <utility>

#include "../../include/gnsilu.h"
#include "block_checks.h"
#include "block_internal.h"
#include "capi_util.h"

using namespace gn_block;

extern "C" {

// ---- RMS norm --------------------------------------------------------------------
int gn_rms_norm(const void *x, const void *residual, const void *weight, void *y, void *total, float *scales,
                float *rstd, int64_t rows, int64_t cols, int64_t inner, const int64_t *strides, float eps, int format,
                int weight_format, void *stream)
{
    if (!strides || (rows != 0 && (!x || !y || !residual != !total))) return GN_ERR_NULL;
    if (!format_ok(format) || (weight && !format_ok(weight_format))) return GN_ERR_FORMAT;
    if (rows < 0 || inner < 1 || (rows > inner && rows > UINT32_MAX)) return GN_ERR_SHAPE;
    if (!norm_cols_ok(cols)) return GN_ERR_CHANNELS;
    if (!std::isfinite(eps) || eps < 0.f) return GN_ERR_EPS;
    const size_t size = format_size(format), wsize = weight ? format_size(weight_format) : 1, ysize = scales ? 1 : size;
    if (addr(x) % size || addr(residual) % size || addr(total) % size || addr(y) % ysize || addr(weight) % wsize ||
        addr(scales) % 4 || addr(rstd) % 4)
        return GN_ERR_ALIGN;
    gn::RmsArgs a = {};
    Range in, res, out, sum;
    if (rows > kMaxElements || !norm_rows(&in, &a.x_at, x, rows, cols, inner, strides, size, true) ||
        (residual && !norm_rows(&res, &a.residual_at, residual, rows, cols, inner, strides + 2, size, true)) ||
        !norm_rows(&out, &a.y_at, y, rows, cols, inner, strides + 4, ysize, false) ||
        (total && !norm_rows(&sum, &a.total_at, total, rows, cols, inner, strides + 6, size, false)))
        return GN_ERR_SHAPE;
    const auto same = [](const gn::RowsAt &p, const gn::RowsAt &q) { return p.stride == q.stride && p.outer == q.outer; };
    const size_t sb = 4u * static_cast<size_t>(rows);
    const Range w = {weight, wsize * static_cast<size_t>(cols)}, sc = {scales, sb}, rs = {rstd, sb};
    if (!(y == x && !residual && !scales && same(a.y_at, a.x_at)) && overlap(out, in)) return GN_ERR_ALIAS;
    if (!(total == x && same(a.total_at, a.x_at)) && overlap(sum, in)) return GN_ERR_ALIAS;
    if (!(total == residual && same(a.total_at, a.residual_at)) && overlap(sum, res)) return GN_ERR_ALIAS;
    if (overlap(out, res) || overlap(out, sum) || overlap(out, w) || overlap(sum, w) || overlap(sc, rs)) return GN_ERR_ALIAS;
    for (const Range &o : {sc, rs})
        for (const Range &i : {in, res, out, sum, w})
            if (overlap(o, i)) return GN_ERR_ALIAS;
    DeviceInfo d;
    const int rc = ready(&d);
    if (rc != GN_OK) return rc;
    if (rows == 0) return GN_OK;
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.y = y;
    a.total = total;
    a.scales = scales;
    a.rstd = rstd;
    a.rows = rows;
    a.cols = static_cast<int>(cols);
    a.inner = inner;
    a.eps = eps;
    a.format = format;
    a.weight_format = weight_format;
    const cudaError_t e = gn::launch_rms_norm(a, d.sm_count, static_cast<cudaStream_t>(stream));
    return launched(e, e == cudaSuccess);
}

size_t gn_rms_norm_workspace_bytes(int64_t rows, int64_t cols)
{
    if (rows < 0 || !norm_cols_ok(cols)) return 0;
    int dev = -1;
    DeviceInfo d;
    if (current_device(&dev, &d) != GN_OK) return 0;
    const size_t bytes = 4u * static_cast<size_t>(cols) *
                         static_cast<size_t>(gn::rms_norm_blocks(rows > 0 ? rows : 1, d.sm_count));
    return (bytes + 255) / 256 * 256;
}

int gn_rms_norm_backward(const void *dy, const void *total, const void *weight, const float *rstd, const void *dtotal,
                         void *dx, void *dweight, int64_t rows, int64_t cols, int64_t inner, const int64_t *strides,
                         int format, int weight_format, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!strides || (rows != 0 && (!dy || !total || !rstd || !dx))) return GN_ERR_NULL;
    if (weight ? (!dweight || !workspace) : dweight != nullptr) return GN_ERR_NULL;
    if (!format_ok(format) || (weight && !format_ok(weight_format))) return GN_ERR_FORMAT;
    if (rows < 0 || inner < 1 || (rows > inner && rows > UINT32_MAX)) return GN_ERR_SHAPE;
    if (!norm_cols_ok(cols)) return GN_ERR_CHANNELS;
    const size_t size = format_size(format), wsize = weight ? format_size(weight_format) : 1;
    if (addr(dy) % size || addr(total) % size || addr(dtotal) % size || addr(dx) % size || addr(rstd) % 4 ||
        addr(weight) % wsize || addr(dweight) % wsize || (weight && addr(workspace) % 256))
        return GN_ERR_ALIGN;
    gn::RmsGradArgs a = {};
    Range g, in, back, out;
    if (rows > kMaxElements || !norm_rows(&g, &a.dy_at, dy, rows, cols, inner, strides, size, true) ||
        !norm_rows(&in, &a.total_at, total, rows, cols, inner, strides + 2, size, true) ||
        (dtotal && !norm_rows(&back, &a.dtotal_at, dtotal, rows, cols, inner, strides + 4, size, true)) ||
        !norm_rows(&out, &a.dx_at, dx, rows, cols, inner, strides + 6, size, false))
        return GN_ERR_SHAPE;
    const auto fits = [&](const void *p, const gn::RowsAt &at, const Range &r) {
        return (dx == p && at.stride == a.dx_at.stride && at.outer == a.dx_at.outer) || !overlap(out, r);
    };
    if (!fits(dy, a.dy_at, g) || !fits(total, a.total_at, in) || (dtotal && !fits(dtotal, a.dtotal_at, back))) return GN_ERR_ALIAS;
    const size_t wb = wsize * static_cast<size_t>(cols);
    const Range w = {weight, wb}, dw = {dweight, wb}, r = {rstd, 4u * static_cast<size_t>(rows)};
    const Range ws = {weight ? workspace : nullptr, workspace_bytes};
    if (overlap(out, w) || overlap(out, r) || overlap(out, dw) || overlap(out, ws) || overlap(dw, ws)) return GN_ERR_ALIAS;
    for (const Range &o : {dw, ws})
        for (const Range &i : {g, in, back, w, r})
            if (overlap(o, i)) return GN_ERR_ALIAS;
    DeviceInfo d;
    const int rc = ready(&d);
    if (rc != GN_OK) return rc;
    if (weight && workspace_bytes < gn_rms_norm_workspace_bytes(rows, cols)) return GN_ERR_WORKSPACE;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (rows == 0) return weight ? launched(cudaMemsetAsync(dweight, 0, wb, s), 0) : GN_OK;
    a.dy = dy;
    a.total = total;
    a.weight = weight;
    a.dtotal = dtotal;
    a.rstd = rstd;
    a.dx = dx;
    a.dweight = dweight;
    a.rows = rows;
    a.cols = static_cast<int>(cols);
    a.inner = inner;
    a.format = format;
    a.weight_format = weight_format;
    a.partial = static_cast<float *>(workspace);
    int launches = 0;
    const cudaError_t e = gn::launch_rms_norm_backward(a, d.sm_count, s, &launches);
    return launched(e, launches);
}

// ---- the paged cache ---------------------------------------------------------------
namespace {

constexpr int64_t kMaxTokens = 1 << 30;

struct Axis {
    int64_t n, stride;
};

// One of the two pools: its bytes, and the bytes that each of its axes spans.
struct Pool {
    Range all;
    Axis axes[3];              // the longest stride first
};

// False if elements lie on one another or it overflows: every axis has to step
// over all that the axes of shorter strides span.
bool pool_of(Pool *r, const void *p, const gn_cache &c, int64_t page, int64_t token, int64_t head)
{
    r->axes[0] = {c.pages, page};
    r->axes[1] = {c.page_size, token};
    r->axes[2] = {c.kv_heads, head};
    for (int i = 0; i < 3; ++i)
        if (r->axes[i].n > 1 && r->axes[i].stride < 0) return false;
    const auto key = [](const Axis &a) { return a.n > 1 ? a.stride : 0; };
    for (int i = 0; i < 2; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (key(r->axes[j]) > key(r->axes[i])) std::swap(r->axes[i], r->axes[j]);
    int64_t span = c.dim;
    for (int i = 2; i >= 0; --i) {
        const Axis &a = r->axes[i];
        if (a.n <= 1) continue;
        if (a.stride < span || a.stride > kMaxElements / a.n) return false;
        span += (a.n - 1) * a.stride;
        if (span > kMaxElements) return false;
    }
    r->all = {p, static_cast<size_t>(span)};
    return true;
}

// Whether the two pools share bytes: not if they are slices of one buffer, side by
// side within the step of some axis.
bool pools_meet(const Pool &a, const Pool &b, int64_t dim)
{
    if (!overlap(a.all, b.all)) return false;
    const uintptr_t lo = addr(a.all.p) < addr(b.all.p) ? addr(a.all.p) : addr(b.all.p);
    const uintptr_t off = (addr(a.all.p) < addr(b.all.p) ? addr(b.all.p) : addr(a.all.p)) - lo;
    for (int i = 0; i < 3; ++i) {
        // the same axes down to this one, and both slices within its step
        if (a.axes[i].n != b.axes[i].n || (a.axes[i].n > 1 && a.axes[i].stride != b.axes[i].stride)) return true;
        if (a.axes[i].n <= 1) continue;
        int64_t sa = dim, sb = dim;
        for (int j = i + 1; j < 3; ++j) {
            if (a.axes[j].n > 1) sa += (a.axes[j].n - 1) * a.axes[j].stride;
            if (b.axes[j].n > 1) sb += (b.axes[j].n - 1) * b.axes[j].stride;
        }
        const int64_t first = addr(a.all.p) == lo ? sa : sb, second = addr(a.all.p) == lo ? sb : sa;
        if (off + static_cast<uintptr_t>(second) > static_cast<uintptr_t>(a.axes[i].stride)) return true;
        if (off >= static_cast<uintptr_t>(first)) return false;
    }
    return true;
}

struct CacheRanges {
    Pool k, v;
    Range ks, vs, table, lengths, cu;
};

int check_cache(const gn_cache *p, int64_t tokens, CacheRanges *r)
{
    if (!p) return GN_ERR_NULL;
    const gn_cache &c = *p;
    if (!c.k_pages || !c.v_pages || !c.k_scales || !c.v_scales || !c.table || !c.lengths) return GN_ERR_NULL;
    if (tokens < 0 || tokens > kMaxTokens || c.sequences < 1 || c.sequences > (1 << 20) || c.pages < 1 ||
        c.pages > INT32_MAX || c.table_width < 1)
        return GN_ERR_SHAPE;
    if (c.page_size < 8 || c.page_size > 256 || c.page_size % 8 || c.kv_heads < 1 || c.kv_heads > 1024 || c.dim < 16 ||
        c.dim > 128 || c.dim % 16)
        return GN_ERR_CHANNELS;
    if (c.table_width > kMaxTokens / c.page_size || (!c.cu && tokens % c.sequences)) return GN_ERR_SHAPE;
    if (addr(c.k_pages) % 16 || addr(c.v_pages) % 16 || c.k_page % 16 || c.k_token % 16 || c.k_head % 16 || c.v_page % 16 ||
        c.v_token % 16 || c.v_head % 16 || addr(c.k_scales) % 4 || addr(c.v_scales) % 4 || addr(c.table) % 4 ||
        addr(c.lengths) % 4 || addr(c.cu) % 4)
        return GN_ERR_ALIGN;
    if (!pool_of(&r->k, c.k_pages, c, c.k_page, c.k_token, c.k_head) ||
        !pool_of(&r->v, c.v_pages, c, c.v_page, c.v_token, c.v_head))
        return GN_ERR_SHAPE;
    const size_t sb = 4u * static_cast<size_t>(c.pages) * static_cast<size_t>(c.kv_heads);
    r->ks = {c.k_scales, sb};
    r->vs = {c.v_scales, sb};
    r->table = {c.table, 4u * static_cast<size_t>(c.sequences) * static_cast<size_t>(c.table_width)};
    r->lengths = {c.lengths, 4u * static_cast<size_t>(c.sequences)};
    r->cu = {c.cu, 4u * (static_cast<size_t>(c.sequences) + 1)};
    return GN_OK;
}

}  // namespace

int gn_cache_append(const gn_cache *cache, const gn_append_args *args, void *stream)
{
    if (!args) return GN_ERR_NULL;
    const gn_append_args &a = *args;
    CacheRanges r;
    int rc = check_cache(cache, a.tokens, &r);
    if (rc != GN_OK) return rc;
    const gn_cache &c = *cache;
    if (a.tokens != 0 && (!a.k || !a.v || (a.heads > 0 && (!a.q || !a.q_out)) || (a.axes > 0 && !a.positions)))
        return GN_ERR_NULL;
    if (a.axes > 0 && !a.axes_dim) return GN_ERR_NULL;
    if (!format_ok(a.format) ||
        (a.axes > 0 && (a.position_format < GN_POSITIONS_INT32 || a.position_format > GN_POSITIONS_FP32)))
        return GN_ERR_FORMAT;
    if (a.heads < 0 || a.heads > (1 << 16) || a.axes < 0 || a.axes > 8) return GN_ERR_CHANNELS;
    int64_t width = 0;
    for (int n = 0; n < a.axes; ++n) {
        if (a.axes_dim[n] < 2 || a.axes_dim[n] % 2 || a.axes_dim[n] > c.dim) return GN_ERR_CHANNELS;
        width += a.axes_dim[n];
    }
    if (width > c.dim) return GN_ERR_CHANNELS;
    if (a.axes > 0 && (!(a.theta > 0.0) || !std::isfinite(a.theta))) return GN_ERR_EPS;
    const size_t size = format_size(a.format);
    const bool with_q = a.heads > 0;
    const size_t psize = a.position_format == GN_POSITIONS_INT64 ? 8 : 4;
    if ((with_q && (addr(a.q) % size || addr(a.q_out) % size)) || addr(a.k) % size || addr(a.v) % size ||
        (a.axes > 0 && addr(a.positions) % psize))
        return GN_ERR_ALIGN;
    Range q, q_out, k, v;
    if ((with_q && (!strided(&q, a.q, a.tokens, a.q_token, a.heads, a.q_head, c.dim, size) ||
                    !strided(&q_out, a.q_out, a.tokens, a.q_out_token, a.heads, a.q_out_head, c.dim, size) ||
                    collide(a.tokens, a.q_out_token, a.heads, a.q_out_head, c.dim))) ||
        !strided(&k, a.k, a.tokens, a.k_token, c.kv_heads, a.k_head, c.dim, size) ||
        !strided(&v, a.v, a.tokens, a.v_token, c.kv_heads, a.v_head, c.dim, size))
        return GN_ERR_SHAPE;
    const Range positions = {a.axes > 0 ? a.positions : nullptr, psize * static_cast<size_t>(a.tokens) * static_cast<size_t>(a.axes)};
    if (pools_meet(r.k, r.v, c.dim) || overlap(r.ks, r.vs)) return GN_ERR_ALIAS;
    for (const Range &o : {r.k.all, r.v.all, r.ks, r.vs})
        for (const Range &i : {q, k, v, positions, r.table, r.lengths, r.cu, q_out})
            if (overlap(o, i)) return GN_ERR_ALIAS;
    for (const Range &o : {r.ks, r.vs})
        if (overlap(o, r.k.all) || overlap(o, r.v.all)) return GN_ERR_ALIAS;
    if (with_q) {
        const TokenSlice so = {a.q_out, a.q_out_token, (a.heads - 1) * a.q_out_head + c.dim};
        const TokenSlice sq = {a.q, a.q_token, (a.heads - 1) * a.q_head + c.dim};
        const TokenSlice sk = {a.k, a.k_token, (c.kv_heads - 1) * a.k_head + c.dim};
        const TokenSlice sv = {a.v, a.v_token, (c.kv_heads - 1) * a.v_head + c.dim};
        const bool place = a.q == a.q_out && a.q_token == a.q_out_token && a.q_head == a.q_out_head;
        if ((!place && overlap(q_out, q) && !side_by_side(so, sq, size)) || (overlap(q_out, k) && !side_by_side(so, sk, size)) ||
            (overlap(q_out, v) && !side_by_side(so, sv, size)))
            return GN_ERR_ALIAS;
        for (const Range &i : {positions, r.table, r.lengths, r.cu})
            if (overlap(q_out, i)) return GN_ERR_ALIAS;
    }
    DeviceInfo d;
    rc = ready(&d);
    if (rc != GN_OK) return rc;
    if (a.tokens == 0) return GN_OK;
    gn::Append p = {};
    p.c = c;
    p.a = a;
    p.pairs = static_cast<int>(width / 2);
    const double log_theta = a.axes > 0 ? std::log(a.theta) : 0.0;
    int pair = 0;
    for (int n = 0; n < a.axes; ++n)
        for (int i = 0; i < a.axes_dim[n] / 2; ++i, ++pair) {
            p.axis[pair] = static_cast<unsigned char>(n);
            // (theta < 1 turns faster than once a unit: whole turns do not matter)
            const double turns = std::exp(-log_theta * (2.0 * i / static_cast<double>(a.axes_dim[n]))) / 6.283185307179586476925;
            p.turns[pair] = static_cast<uint64_t>(std::ldexp(turns - std::floor(turns), 64));
        }
    const cudaError_t e = gn::launch_cache_append(p, d.sm_count, static_cast<cudaStream_t>(stream));
    return launched(e, e == cudaSuccess);
}

size_t gn_attn_cached_workspace_bytes(int64_t tokens, int64_t sequences, int64_t heads, int64_t kv_heads, int64_t dim)
{
    if (tokens < 0 || tokens > kMaxTokens || sequences < 1 || sequences > (1 << 20) || kv_heads < 1 || heads < 1 ||
        heads > 1024 || heads % kv_heads || dim < 16 || dim > 128 || dim % 16)
        return 0;
    int dev = -1;
    DeviceInfo d;
    if (current_device(&dev, &d) != GN_OK) return 0;
    return gn::cached_attn_workspace_bytes(tokens, static_cast<int>(sequences), static_cast<int>(heads),
                                           static_cast<int>(kv_heads), static_cast<int>(dim), d.sm_count);
}

int gn_attn_cached(const gn_cache *cache, const gn_attn_cached_args *args, void *workspace, size_t workspace_bytes,
                   void *stream)
{
    if (!args) return GN_ERR_NULL;
    const gn_attn_cached_args &a = *args;
    CacheRanges r;
    int rc = check_cache(cache, a.tokens, &r);
    if (rc != GN_OK) return rc;
    const gn_cache &c = *cache;
    if (a.tokens != 0 && (!a.q || !a.out || !a.lse || !workspace)) return GN_ERR_NULL;
    if (a.format != GN_FORMAT_BF16 && a.format != GN_FORMAT_FP16) return GN_ERR_FORMAT;
    if (a.heads < 1 || a.heads > 1024 || a.heads % c.kv_heads) return GN_ERR_CHANNELS;
    if (!std::isfinite(a.scale) || !std::isfinite(a.cap) || a.cap < 0.f) return GN_ERR_EPS;
    if (addr(a.q) % 16 || addr(a.out) % 16 || addr(a.lse) % 4 || addr(a.slopes) % 4 || addr(workspace) % 256 ||
        a.q_token % 8 || a.q_head % 8)
        return GN_ERR_ALIGN;
    Range q;
    if (!strided(&q, a.q, a.tokens, a.q_token, a.heads, a.q_head, c.dim, 2) || (a.tokens > 1 && a.q_token < c.dim) ||
        (a.heads > 1 && a.q_head < c.dim))
        return GN_ERR_SHAPE;
    const size_t rows = static_cast<size_t>(a.tokens) * static_cast<size_t>(a.heads);
    const Range outs[] = {{a.out, 2u * rows * static_cast<size_t>(c.dim)}, {a.lse, 4u * rows}, {workspace, workspace_bytes}};
    const Range slopes = {a.slopes, 4u * static_cast<size_t>(a.heads)};
    for (int n = 0; n < 3; ++n) {
        for (const Range &i : {q, slopes, r.k.all, r.v.all, r.ks, r.vs, r.table, r.lengths, r.cu})
            if (overlap(outs[n], i)) return GN_ERR_ALIAS;
        for (int m = 0; m < n; ++m)
            if (overlap(outs[n], outs[m])) return GN_ERR_ALIAS;
    }
    DeviceInfo d;
    rc = ready(&d);
    if (rc != GN_OK) return rc;
    if (a.tokens == 0) return GN_OK;
    if (workspace_bytes < gn::cached_attn_workspace_bytes(a.tokens, c.sequences, a.heads, c.kv_heads, c.dim, d.sm_count))
        return GN_ERR_WORKSPACE;
    gn::CachedAttn p = {};
    p.c = c;
    p.a = a;
    p.group = a.heads / c.kv_heads;
    p.workspace = workspace;
    int launches = 0;
    const cudaError_t e = gn::launch_cached_attn(p, d.sm_count, {wait_timeout_ns(), d.status_word, d.status_host},
                                                 static_cast<cudaStream_t>(stream), &launches);
    return launched(e, launches);
}

}  // extern "C"
