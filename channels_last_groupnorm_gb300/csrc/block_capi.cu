// block_capi.cu -- the extern "C" entries (declared in include/gnsilu.h) of
// the transformer-block operations: layer norm, rotary positions over several
// axes and attention of packed documents.  Argument validation here; the
// kernels are in norm_kernels.cu, rope_kernels.cu and pattn_kernels.cu.
#include <cmath>
#include <cstdint>

#include "../../include/gnsilu.h"
#include "block_checks.h"
#include "block_internal.h"
#include "capi_util.h"

using namespace gn_block;

extern "C" {

// ---- layer norm --------------------------------------------------------------
int gn_layer_norm(const void *x, const void *weight, const void *bias, void *y, float *mean, float *rstd,
                  int64_t rows, int64_t cols, int64_t inner, const int64_t *strides, float eps, int format,
                  int weight_format, void *stream)
{
    if (!strides || (rows != 0 && (!x || !y))) return GN_ERR_NULL;
    if (bias && !weight) return GN_ERR_NULL;
    if (!format_ok(format) || (weight && !format_ok(weight_format))) return GN_ERR_FORMAT;
    if (rows < 0 || inner < 1 || (rows > inner && rows > UINT32_MAX)) return GN_ERR_SHAPE;
    if (!norm_cols_ok(cols)) return GN_ERR_CHANNELS;
    if (!std::isfinite(eps) || eps < 0.f) return GN_ERR_EPS;
    const size_t size = format_size(format), wsize = weight ? format_size(weight_format) : 1;
    if (addr(x) % size || addr(y) % size || addr(weight) % wsize || addr(bias) % wsize || addr(mean) % 4 ||
        addr(rstd) % 4)
        return GN_ERR_ALIGN;
    Range in, out;
    gn::RowsAt x_at, y_at;
    if (rows > kMaxElements || !norm_rows(&in, &x_at, x, rows, cols, inner, strides, size, true) ||
        !norm_rows(&out, &y_at, y, rows, cols, inner, strides + 2, size, false))
        return GN_ERR_SHAPE;
    const size_t wb = wsize * static_cast<size_t>(cols), sb = 4u * static_cast<size_t>(rows);
    const Range w = {weight, wb}, b = {bias, wb}, m = {mean, sb}, r = {rstd, sb};
    const bool place = x == y && x_at.stride == y_at.stride && x_at.outer == y_at.outer;
    if (!place && overlap(out, in)) return GN_ERR_ALIAS;
    for (const Range &o : {out, m, r})
        if (overlap(o, w) || overlap(o, b)) return GN_ERR_ALIAS;
    if (overlap(m, r) || overlap(m, in) || overlap(r, in) || overlap(m, out) || overlap(r, out)) return GN_ERR_ALIAS;
    DeviceInfo d;
    const int rc = ready(&d);
    if (rc != GN_OK) return rc;
    if (rows == 0) return GN_OK;
    gn::NormArgs a = {x, weight, bias, y, mean, rstd, rows, static_cast<int>(cols), x_at, y_at, inner, eps, format,
                      weight_format};
    const cudaError_t e = gn::launch_layer_norm(a, d.sm_count, {wait_timeout_ns(), d.status_word, d.status_host},
                                               static_cast<cudaStream_t>(stream));
    return launched(e, e == cudaSuccess);
}

size_t gn_layer_norm_workspace_bytes(int64_t rows, int64_t cols)
{
    if (rows < 0 || !norm_cols_ok(cols)) return 0;
    int dev = -1;
    DeviceInfo d;
    if (current_device(&dev, &d) != GN_OK) return 0;
    const size_t bytes = 8u * static_cast<size_t>(cols) *
                         static_cast<size_t>(gn::layer_norm_blocks(rows > 0 ? rows : 1, static_cast<int>(cols), d.sm_count));
    return (bytes + 255) / 256 * 256;
}

int gn_layer_norm_backward(const void *dy, const void *x, const void *weight, const float *mean, const float *rstd,
                           void *dx, void *dweight, void *dbias, int64_t rows, int64_t cols, int64_t inner,
                           const int64_t *strides, int format, int weight_format, void *workspace,
                           size_t workspace_bytes, void *stream)
{
    if (!strides) return GN_ERR_NULL;
    if (rows != 0 && (!dy || !x || !mean || !rstd || !dx)) return GN_ERR_NULL;
    if (weight ? (!dweight || !dbias || !workspace) : (dweight || dbias)) return GN_ERR_NULL;
    if (!format_ok(format) || (weight && !format_ok(weight_format))) return GN_ERR_FORMAT;
    if (rows < 0 || inner < 1 || (rows > inner && rows > UINT32_MAX)) return GN_ERR_SHAPE;
    if (!norm_cols_ok(cols)) return GN_ERR_CHANNELS;
    const size_t size = format_size(format), wsize = weight ? format_size(weight_format) : 1;
    if (addr(dy) % size || addr(x) % size || addr(dx) % size || addr(mean) % 4 || addr(rstd) % 4 ||
        addr(weight) % wsize || addr(dweight) % wsize || addr(dbias) % wsize || (weight && addr(workspace) % 256))
        return GN_ERR_ALIGN;
    Range g, in, out;
    gn::RowsAt dy_at, x_at, dx_at;
    if (rows > kMaxElements || !norm_rows(&g, &dy_at, dy, rows, cols, inner, strides, size, true) ||
        !norm_rows(&in, &x_at, x, rows, cols, inner, strides + 2, size, true) ||
        !norm_rows(&out, &dx_at, dx, rows, cols, inner, strides + 4, size, false))
        return GN_ERR_SHAPE;
    const auto same = [&](const gn::RowsAt &o) { return o.stride == dx_at.stride && o.outer == dx_at.outer; };
    const size_t wb = wsize * static_cast<size_t>(cols), sb = 4u * static_cast<size_t>(rows);
    const Range w = {weight, wb}, dw = {dweight, wb}, db = {dbias, wb}, m = {mean, sb}, r = {rstd, sb};
    const Range ws = {weight ? workspace : nullptr, workspace_bytes};
    if (!(dx == dy && same(dy_at)) && overlap(out, g)) return GN_ERR_ALIAS;
    if (!(dx == x && same(x_at)) && overlap(out, in)) return GN_ERR_ALIAS;
    if (overlap(out, w) || overlap(out, m) || overlap(out, r) || overlap(dw, db) || overlap(ws, out) ||
        overlap(ws, dw) || overlap(ws, db) || overlap(dw, out) || overlap(db, out))
        return GN_ERR_ALIAS;
    for (const Range &o : {dw, db, ws})
        for (const Range &i : {g, in, w, m, r})
            if (overlap(o, i)) return GN_ERR_ALIAS;
    DeviceInfo d;
    const int rc = ready(&d);
    if (rc != GN_OK) return rc;
    if (weight && workspace_bytes < gn_layer_norm_workspace_bytes(rows, cols)) return GN_ERR_WORKSPACE;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (rows == 0) {
        if (!weight) return GN_OK;
        cudaError_t e = cudaMemsetAsync(dweight, 0, wb, s);
        if (e == cudaSuccess) e = cudaMemsetAsync(dbias, 0, wb, s);
        return launched(e, 0);
    }
    gn::NormGradArgs a = {dy, x, weight, mean, rstd, dx, dweight, dbias, rows, static_cast<int>(cols), dy_at,
                          x_at, dx_at, inner, format, weight_format, static_cast<float *>(workspace)};
    int launches = 0;
    const cudaError_t e = gn::launch_layer_norm_backward(a, d.sm_count, {wait_timeout_ns(), d.status_word, d.status_host}, s,
                                                         &launches);
    return launched(e, launches);
}

// ---- rotary positions over several axes ----------------------------------------
int gn_rope_nd(const void *q, const void *k, void *q_out, void *k_out, const int64_t *strides, int64_t tokens,
               int64_t heads, int64_t kv_heads, int64_t dim, const void *positions, int position_format, int64_t axes,
               const int64_t *axes_dim, double theta, int interleaved, int inverse, int format, void *stream)
{
    if (!strides || !axes_dim) return GN_ERR_NULL;
    if (tokens != 0 && (!q || !q_out || !positions)) return GN_ERR_NULL;
    if (!k != !k_out || (!k && kv_heads != 0 && tokens != 0)) return GN_ERR_NULL;
    if (!format_ok(format) || position_format < GN_POSITIONS_INT32 || position_format > GN_POSITIONS_FP32)
        return GN_ERR_FORMAT;
    if (tokens < 0 || heads < 1 || kv_heads < 0 || heads > (1 << 16) || kv_heads > (1 << 16) || (k && kv_heads < 1))
        return GN_ERR_SHAPE;
    if (dim < 2 || dim > 65536 || axes < 1 || axes > 8) return GN_ERR_CHANNELS;
    if ((heads + kv_heads) * dim > gn::kRopeMaxElements) return GN_ERR_SHAPE;
    int64_t width = 0;
    for (int64_t n = 0; n < axes; ++n) {
        if (axes_dim[n] < 2 || axes_dim[n] % 2 || axes_dim[n] > 2 * gn::kRopeMaxPairs) return GN_ERR_CHANNELS;
        width += axes_dim[n];
    }
    if (width > dim || width > 2 * gn::kRopeMaxPairs) return GN_ERR_CHANNELS;
    if (!(theta > 0.0) || !std::isfinite(theta)) return GN_ERR_EPS;
    const size_t size = format_size(format);
    const size_t psize = position_format == GN_POSITIONS_INT64 ? 8 : 4;
    for (const void *p : {q, k, static_cast<const void *>(q_out), static_cast<const void *>(k_out)})
        if (addr(p) % size) return GN_ERR_ALIGN;
    if (addr(positions) % psize) return GN_ERR_ALIGN;

    gn::RopeArgs a = {};
    const void *in[2] = {q, k};
    void *out[2] = {q_out, k_out};
    const int64_t count[2] = {heads, k ? kv_heads : 0};
    Range ri[2], ro[2];
    if (tokens > kMaxElements / 64) return GN_ERR_SHAPE;
    const Range rp = {positions, psize * static_cast<size_t>(tokens * axes)};
    for (int i = 0; i < 2; ++i) {
        a.in[i] = in[i];
        a.out[i] = out[i];
        a.heads[i] = static_cast<int>(count[i]);
        a.in_token[i] = strides[2 * i];
        a.in_head[i] = strides[2 * i + 1];
        a.out_token[i] = strides[4 + 2 * i];
        a.out_head[i] = strides[4 + 2 * i + 1];
        if (!in[i]) continue;
        if (!strided(&ri[i], in[i], tokens, a.in_token[i], count[i], a.in_head[i], dim, size) ||
            !strided(&ro[i], out[i], tokens, a.out_token[i], count[i], a.out_head[i], dim, size))
            return GN_ERR_SHAPE;
        if (collide(tokens, a.out_token[i], count[i], a.out_head[i], dim)) return GN_ERR_SHAPE;
    }
    for (int i = 0; i < 2; ++i) {
        if (!in[i]) continue;
        if (overlap(ro[i], rp)) return GN_ERR_ALIAS;
        const bool place = in[i] == out[i] && a.in_token[i] == a.out_token[i] && a.in_head[i] == a.out_head[i];
        const TokenSlice so = {out[i], a.out_token[i], (count[i] - 1) * a.out_head[i] + dim};
        for (int n = 0; n < 2; ++n) {
            const TokenSlice si = {in[n], a.in_token[n], (count[n] - 1) * a.in_head[n] + dim};
            if (!(place && n == i) && overlap(ro[i], ri[n]) && !side_by_side(so, si, size)) return GN_ERR_ALIAS;
        }
        const TokenSlice other = {out[1 - i], a.out_token[1 - i], (count[1 - i] - 1) * a.out_head[1 - i] + dim};
        if (overlap(ro[i], ro[1 - i]) && !side_by_side(so, other, size)) return GN_ERR_ALIAS;
    }
    DeviceInfo d;
    const int rc = ready(&d);
    if (rc != GN_OK) return rc;
    if (tokens == 0) return GN_OK;
    a.tokens = tokens;
    a.dim = static_cast<int>(dim);
    a.pairs = static_cast<int>(width / 2);
    a.positions = positions;
    a.axes = static_cast<int>(axes);
    a.position_format = position_format;
    a.interleaved = interleaved != 0;
    a.inverse = inverse != 0;
    a.format = format;
    const double log_theta = std::log(theta);
    int p = 0;
    for (int n = 0; n < a.axes; ++n)
        for (int i = 0; i < axes_dim[n] / 2; ++i, ++p) {
            a.axis[p] = static_cast<unsigned char>(n);
            a.turns[p] = std::exp(-log_theta * (2.0 * i / static_cast<double>(axes_dim[n]))) / 6.283185307179586476925;
        }
    const cudaError_t e = gn::launch_rope(a, d.sm_count, static_cast<cudaStream_t>(stream));
    return launched(e, e == cudaSuccess);
}

// ---- attention of packed documents -----------------------------------------------
namespace {

bool apart(int64_t tokens, int64_t token, int heads, int64_t head, int dim)
{
    return (tokens <= 1 || token >= dim) && (heads <= 1 || head >= dim);
}

struct AttnRanges {
    Range q, k, v, out, lse, cu_q, cu_k, prefix, slopes;
};

int check_attn(const gn_attn_packed_args *a, AttnRanges *r)
{
    if (!a) return GN_ERR_NULL;
    if (a->tokens_q != 0 && (!a->q || !a->out || !a->lse)) return GN_ERR_NULL;
    if (a->tokens_k != 0 && (!a->k || !a->v)) return GN_ERR_NULL;
    if (a->format != GN_FORMAT_BF16 && a->format != GN_FORMAT_FP16) return GN_ERR_FORMAT;
    constexpr int64_t most = 1 << 30;
    if (a->tokens_q < 0 || a->tokens_k < 0 || a->tokens_q > most || a->tokens_k > most || a->docs < 1 ||
        a->docs > (1 << 24))
        return GN_ERR_SHAPE;
    if (a->docs > 1 && (!a->cu_q || !a->cu_k)) return GN_ERR_NULL;
    if (a->kv_heads < 1 || a->heads < 1 || a->heads > 1024 || a->heads % a->kv_heads || a->dim < 8 || a->dim > 128 ||
        a->dim % 8)
        return GN_ERR_CHANNELS;
    if (!std::isfinite(a->scale) || !std::isfinite(a->cap) || a->cap < 0.f) return GN_ERR_EPS;
    if (a->prefix && !a->causal) return GN_ERR_VARIANT;
    if (addr(a->q) % 16 || addr(a->k) % 16 || addr(a->v) % 16 || addr(a->out) % 16 || addr(a->lse) % 4 ||
        addr(a->cu_q) % 4 || addr(a->cu_k) % 4 || addr(a->prefix) % 4 || addr(a->slopes) % 4 || a->q_token % 8 ||
        a->q_head % 8 || a->k_token % 8 || a->k_head % 8 || a->v_token % 8 || a->v_head % 8)
        return GN_ERR_ALIGN;
    if (!strided(&r->q, a->q, a->tokens_q, a->q_token, a->heads, a->q_head, a->dim, 2) ||
        !strided(&r->k, a->k, a->tokens_k, a->k_token, a->kv_heads, a->k_head, a->dim, 2) ||
        !strided(&r->v, a->v, a->tokens_k, a->v_token, a->kv_heads, a->v_head, a->dim, 2) ||
        !strided(&r->out, a->out, a->tokens_q, static_cast<int64_t>(a->heads) * a->dim, 1, 0, static_cast<int64_t>(a->heads) * a->dim, 2))
        return GN_ERR_SHAPE;
    // one head's channels of one token must not run into the next one's
    if (!apart(a->tokens_q, a->q_token, a->heads, a->q_head, a->dim) ||
        !apart(a->tokens_k, a->k_token, a->kv_heads, a->k_head, a->dim) ||
        !apart(a->tokens_k, a->v_token, a->kv_heads, a->v_head, a->dim))
        return GN_ERR_SHAPE;
    r->lse = {a->lse, 4u * static_cast<size_t>(a->tokens_q) * static_cast<size_t>(a->heads)};
    r->cu_q = {a->cu_q, 4u * (static_cast<size_t>(a->docs) + 1)};
    r->cu_k = {a->cu_k, 4u * (static_cast<size_t>(a->docs) + 1)};
    r->prefix = {a->prefix, 4u * static_cast<size_t>(a->docs)};
    r->slopes = {a->slopes, 4u * static_cast<size_t>(a->heads)};
    return GN_OK;
}

}  // namespace

int gn_attn_packed(const gn_attn_packed_args *args, void *stream)
{
    AttnRanges r;
    int rc = check_attn(args, &r);
    if (rc != GN_OK) return rc;
    for (const Range &o : {r.out, r.lse})
        for (const Range &i : {r.q, r.k, r.v, r.cu_q, r.cu_k, r.prefix, r.slopes})
            if (overlap(o, i)) return GN_ERR_ALIAS;
    if (overlap(r.out, r.lse)) return GN_ERR_ALIAS;
    DeviceInfo d;
    rc = ready(&d);
    if (rc != GN_OK) return rc;
    if (args->tokens_q == 0) return GN_OK;
    gn::PackedAttn p = {};
    p.a = *args;
    p.group = args->heads / args->kv_heads;
    int launches = 0;
    const cudaError_t e = gn::launch_packed_attn(p, d.sm_count, {wait_timeout_ns(), d.status_word, d.status_host},
                                                 static_cast<cudaStream_t>(stream), &launches);
    return launched(e, launches);
}

size_t gn_attn_packed_workspace_bytes(int64_t tokens_q, int64_t heads)
{
    if (tokens_q < 0 || tokens_q > (1 << 30) || heads < 1 || heads > 1024) return 0;
    return gn::packed_attn_workspace_bytes(tokens_q > 0 ? tokens_q : 1, static_cast<int>(heads));
}

int gn_attn_packed_backward(const gn_attn_packed_args *args, const void *dout, int64_t dout_token, int64_t dout_head,
                            void *dq, void *dk, void *dv, void *workspace, size_t workspace_bytes, void *stream)
{
    AttnRanges r;
    int rc = check_attn(args, &r);
    if (rc != GN_OK) return rc;
    const gn_attn_packed_args &a = *args;
    if (a.tokens_q != 0 && (!dout || !dq || !workspace)) return GN_ERR_NULL;
    if (a.tokens_k != 0 && (!dk || !dv)) return GN_ERR_NULL;
    if (addr(dout) % 16 || addr(dq) % 16 || addr(dk) % 16 || addr(dv) % 16 || addr(workspace) % 256 ||
        dout_token % 8 || dout_head % 8)
        return GN_ERR_ALIGN;
    Range g;
    if (!strided(&g, dout, a.tokens_q, dout_token, a.heads, dout_head, a.dim, 2) ||
        !apart(a.tokens_q, dout_token, a.heads, dout_head, a.dim))
        return GN_ERR_SHAPE;
    const size_t qb = 2u * static_cast<size_t>(a.tokens_q) * static_cast<size_t>(a.heads) * static_cast<size_t>(a.dim);
    const size_t kb = 2u * static_cast<size_t>(a.tokens_k) * static_cast<size_t>(a.kv_heads) * static_cast<size_t>(a.dim);
    const Range outs[] = {{dq, qb}, {dk, kb}, {dv, kb}, {workspace, workspace_bytes}};
    for (int n = 0; n < 4; ++n) {
        for (const Range &i : {r.q, r.k, r.v, r.out, r.lse, r.cu_q, r.cu_k, r.prefix, r.slopes, g})
            if (overlap(outs[n], i)) return GN_ERR_ALIAS;
        for (int m = 0; m < n; ++m)
            if (overlap(outs[n], outs[m])) return GN_ERR_ALIAS;
    }
    if (a.tokens_q != 0 && workspace_bytes < gn_attn_packed_workspace_bytes(a.tokens_q, a.heads)) return GN_ERR_WORKSPACE;
    DeviceInfo d;
    rc = ready(&d);
    if (rc != GN_OK) return rc;
    gn::PackedAttn p = {};
    p.a = a;
    p.group = a.heads / a.kv_heads;
    p.dout = dout;
    p.dout_token = dout_token;
    p.dout_head = dout_head;
    p.dq = dq;
    p.dk = dk;
    p.dv = dv;
    p.workspace = workspace;
    int launches = 0;
    const cudaError_t e = gn::launch_packed_attn_backward(p, d.sm_count, {wait_timeout_ns(), d.status_word, d.status_host},
                                                          static_cast<cudaStream_t>(stream), &launches);
    return launched(e, launches);
}

}  // extern "C"
