// block_checks.h -- checks of arguments that the C entries of the transformer-block
// operators share (block_capi.cu, serve_capi.cu).
#pragma once

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/gnsilu.h"
#include "block_internal.h"
#include "capi_util.h"

namespace gn_block {

using gn_capi::DeviceInfo;
using gn_capi::count_launches;
using gn_capi::current_device;
using gn_capi::ranges_overlap;
using gn_capi::wait_timeout_ns;

constexpr int64_t kMaxElements = INT64_MAX / 16;

inline uintptr_t addr(const void *p) { return reinterpret_cast<uintptr_t>(p); }

inline size_t format_size(int format) { return format == GN_FORMAT_FP32 ? 4 : 2; }

inline bool format_ok(int format) { return format >= GN_FORMAT_BF16 && format <= GN_FORMAT_FP32; }

// A buffer's address range: `n0` steps of stride s0, `n1` of stride s1, then
// `inner` contiguous elements.  False if it overflows.
struct Range {
    const void *p = nullptr;
    size_t bytes = 0;
};

inline bool strided(Range *r, const void *p, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t inner, size_t size)
{
    r->p = p;
    r->bytes = 0;
    if (n0 == 0 || n1 == 0 || !p) return true;
    if (s0 < 0 || s1 < 0) return false;
    if (n0 > 1 && s0 > kMaxElements / n0) return false;
    if (n1 > 1 && s1 > kMaxElements / n1) return false;
    const int64_t last = (n0 - 1) * s0 + (n1 - 1) * s1 + inner;
    if (last > kMaxElements) return false;
    r->bytes = static_cast<size_t>(last) * size;
    return true;
}

inline bool overlap(const Range &a, const Range &b) { return a.p && b.p && ranges_overlap(a.p, a.bytes, b.p, b.bytes); }

// Slices of one buffer (the heads of q and of k in a fused projection): the
// ranges interleave, but token by token the one ends before the other begins.
struct TokenSlice {
    const void *p;
    int64_t token, extent;   // elements from token to token, and used of them
};

inline bool side_by_side(const TokenSlice &a, const TokenSlice &b, size_t size)
{
    if (a.token != b.token) return false;
    const TokenSlice &lo = addr(a.p) <= addr(b.p) ? a : b, &hi = addr(a.p) <= addr(b.p) ? b : a;
    const uintptr_t off = addr(hi.p) - addr(lo.p);
    return off >= static_cast<uintptr_t>(lo.extent) * size &&
           off + static_cast<uintptr_t>(hi.extent) * size <= static_cast<uintptr_t>(lo.token) * size;
}

// Whether some of tokens x heads runs of `dim` elements lie on one another.
inline bool collide(int64_t tokens, int64_t token, int64_t heads, int64_t head, int64_t dim)
{
    if ((tokens > 1 && token < dim) || (heads > 1 && head < dim)) return true;
    if (tokens <= 1 || heads <= 1) return false;
    // heads within tokens, or tokens within heads
    if (token - dim >= (heads - 1) * head || head - dim >= (tokens - 1) * token) return false;
    // some heads further on, and some tokens further back
    for (int64_t h = 1; h < heads; ++h) {
        const int64_t t = h * head / token, left = h * head - t * token;
        if ((t < tokens && left < dim) || (t + 1 < tokens && token - left < dim)) return true;
    }
    return false;
}

// The device's properties, or the status to return.
inline int ready(DeviceInfo *d)
{
    int dev = -1;
    const int rc = current_device(&dev, d);
    if (rc != GN_OK) return rc;
    return gn_capi::kernel_status_raised(dev) ? GN_ERR_KERNEL : GN_OK;
}

inline int launched(cudaError_t e, int launches)
{
    count_launches(static_cast<uint64_t>(launches));
    if (e == cudaSuccess) return GN_OK;
    cudaGetLastError();
    return GN_ERR_CUDA;
}

// Rows in two levels: false if they run into one another or overflow.  Rows that
// are only read may be broadcast (a stride of 0).  A flat tensor's outer stride
// is made to fit.
inline bool norm_rows(Range *r, gn::RowsAt *at, const void *p, int64_t rows, int64_t cols, int64_t inner, const int64_t *strides,
               size_t size, bool read_only)
{
    *at = {strides[0], strides[1]};
    if (at->stride < cols && !(read_only && at->stride == 0)) return false;
    const int64_t in = rows < inner ? rows : inner;
    if (in > 1 && at->stride > kMaxElements / in) return false;
    if (rows <= inner) {
        at->outer = 0;
        return strided(r, p, rows, at->stride, 1, 0, cols, size);
    }
    if (at->outer < (in - 1) * at->stride + cols && !(read_only && at->outer == 0)) return false;
    return strided(r, p, (rows + inner - 1) / inner, at->outer, inner, at->stride, cols, size);
}

inline bool norm_cols_ok(int64_t cols) { return cols >= 1 && cols <= gn::kNormMaxCols; }

}  // namespace gn_block
