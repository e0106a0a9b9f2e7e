// cache_common.cuh -- what the kernels of the paged cache share: the sequences'
// runs of packed tokens and where a run's pieces are found from a block's number.
#pragma once

#include <cstdint>

#include "block_internal.h"

namespace gn {
namespace cache {

__host__ __device__ __forceinline__ int read(const int32_t *p)
{
#ifdef __CUDA_ARCH__
    return __ldg(p);
#else
    return *p;
#endif
}

// Sequence n of the call: its packed tokens [begin, end), its length, by which its tokens
// have their places, and how much of it the table has room for.  With `cu`, n = -1 and n = sequences are the tokens ahead of the first
// sequence and behind the last: they have no cache (length 0).
struct Sequence {
    int begin, end, length, held;
    __host__ __device__ __forceinline__ int first_place() const { return length - (end - begin); }
};

__host__ __device__ __forceinline__ Sequence sequence_of(const gn_cache &c, int64_t tokens, int n)
{
    const int t = static_cast<int>(tokens);
    Sequence s;
    const bool real = n >= 0 && n < c.sequences;
    if (c.cu) {
        s.begin = n < 0 ? 0 : min(max(read(c.cu + min(n, c.sequences)), 0), t);
        s.end = n >= c.sequences ? t : min(max(read(c.cu + n + 1), s.begin), t);
    } else {
        const int each = t / c.sequences;
        s.begin = n * each;
        s.end = s.begin + each;
    }
    s.length = real ? min(max(read(c.lengths + n), 0), 1 << 30) : 0;
    s.held = min(s.length, static_cast<int>(c.table_width) * c.page_size);
    return s;
}

// The page of a place, or -1.
__device__ __forceinline__ int page_of(const gn_cache &c, int n, int page)
{
    if (n < 0 || n >= c.sequences || page < 0 || page >= c.table_width) return -1;
    const int p = __ldg(c.table + static_cast<int64_t>(n) * c.table_width + page);
    return p >= 0 && p < c.pages ? p : -1;
}

// Where a run of at most floor(n / step) + more pieces of each sequence (n its packed
// tokens) is found from a block's number: sequence n's pieces begin at floor(begin /
// step) + more (n + 1), which leaves room for that many whatever the runs are, and
// needs one look-up to be known.  (The sequences with n = -1 and n = sequences count.)
__device__ __forceinline__ int64_t first_piece(const gn_cache &c, int64_t tokens, int n, int step, int more)
{
    const int begin = n < 0 ? 0 : min(max(__ldg(c.cu + n), 0), static_cast<int>(tokens));
    return begin / step + static_cast<int64_t>(more) * (n + 1);
}

// The sequence that piece u falls to, for a whole warp: 32 look-ups at a time.
__device__ __forceinline__ int sequence_of_piece(const gn_cache &c, int64_t tokens, int64_t u, int step, int more, int lane)
{
    int low = -1, count = c.sequences + 2;      // among low .. low + count - 1
    while (count > 1) {
        const int each = (count + 31) / 32, n = low + lane * each;
        const bool in = lane * each < count && first_piece(c, tokens, n, step, more) <= u;
        const int take = max(__popc(__ballot_sync(0xffffffffu, in)) - 1, 0);
        low += take * each;
        count = min(each, count - take * each);
    }
    return low;
}

}  // namespace cache
}  // namespace gn
