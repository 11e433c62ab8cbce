// Device helpers of the paged MXFP4 key/value cache, shared by the write and
// read kernels (kq_cache.hip) and the attention (kq_attention.hip): where the
// rows of a batch lie in the cache.
//
// A batch is the page table [seqs, width], row_start [seqs + 1] and lengths
// [seqs], all int32 in device memory, so their values are only known here:
// nothing below trusts them.  A sequence whose rows do not lie inside [0,
// rows) in order has none, a position outside [0, width * page_size) has no
// slot, and neither has a page number outside [0, pages).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/kroquant.h"

namespace kq {

// Largest s of [0, S) with key(s) <= t for a non-decreasing key (0 if there
// is none): the 64 lanes of a wave probe 64 places at a time, so up to 64
// sequences take one round of loads and up to 4096 two.  All lanes of the
// wave take part; t is the same in all of them.
template <class Key>
__device__ __forceinline__ int wave_search(int S, int64_t t, int lane, Key key)
{
    int lo = 0, n = S;
    while (n > 1) {
        const int step = (n + 63) / 64;
        const int i = lane * step;
        const bool le = i < n && key(lo + i) <= t;
        int hits = __popcll(__builtin_amdgcn_ballot_w64(le));
        hits = hits < 1 ? 1 : hits;
        lo += (hits - 1) * step;
        n -= (hits - 1) * step;
        n = n < step ? n : step;
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// Rows [first, first + rows) of the batch belong to the sequence; the i-th
// is position pos0 + i.  (A negative length is taken as 0: either way every
// position is negative, and positions then fit 32 bits.)
struct SeqRows {
    int first, rows;
    int64_t pos0;
};

__device__ __forceinline__ SeqRows seq_rows(const mx_batch &b, int s)
{
    const int64_t a = b.row_start[s], e = b.row_start[s + 1];
    SeqRows r;
    const bool ok = a >= 0 && a < e && e <= b.rows;
    r.first = ok ? (int)a : 0;
    r.rows = ok ? (int)(e - a) : 0;
    const int length = b.lengths[s];
    r.pos0 = (int64_t)(length < 0 ? 0 : length) - (e - a);
    return r;
}

// Slot of position p of sequence s: page * page_size + offset, or -1.
__device__ __forceinline__ int64_t cache_slot(const mx_cache &c, const mx_batch &b, int s, int64_t p)
{
    const int size = (int)c.page_size;
    if (p < 0 || p >= b.width * size)
        return -1;
    const int at = (int)p / size, off = (int)p - at * size;
    const int page = b.page_table[(int64_t)s * b.width + at];
    return page < 0 || page >= c.pages ? -1 : (int64_t)page * size + off;
}

} // namespace kq
