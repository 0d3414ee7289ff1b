// The paged 4-bit key/value cache: geometry shared by its kernels.
//
// A page holds P tokens of every kv head; the codes of one (page, kv head) are
// P rows of D/8 words, its scales D/g rows of P floats (tokens contiguous).
// Codes are offset binary (u = q + 8), LSB first.  Inside a row they lie in
// the order in which the attention kernel's matrix operands want them:
//   keys:   dimension 32 i + 8 r + e is code e of word r (D/32) + i
//           (r = 0..3, e = 0..7), so the lanes of one token that hold operand
//           rows of every 32-dimension step read D/32 consecutive words;
//   values: dimension 16 j + c is code c (D/16) + j of the row (c = 0..15), so
//           the codes that a lane turns into D/16 operand rows are consecutive.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dq {

struct Cache4 {
    uint32_t* k_codes;  // [pages, heads, P, D/8]
    uint32_t* v_codes;
    float* k_scales;  // [pages, heads, D/g, P]
    float* v_scales;
    int64_t pages;
    int32_t heads;       // kv heads
    int32_t dim;         // D: 64, 128 or 256
    int32_t page_shift;  // P = 1 << page_shift, 16 .. 256
    int32_t group;       // g: 32, 64 or 128
};

// The sequences of a call: sequence b's new tokens are rows starts[b] ..
// starts[b+1] - 1 of the call's token arrays and the last of its lens[b]
// cached ones; position p lies in page table[b * width + p / P].
struct Cache4Batch {
    const int32_t* starts;  // [count + 1]
    const int32_t* lens;    // [count]
    const int32_t* table;   // [count, width]
    int64_t width;
    int64_t count;
};

// Row range of sequence b, clamped to the call's token rows.
__device__ __forceinline__ void cache4_rows(const Cache4Batch& bt, int64_t b, int64_t tokens,
                                            int64_t& first, int64_t& n)
{
    int64_t s = bt.starts[b], e = bt.starts[b + 1];
    s = s < 0 ? 0 : (s > tokens ? tokens : s);
    e = e < s ? s : (e > tokens ? tokens : e);
    first = s;
    n = e - s;
}

// The sequence of token row t of the call: the last one whose first row is at or
// before t (its rows are [first, first + n); t may lie behind them).
__device__ __forceinline__ int64_t cache4_sequence(const Cache4Batch& bt, int64_t t)
{
    int64_t lo = 0, hi = bt.count;
    while (lo + 1 < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if ((int64_t)bt.starts[mid] <= t)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// page * P + offset of position pos of sequence b, or -1 where the cache does not
// hold it (a position below 0 or past the table, a page outside the cache).
__device__ __forceinline__ int64_t cache4_slot(const Cache4& c, const Cache4Batch& bt, int64_t b, int64_t pos)
{
    if (pos < 0) return -1;
    const int64_t idx = pos >> c.page_shift;
    if (idx >= bt.width) return -1;
    const int64_t page = bt.table[b * bt.width + idx];
    if (page < 0 || page >= c.pages) return -1;
    return (page << c.page_shift) + (pos & ((1LL << c.page_shift) - 1));
}

}  // namespace dq
