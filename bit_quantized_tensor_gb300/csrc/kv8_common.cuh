// A paged cache of keys and values in 8-bit codes, and the batch that works on it.
//
//   codes   pages x heads x page x D bytes, a scale (fp32) for each page and head
//   table   B x table_cols page numbers: token j of sequence b is token j % page of
//           page table[b][j / page]
//   starts  B + 1 row numbers: sequence b's new tokens (or queries) are rows
//           starts[b] .. starts[b + 1]
//   lengths B: tokens of the sequence; the rows above are its last ones
// A page's scale is s = max(fl(amax / 127), 2^-64) over its tokens, or NaN once one of
// its values was not finite; codes as in s8_common.cuh.
//
// starts, lengths and the table live on the device, so nothing about them is known
// when a kernel is launched: rows of a sequence that leave [0, rows) or run backwards
// are no rows, tokens ahead of the first do not exist, and a page number outside the
// cache (or a token behind the table) reads as NaN and is not written.
#pragma once
#include "s8_common.cuh"

namespace qg {

constexpr float kPageScaleFloor = 0x1p-64f;

struct Kv8Cache {
    int8_t *kq, *vq;
    float *ks, *vs;
    const int32_t* table;
    int table_cols, pages;
    int heads, page_log2, D;
};
struct Kv8Batch {
    const int32_t *starts, *lengths;
    int B, rows;
};

struct Kv8Seq {
    int row0, n;       // its rows
    int len;           // tokens the table has room for, at most
    int64_t first;     // position of its first row's token; negative: it does not exist
    bool cut;          // more tokens than the table has room for
};
__device__ __forceinline__ Kv8Seq kv8_seq(const Kv8Batch& bt, const Kv8Cache& c, int b) {
    Kv8Seq s;
    const int r0 = bt.starts[b], r1 = bt.starts[b + 1], len = bt.lengths[b];
    const bool ok = r0 >= 0 && r1 >= r0 && r1 <= bt.rows;
    s.row0 = ok ? r0 : 0;
    s.n = ok ? r1 - r0 : 0;
    const int64_t room = static_cast<int64_t>(c.table_cols) << c.page_log2;
    s.first = static_cast<int64_t>(len) - s.n;
    s.cut = len > room;
    s.len = len < 0 ? 0 : s.cut ? static_cast<int>(room) : len;
    return s;
}

// Page of a sequence's `i`-th, -1 if there is none.
__device__ __forceinline__ int kv8_page(const Kv8Cache& c, int b, int i) {
    if (i < 0 || i >= c.table_cols) return -1;
    const int page = c.table[static_cast<int64_t>(b) * c.table_cols + i];
    return page >= 0 && page < c.pages ? page : -1;
}

// Which sequence item `u` falls to, when sequence b has count(b) items: its number and
// the item's place in it; b = B if there are fewer items.  All THREADS threads of the
// CTA call it; `mem` holds THREADS / 32 + 2 64-bit words.  Each thread adds up the counts
// of a run of sequences, so a batch costs a few dependent loads and not one for each.
struct Kv8Place {
    int b;
    int64_t at, total;
};
template <int THREADS, class COUNT>
__device__ __forceinline__ Kv8Place kv8_find(int B, int64_t u_num, int64_t u_den, int64_t* mem, COUNT&& count) {
    constexpr int WARPS = THREADS / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int run = (B + THREADS - 1) / THREADS, b0 = threadIdx.x * run, b1 = min(B, b0 + run);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += count(b);
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    __syncthreads();  // `mem` may still be read from an earlier call
    if (lane == 31) mem[warp] = upto;
    __syncthreads();
    int64_t total = 0, before = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        before = w == warp ? total : before;
        total += mem[w];
    }
    upto += before;
    // item u_num of u_den equal parts of all items, or item u_num itself (u_den = 0)
    const int64_t u = u_den ? total * u_num / u_den : u_num;
    if (threadIdx.x == 0 && u >= total) mem[WARPS] = B, mem[WARPS + 1] = 0;
    if (u < upto && u >= upto - mine) {
        int64_t at = u - (upto - mine);
        int b = b0;
        for (;; ++b) {
            const int64_t n = count(b);
            if (at < n) break;
            at -= n;
        }
        mem[WARPS] = b;
        mem[WARPS + 1] = at;
    }
    __syncthreads();
    return {static_cast<int>(mem[WARPS]), mem[WARPS + 1], total};
}

}  // namespace qg
