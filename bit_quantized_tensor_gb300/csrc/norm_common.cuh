// Pieces shared by layer norm's forward and backward kernels.
#pragma once
#include "fp4_common.cuh"
#include "qg_ptx.cuh"
#include "row_pieces.h"

namespace qg {

// A value of gamma or beta: fp32, or the type T of the rows.
template <class T>
__device__ __forceinline__ float weight_at(const void* w, bool f32, int64_t i) {
    return f32 ? static_cast<const float*>(w)[i] : to_f32<T>(static_cast<const T*>(w)[i]);
}

// 8 values from index i on, i a multiple of 8 and w 16-byte aligned when `vec`.
template <class T>
__device__ __forceinline__ void weights8(const void* w, bool f32, bool vec, int64_t i, int n, float none,
                                         float (&g)[8]) {
    if (!w) {
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = none;
    } else if (f32) {
        load_some<float, 8>(static_cast<const float*>(w) + i, n, vec, g);
    } else {
        load_some<T, 8>(static_cast<const T*>(w) + i, n, vec, g);
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over the TPR threads of a row (the whole CTA where TPR > 32), the same
// value in all of them.  `red` holds one value a warp; two calls in a row use
// two of them, so one barrier a call is enough.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
    v = warp_sum(v);
    if constexpr (TPR > 32) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = warp_sum((threadIdx.x & 31) < TPR / 32 ? red[threadIdx.x & 31] : 0.f);
    }
    return v;
}

// ------------------------------------------------------- rows through shared memory
//
// With many rows the kernels walk over them with a ring of rows in shared
// memory that cp.async.bulk fills some rows ahead, so the loads of the next
// rows are in flight while a row goes through its reductions, at no cost in
// registers.  A bulk copy moves whole 16-byte pieces, so a row that starts or
// ends inside one comes with a few bytes of its neighbours.
//
// A group of TPR threads (a warp, or the CTA) has a ring of its own.

struct RowRing {
    uint32_t bar0;      // mbarriers, one a slot
    uint8_t* slots;     // this group's slots
    int slot_bytes;
    int64_t row_bytes;
};

// Bytes of a slot: a row at any offset inside its first 16-byte piece, readable
// to the end of its last 32 bytes.
__host__ __device__ inline int64_t row_slot_bytes(int64_t row_bytes) { return (row_bytes + 15 + 31) / 32 * 32; }

// The rest of a row at an end of the matrix, two bytes a thread (elements are 2 or 4
// bytes, at addresses that are multiples of 2).  Later bulk copies into the slot
// have to come behind these stores.
__device__ __forceinline__ void row_edges(const RowPieces& q, uint8_t* dst, int t) {
    if (t >= 32) return;
    const uintptr_t h = q.start + 2 * t, e = q.tail() + 2 * t;
    if (h < q.head_end()) *reinterpret_cast<uint16_t*>(dst + (h - q.base)) = *reinterpret_cast<const uint16_t*>(h);
    if (e < q.end) *reinterpret_cast<uint16_t*>(dst + (e - q.base)) = *reinterpret_cast<const uint16_t*>(e);
    fence_proxy_async_smem();
}

__device__ __forceinline__ void row_copy(const RowPieces& q, uint8_t* dst, uint32_t bar) {
    if (q.bytes) bulk_copy_g2s(smem_u32(dst + (q.a - q.base)), reinterpret_cast<const void*>(q.a), q.bytes, bar);
}

// Starts the copy of row i of the matrix m into slot s.  All threads of the group
// call it, after all of them have read the slot's previous row and synchronized;
// what row_edges copies is visible after the group's next synchronization.
// EDGES: rows may start or end inside a piece.
template <int TPR, bool EDGES>
__device__ __forceinline__ void row_fetch(const RowRing& r, int s, const void* row, int64_t i, const RowBounds& m) {
    const int t = threadIdx.x % TPR;
    const bool at_end = EDGES && m.at_end(i);
    if (t && !at_end) return;
    uint8_t* dst = r.slots + static_cast<int64_t>(s) * r.slot_bytes;
    const RowPieces q = row_pieces(reinterpret_cast<uintptr_t>(row), r.row_bytes, m, at_end);
    const uint32_t bar = r.bar0 + 8 * s;
    if (t == 0) {
        mbar_arrive_expect_tx(bar, q.bytes);
        row_copy(q, dst, bar);
    }
    if (at_end) row_edges(q, dst, t);
}

// The same for two rows of one length that share a slot: x, then y half a slot on;
// at_end: either row is at an end of its matrix.
template <int TPR>
__device__ __forceinline__ void row_fetch2(const RowRing& r, int s, const void* x, const void* y, bool at_end,
                                           const RowBounds& mx, const RowBounds& my) {
    const int t = threadIdx.x % TPR;
    uint8_t* dx = r.slots + static_cast<int64_t>(s) * r.slot_bytes;
    uint8_t* dy = dx + r.slot_bytes / 2;
    const uint32_t bar = r.bar0 + 8 * s;
    auto copy = [&](const RowPieces& p, const RowPieces& q) {
        if (t == 0) {
            mbar_arrive_expect_tx(bar, p.bytes + q.bytes);
            row_copy(p, dx, bar);
            row_copy(q, dy, bar);
        }
    };
    const uintptr_t ax = reinterpret_cast<uintptr_t>(x), ay = reinterpret_cast<uintptr_t>(y);
    if (!at_end) {
        if (t == 0) copy(row_pieces(ax, r.row_bytes, mx, false), row_pieces(ay, r.row_bytes, my, false));
    } else {
        const RowPieces p = row_pieces(ax, r.row_bytes, mx, true), q = row_pieces(ay, r.row_bytes, my, true);
        copy(p, q);
        row_edges(p, dx, t);
        row_edges(q, dy, t);
    }
}

template <class T>
__device__ __forceinline__ const T* row_in_slot(const RowRing& r, int s, const void* row) {
    return reinterpret_cast<const T*>(r.slots + static_cast<int64_t>(s) * r.slot_bytes +
                                      (reinterpret_cast<uintptr_t>(row) & 15));
}

// Pairs of fp32 values in one 64-bit register: two results an instruction.
__device__ __forceinline__ uint64_t two(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float2 both(uint64_t v) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}
__device__ __forceinline__ uint64_t add_two(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul_two(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma_two(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// 8 values at a 16-byte aligned address as four pairs, and back.
template <class T>
__device__ __forceinline__ void load_pairs(const T* p, uint64_t (&v)[4]) {
    float x[8];
    load_vec<T, 8>(p, x);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = two(x[2 * j], x[2 * j + 1]);
}
template <class T>
__device__ __forceinline__ void store_pairs(T* p, const uint64_t (&v)[4]) {
    float x[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = both(v[j]);
        x[2 * j] = f.x;
        x[2 * j + 1] = f.y;
    }
    store_vec<T, 8>(p, x);
}
// The rows of a group may start inside a 16-byte piece, but all at the same
// place (`lead` values into it): its columns then come in aligned pieces of 8
// that begin at column -lead.  Pieces that reach outside [0, D) are cut.
__device__ __forceinline__ bool piece_cut(int k, int D) { return k < 0 || k + 8 > D; }
__device__ __forceinline__ void cut_piece(uint64_t (&v)[4], int k, int D) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = both(v[j]);
        const int a = k + 2 * j;
        v[j] = two(a >= 0 && a < D ? f.x : 0.f, a + 1 >= 0 && a + 1 < D ? f.y : 0.f);
    }
}
// What is left of a piece, as a mask on its words in memory; at most the first
// and the last piece of a row are cut, so a thread keeps one mask for each.
template <class T>
struct PieceMask {
    uint32_t w[2 * sizeof(T)];
};
template <class T>
__device__ __forceinline__ PieceMask<T> piece_mask(int k, int D) {
    PieceMask<T> m;
    auto in = [&](int j) { return k + j >= 0 && k + j < D; };
#pragma unroll
    for (int i = 0; i < 2 * static_cast<int>(sizeof(T)); ++i) {
        if constexpr (sizeof(T) == 4)
            m.w[i] = in(i) ? 0xffffffffu : 0u;
        else
            m.w[i] = (in(2 * i) ? 0xffffu : 0u) | (in(2 * i + 1) ? 0xffff0000u : 0u);
    }
    return m;
}
template <class T>
__device__ __forceinline__ void load_piece(const T* p, uint64_t (&v)[4], const PieceMask<T>& a, bool use_a,
                                           const PieceMask<T>& b, bool use_b) {
    constexpr int W = 2 * static_cast<int>(sizeof(T));
    uint32_t w[W];
#pragma unroll
    for (int i = 0; i < W; i += 4) {
        const uint4 q = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(p) + i);
        w[i] = q.x; w[i + 1] = q.y; w[i + 2] = q.z; w[i + 3] = q.w;
    }
    if (use_a) {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] &= a.w[i];
    }
    if (use_b) {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] &= b.w[i];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4) {
            v[j] = two(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
        } else {
            const float2 f = unpack2<T>(w[j]);
            v[j] = two(f.x, f.y);
        }
    }
}
// To memory: whole where p is the start of a 16-byte piece, else one by one.
template <class T>
__device__ __forceinline__ void store_piece(T* row, int k, int D, bool whole, const uint64_t (&v)[4]) {
    if (whole && !piece_cut(k, D)) {
        store_pairs<T>(row + k, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 f = both(v[j / 2]);
            if (k + j >= 0 && k + j < D) row[k + j] = from_f32<T>(j & 1 ? f.y : f.x);
        }
    }
}
// gamma or beta of a piece, 0 outside [0, D), `none` without one; vec: w is 16-byte
// aligned (then whole pieces from a multiple of 8 on come in one or two loads).
template <class T>
__device__ __forceinline__ void weight_piece(const void* w, bool f32, bool vec, int k, int D, float none,
                                             uint64_t (&g)[4]) {
    float f[8];
    if (vec && (k & 7) == 0 && !piece_cut(k, D)) {
        weights8<T>(w, f32, true, k, 8, none, f);
#pragma unroll
        for (int j = 0; j < 4; ++j) g[j] = two(f[2 * j], f[2 * j + 1]);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        f[j] = k + j < 0 || k + j >= D ? 0.f : w ? weight_at<T>(w, f32, k + j) : none;
#pragma unroll
    for (int j = 0; j < 4; ++j) g[j] = two(f[2 * j], f[2 * j + 1]);
}

// gamma or beta as fp32 in shared memory, for rows that are not read in pieces.
template <class T>
__device__ __forceinline__ void stage_weights(float* dst, const void* w, bool f32, int D, float none) {
    for (int k = threadIdx.x; k < D; k += blockDim.x) dst[k] = w ? weight_at<T>(w, f32, k) : none;
}

constexpr int kRingMax = 8;  // slots of a ring, at most
constexpr int kSiteNormRow = 401;

// Shared memory that the rings of an SM's CTAs may fill; the rest of the 256 KB
// that an SM has for shared memory and L1 keeps gamma and beta near.
constexpr int64_t kRingSmem = 160 * 1024;

// Slots of a ring: as many as an SM's share holds, `least` at least.
inline int ring_slots(int64_t slot_bytes, int64_t rings_per_sm, int least, int64_t smem = kRingSmem) {
    const int64_t n = smem / (slot_bytes * rings_per_sm);
    return static_cast<int>(n < least ? least : n > kRingMax ? kRingMax : n);
}

inline bool vec_ok(const void* p, int64_t ld, size_t elem, int64_t rows) {
    return aligned16(p) && (rows <= 1 || (static_cast<size_t>(ld) * elem) % 16 == 0);
}

// Rows a step must be a multiple of for all rows of a group to start at the same
// place inside a 16-byte piece.
inline int64_t same_place_rows(int64_t ld, size_t elem) {
    int64_t n = 1;
    while ((static_cast<size_t>(ld) * elem * static_cast<size_t>(n)) % 16 != 0) n *= 2;
    return n;  // at most 8: elements are 2 or 4 bytes
}

// CTAs to launch for M rows, at most `most`: with more rows than groups, rounded
// down so that a group's rows lie a multiple of `same` apart (0: cannot be).
inline int64_t norm_ctas(int64_t M, int64_t groups, int64_t most, int64_t same) {
    const int64_t want = (M + groups - 1) / groups;
    if (want <= most) return want;
    int64_t n = most;
    while (n > 0 && n * groups % same != 0) --n;
    return n;
}

// Argument checks of the norm's calls (qg_norm.cu).
int check_rows(int dtype, int64_t M, int64_t D, const void* X, int64_t ldx);
int check_weight(const void* w, int dtype);
int check_f32(const float* v);
int check_norm(int dtype, int wdtype, int64_t M, int64_t D, float eps);

constexpr int kLongThreads = 1024;  // CTAs of the kernels for rows too long to hold

}  // namespace qg
