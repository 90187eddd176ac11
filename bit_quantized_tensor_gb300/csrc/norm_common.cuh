// Pieces shared by layer norm's forward and backward kernels.
#pragma once
#include "fp4_common.cuh"
#include "qg_ptx.cuh"

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
// registers.  A bulk copy wants whole 16-byte pieces: of a row that starts or
// ends inside one, the few bytes of the edge pieces are copied by threads.
//
// A group of TPR threads (a warp, or the CTA) has a ring of its own.

template <int TPR>
__device__ __forceinline__ void group_sync() {
    if constexpr (TPR == 32)
        __syncwarp();
    else
        __syncthreads();
}

struct RowRing {
    uint32_t bar0;      // mbarriers, one a slot
    uint8_t* slots;     // this group's slots
    int slot_bytes;
    int64_t row_bytes;
};

// Bytes of a slot: a row at any offset inside its first 16-byte piece.
__host__ __device__ inline int64_t row_slot_bytes(int64_t row_bytes) { return (row_bytes + 15 + 15) / 16 * 16; }

// A row in memory cut at 16-byte boundaries.
struct RowPieces {
    uintptr_t start, end, base;  // the row; the 16-byte piece it starts in
    uintptr_t a;                 // first whole piece
    uint32_t whole;              // bytes of whole pieces
};
__device__ __forceinline__ RowPieces row_pieces(const void* row, int64_t bytes) {
    RowPieces q;
    q.start = reinterpret_cast<uintptr_t>(row);
    q.end = q.start + bytes;
    q.base = q.start & ~uintptr_t(15);
    q.a = (q.start + 15) & ~uintptr_t(15);
    const uintptr_t b = q.end & ~uintptr_t(15);
    q.whole = b > q.a ? static_cast<uint32_t>(b - q.a) : 0u;
    return q;
}
// The bytes outside the whole pieces, two a thread (elements are 2 or 4 bytes
// at addresses that are multiples of 2).
__device__ __forceinline__ void row_edges(const RowPieces& q, uint8_t* dst, int t) {
    const uintptr_t head_end = q.whole ? q.a : q.end;
    const uintptr_t h = q.start + 2 * t;
    if (t < 32 && h < head_end)
        *reinterpret_cast<uint16_t*>(dst + (h - q.base)) = *reinterpret_cast<const uint16_t*>(h);
    const uintptr_t e = q.a + q.whole + 2 * t;
    if (q.whole && t < 8 && e < q.end)
        *reinterpret_cast<uint16_t*>(dst + (e - q.base)) = *reinterpret_cast<const uint16_t*>(e);
}

// Starts the copy of a row into slot s.  All threads of the group call it, after
// all of them have read the slot's previous row and synchronized; the edges are
// visible after the group's next synchronization.
template <int TPR>
__device__ __forceinline__ void row_fetch(const RowRing& r, int s, const void* row) {
    const int t = threadIdx.x % TPR;
    uint8_t* dst = r.slots + static_cast<int64_t>(s) * r.slot_bytes;
    const RowPieces q = row_pieces(row, r.row_bytes);
    const uint32_t bar = r.bar0 + 8 * s;
    if (t == 0) {
        mbar_arrive_expect_tx(bar, q.whole);
        if (q.whole) bulk_copy_g2s(smem_u32(dst + (q.a - q.base)), reinterpret_cast<const void*>(q.a), q.whole, bar);
    }
    if ((q.start | q.end) & 15) row_edges(q, dst, t);
}

// The same for two rows of one length that share a slot: x, then y half a slot on.
template <int TPR>
__device__ __forceinline__ void row_fetch2(const RowRing& r, int s, const void* x, const void* y) {
    const int t = threadIdx.x % TPR;
    uint8_t* dx = r.slots + static_cast<int64_t>(s) * r.slot_bytes;
    uint8_t* dy = dx + r.slot_bytes / 2;
    const RowPieces p = row_pieces(x, r.row_bytes), q = row_pieces(y, r.row_bytes);
    const uint32_t bar = r.bar0 + 8 * s;
    if (t == 0) {
        mbar_arrive_expect_tx(bar, p.whole + q.whole);
        if (p.whole) bulk_copy_g2s(smem_u32(dx + (p.a - p.base)), reinterpret_cast<const void*>(p.a), p.whole, bar);
        if (q.whole) bulk_copy_g2s(smem_u32(dy + (q.a - q.base)), reinterpret_cast<const void*>(q.a), q.whole, bar);
    }
    if ((p.start | p.end) & 15) row_edges(p, dx, t);
    if ((q.start | q.end) & 15) row_edges(q, dy, t);
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
// gamma or beta of 8 columns (w 16-byte aligned, k a multiple of 8); `none` without one.
template <class T>
__device__ __forceinline__ void weight_pairs(const void* w, bool f32, int k, float none, uint64_t (&g)[4]) {
    if (!w) {
#pragma unroll
        for (int j = 0; j < 4; ++j) g[j] = two(none, none);
    } else if (f32) {
        load_pairs<float>(static_cast<const float*>(w) + k, g);
    } else {
        load_pairs<T>(static_cast<const T*>(w) + k, g);
    }
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
inline int ring_slots(int64_t slot_bytes, int64_t rings_per_sm, int least) {
    const int64_t n = kRingSmem / (slot_bytes * rings_per_sm);
    return static_cast<int>(n < least ? least : n > kRingMax ? kRingMax : n);
}

inline bool vec_ok(const void* p, int64_t ld, size_t elem, int64_t rows) {
    return aligned16(p) && (rows <= 1 || (static_cast<size_t>(ld) * elem) % 16 == 0);
}

// Argument checks of the norm's calls (qg_norm.cu).
int check_rows(int dtype, int64_t M, int64_t D, const void* X, int64_t ldx);
int check_weight(const void* w, int dtype);
int check_norm(int dtype, int wdtype, int64_t M, int64_t D, float eps);

constexpr int kLongThreads = 1024;  // CTAs of the kernels for rows too long to hold

}  // namespace qg
