// Which bytes of a matrix's row a bulk copy may fetch: plain arithmetic on
// addresses, for host and device.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define QG_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define QG_HOST_DEVICE inline
#endif

namespace qg {

// The whole 16-byte pieces inside a matrix, [lo, hi), and how many rows at each of
// its ends may reach out of them (one, but up to eight if rows are shorter than a
// piece): row i starts i ld_bytes behind the matrix, and only one that starts
// less than a piece behind it can start ahead of lo.
struct RowBounds {
    uintptr_t lo, hi;
    int64_t near, far;  // rows from 0 to near, and from far on
    QG_HOST_DEVICE bool at_end(int64_t i) const { return i < near || i >= far; }
};
inline RowBounds row_bounds(const void* matrix, int64_t rows, int64_t ld_bytes, int64_t row_bytes) {
    const uintptr_t start = reinterpret_cast<uintptr_t>(matrix);
    RowBounds b;
    b.lo = (start + 15) & ~uintptr_t(15);
    b.hi = (start + (rows > 0 ? static_cast<uintptr_t>((rows - 1) * ld_bytes + row_bytes) : 0)) & ~uintptr_t(15);
    b.near = ld_bytes > 0 && ld_bytes < 16 ? (15 + ld_bytes) / ld_bytes : 1;
    b.far = rows - b.near;
    return b;
}

// The 16-byte pieces that a bulk copy fetches for a row: all that it touches, but
// none that begins ahead of the matrix or ends behind it (memory there need not be
// the caller's).  What that leaves of the row, [start, head_end) and [tail, end), is
// copied by hand: at most two pieces of a row at an end of the matrix.
struct RowPieces {
    uintptr_t start, end, base;  // the row; the piece it starts in
    uintptr_t a;                 // first piece fetched
    uint32_t bytes;              // of pieces fetched
    QG_HOST_DEVICE uintptr_t head_end() const { return bytes ? a : end; }
    QG_HOST_DEVICE uintptr_t tail() const { return bytes ? a + bytes : end; }
};
QG_HOST_DEVICE RowPieces row_pieces(uintptr_t row, int64_t row_bytes, const RowBounds& m, bool at_end) {
    RowPieces q;
    q.start = row;
    q.end = row + static_cast<uintptr_t>(row_bytes);
    q.base = q.start & ~uintptr_t(15);
    q.a = q.base;
    uintptr_t b = (q.end + 15) & ~uintptr_t(15);
    if (at_end) {
        if (q.a < m.lo) q.a = m.lo;
        if (b > m.hi) b = m.hi;
    }
    q.bytes = b > q.a ? static_cast<uint32_t>(b - q.a) : 0u;
    return q;
}

}  // namespace qg
