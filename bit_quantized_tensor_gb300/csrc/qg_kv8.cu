// New tokens into the paged 8-bit cache (kv8_common.cuh), and tokens of it back.
#include "kv8_common.cuh"
#include "kv8_host.h"

namespace qg {

// ------------------------------------------------------------ append
//
// A warp takes a page that new tokens go to, for one head and K or V: the largest
// magnitude of the page's new values, the page's new scale, its older codes rounded to
// that scale if it grew, and the new codes.  Only the first page of a sequence's new
// tokens can hold older ones; a page is started afresh with its token 0.  The warps of a
// CTA share the page, which takes three dependent loads to find.  Measured, with the read of the same
// pages behind it: one token each for 64 sequences (8 heads of 128 values) 10.8 us, 1333 tokens of 7
// sequences 10.7; latency of two kernels of four or five dependent loads each.  Where bytes count the loads
// in flight are too few: 4096 tokens of 8 sequences (8 heads of 128 values, pages of 64) 68 us, 3.0 TB/s.
constexpr int kAppendThreads = 256, kAppendWarps = kAppendThreads / 32;
constexpr int kAppendHeld = 4;  // pieces of 8 values that a lane keeps between the two passes

struct AppendParams {
    Kv8Cache c;
    Kv8Batch bt;
    const void *K, *V;
    int64_t ldk, ldv;
    bool k_aligned, v_aligned;
};

template <class T>
__global__ void __launch_bounds__(kAppendThreads) k_kv8_append(const AppendParams p) {
    __shared__ int64_t mem[kAppendThreads / 32 + 2];
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const Kv8Cache& c = p.c;
    const int page_log2 = c.page_log2, page = 1 << page_log2;
    // positions of a sequence's new tokens that exist
    auto range = [&](const Kv8Seq& s, int64_t& lo, int64_t& hi) {
        lo = s.first < 0 ? 0 : s.first;
        hi = s.len;
    };
    const Kv8Place at = kv8_find<kAppendThreads>(p.bt.B, blockIdx.x, 0, mem, [&](int b) -> int64_t {
        const Kv8Seq s = kv8_seq(p.bt, c, b);
        int64_t lo, hi;
        range(s, lo, hi);
        return s.n && hi > lo ? ((hi + page - 1) >> page_log2) - (lo >> page_log2) : 0;
    });
    if (at.b >= p.bt.B) return;
    const Kv8Seq s = kv8_seq(p.bt, c, at.b);
    int64_t lo, hi;
    range(s, lo, hi);
    const int64_t which = (lo >> page_log2) + at.at;
    const int64_t start = which << page_log2;
    lo = lo > start ? lo : start;
    hi = hi < start + page ? hi : start + page;
    const int number = kv8_page(c, at.b, static_cast<int>(which));
    if (number < 0) return;
    const int kept = static_cast<int>(lo - start), count = static_cast<int>(hi - lo);
    const int lane = threadIdx.x & 31;
    const int log_d8 = 31 - __clz(c.D) - 3, pieces = count << log_d8;  // D is 64, 128 or 256

    const int job = blockIdx.y * kAppendWarps + (threadIdx.x >> 5);
    if (job >= 2 * c.heads) return;
    const int head = job >> 1;
    const bool value = job & 1;
    const bool aligned = value ? p.v_aligned : p.k_aligned;
    const int64_t ld = value ? p.ldv : p.ldk;
    const T* x = static_cast<const T*>(value ? p.V : p.K) + (s.row0 + (lo - s.first)) * ld + head * c.D;
    const int64_t unit = static_cast<int64_t>(number) * c.heads + head;
    int8_t* codes = (value ? c.vq : c.kq) + unit * page * c.D;
    float* scale = (value ? c.vs : c.ks) + unit;
    const float old = kept ? *scale : 0.f;
    auto piece = [&](int i, S8Piece<T>& v) {
        v.load(x + (i >> log_d8) * ld + 8 * (i & ((1 << log_d8) - 1)), 8, aligned);
    };

    S8Piece<T> held[kAppendHeld];
    uint32_t amax = 0;
#pragma unroll
    for (int k = 0; k < kAppendHeld; ++k)
        if (lane + 32 * k < pieces) piece(lane + 32 * k, held[k]);
#pragma unroll
    for (int k = 0; k < kAppendHeld; ++k)
        if (lane + 32 * k < pieces) amax = held[k].largest(amax);
#pragma unroll 4
    for (int i = lane + 32 * kAppendHeld; i < pieces; i += 32) {
        S8Piece<T> v;
        piece(i, v);
        amax = v.largest(amax);
    }
    amax = S8Piece<T>::bits(amax);
    amax = warp_max_u32(amax);
    float now = s8_scale(amax, kPageScaleFloor);
    if (kept && (old > now || old != old)) now = old;
    const float r = s8_inverse(now);
    if (kept && old != now) {  // also where one of them is NaN: 0 then
        const float ratio = __fdiv_rn(old, now);
        for (int i = lane; i < kept * c.D / 16; i += 32) {
            uint4 w = reinterpret_cast<uint4*>(codes)[i];
            uint32_t* q = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                int v[4];
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    v[m] = __float2int_rn(__fmul_rn(static_cast<float>(static_cast<int8_t>(q[k] >> (8 * m))), ratio));
                q[k] = pack_s8(v[0], v[1], v[2], v[3]);
            }
            reinterpret_cast<uint4*>(codes)[i] = w;
        }
    }
    int8_t* to = codes + kept * c.D;
    auto store = [&](int i, const S8Piece<T>& v) {
        float f[8];
        v.values(f);
        *reinterpret_cast<uint2*>(to + i * 8) = make_uint2(s8_pack(f, r), s8_pack(f + 4, r));
    };
#pragma unroll
    for (int k = 0; k < kAppendHeld; ++k)
        if (lane + 32 * k < pieces) store(lane + 32 * k, held[k]);
#pragma unroll 4
    for (int i = lane + 32 * kAppendHeld; i < pieces; i += 32) {
        S8Piece<T> v;
        piece(i, v);
        store(i, v);
    }
    if (lane == 0) *scale = now;
}

// ------------------------------------------------------------ gather

struct GatherParams {
    Kv8Cache c;
    Kv8Batch bt;
    void *K, *V;
    int64_t ldk, ldv;
    bool k_aligned, v_aligned;
};

// A CTA takes kGatherRows rows one after another, a warp a row at a time: its token's codes
// of all heads, 16 a lane.  The CTA finds its first row's sequence, a warp goes on from there.
// Measured: 4096 tokens of 8 sequences (8 heads of 128 values) 49 us, 4.1 TB/s.
constexpr int kGatherThreads = 256, kGatherWarps = kGatherThreads / 32;
constexpr int kGatherRows = 16;

template <class T>
__global__ void __launch_bounds__(kGatherThreads) k_kv8_gather(const GatherParams p) {
    __shared__ int64_t mem[kGatherThreads / 32 + 2];
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const Kv8Cache& c = p.c;
    // rows are counted among the sequences that have any
    const Kv8Place at = kv8_find<kGatherThreads>(p.bt.B, static_cast<int64_t>(blockIdx.x) * kGatherRows, 0, mem,
                                                 [&](int b) -> int64_t { return kv8_seq(p.bt, c, b).n; });
    if (at.b >= p.bt.B) return;
    const int lane = threadIdx.x & 31;
    const int per = c.D / 16, pieces = c.heads * per, page = 1 << c.page_log2;
    int b = at.b;
    int64_t i = at.at + (threadIdx.x >> 5);  // place in sequence b
    Kv8Seq s = kv8_seq(p.bt, c, b);
    for (int k = threadIdx.x >> 5; k < kGatherRows; k += kGatherWarps, i += kGatherWarps) {
        while (i >= s.n) {
            i -= s.n;
            if (++b >= p.bt.B) return;
            s = kv8_seq(p.bt, c, b);
        }
        const int64_t row = s.row0 + i, pos = s.first + i;
        const int number = pos < 0 || pos >= s.len ? -1 : kv8_page(c, b, static_cast<int>(pos >> c.page_log2));
        const int offset = static_cast<int>(pos & (page - 1));
#pragma unroll 2
        for (int j = lane; j < 2 * pieces; j += 32) {
            const bool value = j >= pieces;
            const int at_piece = value ? j - pieces : j, head = at_piece / per, d = at_piece % per * 16;
            uint4 w = make_uint4(0, 0, 0, 0);
            float scale = __uint_as_float(0x7fc00000u);
            if (number >= 0) {
                const int64_t unit = static_cast<int64_t>(number) * c.heads + head;
                w = *reinterpret_cast<const uint4*>((value ? c.vq : c.kq) + (unit * page + offset) * c.D + d);
                scale = (value ? c.vs : c.ks)[unit];
            }
            float f[16];
            const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int m = 0; m < 16; ++m) f[m] = static_cast<float>(static_cast<int8_t>(q[m / 4] >> (8 * (m % 4)))) * scale;
            T* to = static_cast<T*>(value ? p.V : p.K) + row * (value ? p.ldv : p.ldk) + head * c.D + d;
            store_some<T, 16>(to, 16, value ? p.v_aligned : p.k_aligned, f);
        }
    }
}

// ------------------------------------------------------------ checks

int check_kv8(const Kv8Args& a) {
    if (a.B < 0 || a.rows < 0 || a.pages < 0 || a.heads < 1 || a.table_cols < 0 || a.page < 1 || a.D < 1)
        return QG_ERR_INVALID_ARG;
    if (a.page != 16 && a.page != 32 && a.page != 64 && a.page != 128) return QG_ERR_UNSUPPORTED;
    if (a.D != 64 && a.D != 128 && a.D != 256) return QG_ERR_UNSUPPORTED;
    if (a.heads > 1024 || a.B > (1 << 20) || a.rows > (1 << 27) || a.pages > (int64_t(1) << 30) ||
        a.table_cols * a.page > (int64_t(1) << 30) || a.pages * a.heads > INT32_MAX)
        return QG_ERR_INVALID_ARG;
    if (a.B == 0 || a.rows == 0) return QG_OK;
    if (!a.kq || !a.vq || !a.ks || !a.vs || !a.table || !a.starts || !a.lengths || a.pages < 1 || a.table_cols < 1)
        return QG_ERR_INVALID_ARG;
    auto word = [](const void* q) { return reinterpret_cast<uintptr_t>(q) % 4 == 0; };
    if (!aligned16(a.kq) || !aligned16(a.vq) || !word(a.ks) || !word(a.vs) || !word(a.table) || !word(a.starts) ||
        !word(a.lengths))
        return QG_ERR_MISALIGNED;
    return QG_OK;
}

void kv8_params(const Kv8Args& a, Kv8Cache* c, Kv8Batch* bt) {
    *c = {};
    c->kq = a.kq; c->vq = a.vq; c->ks = a.ks; c->vs = a.vs; c->table = a.table;
    c->table_cols = static_cast<int>(a.table_cols); c->pages = static_cast<int>(a.pages);
    c->heads = static_cast<int>(a.heads); c->D = static_cast<int>(a.D);
    while ((1 << c->page_log2) < a.page) ++c->page_log2;
    *bt = {a.starts, a.lengths, static_cast<int>(a.B), static_cast<int>(a.rows)};
}

int check_kv8_rows(int dtype, const void* X, int64_t ld, int64_t values, int64_t rows) {
    if (!X || (rows > 1 && ld < values)) return QG_ERR_INVALID_ARG;
    return reinterpret_cast<uintptr_t>(X) % dtype_bytes(dtype) ? QG_ERR_MISALIGNED : QG_OK;
}

static bool rows_aligned(int dtype, const void* X, int64_t ld) {
    return aligned16(X) && ld * static_cast<int64_t>(dtype_bytes(dtype)) % 16 == 0;
}

#define QG_KV8_BUDGETS(T, NAME)                                                                                      \
    QG_BLOCK_KERNEL_BUDGET("k_kv8_append<" NAME ">", reinterpret_cast<const void*>(k_kv8_append<T>), kAppendThreads, 0, \
                           0, 1, 4);                                                                                \
    QG_BLOCK_KERNEL_BUDGET("k_kv8_gather<" NAME ">", reinterpret_cast<const void*>(k_kv8_gather<T>), kGatherThreads, 0, \
                           0, 1, 2)
QG_KV8_BUDGETS(__half, "f16");
QG_KV8_BUDGETS(__nv_bfloat16, "bf16");
QG_KV8_BUDGETS(float, "f32");

}  // namespace qg

using namespace qg;

extern "C" {

int kv8_append(int dtype, int64_t B, int64_t rows, int64_t heads, int64_t D, const void* K, int64_t ldk, const void* V,
               int64_t ldv, int8_t* kq, int8_t* vq, float* ks, float* vs, int64_t pages, int64_t page,
               const int32_t* table, int64_t table_cols, const int32_t* starts, const int32_t* lengths, void* stream) {
    const NvtxRange nvtx_range("kv8_append");
    if (!dtype_ok(dtype)) return QG_ERR_UNSUPPORTED;
    const Kv8Args a = {kq, vq, ks, vs, table, starts, lengths, B, rows, pages, page, heads, D, table_cols};
    int rc = check_kv8(a);
    if (rc || B == 0 || rows == 0) return rc;
    rc = check_kv8_rows(dtype, K, ldk, heads * D, rows);
    if (!rc) rc = check_kv8_rows(dtype, V, ldv, heads * D, rows);
    if (rc) return rc;
    if (current_device() < 0) return QG_ERR_CUDA;
    AppendParams p = {};
    kv8_params(a, &p.c, &p.bt);
    p.K = K; p.V = V; p.ldk = ldk; p.ldv = ldv;
    p.k_aligned = rows_aligned(dtype, K, ldk);
    p.v_aligned = rows_aligned(dtype, V, ldv);
    // a sequence's n new tokens touch at most n pages, and at most n / page + 2
    const int64_t bound = rows / page + 2 * B, units = rows < bound ? rows : bound;
    return by_dtype(dtype, [&](auto t) {
        return launch_serialized(k_kv8_append<decltype(t)>,
                                 dim3(static_cast<unsigned>(units),
                                      static_cast<unsigned>((2 * heads + kAppendWarps - 1) / kAppendWarps)),
                                 kAppendThreads, 0,
                                 1, static_cast<cudaStream_t>(stream), p);
    });
}

int kv8_gather(int dtype, int64_t B, int64_t rows, int64_t heads, int64_t D, const int8_t* kq, const int8_t* vq,
               const float* ks, const float* vs, int64_t pages, int64_t page, const int32_t* table, int64_t table_cols,
               const int32_t* starts, const int32_t* lengths, void* K, int64_t ldk, void* V, int64_t ldv,
               void* stream) {
    const NvtxRange nvtx_range("kv8_gather");
    if (!dtype_ok(dtype)) return QG_ERR_UNSUPPORTED;
    const Kv8Args a = {const_cast<int8_t*>(kq), const_cast<int8_t*>(vq), const_cast<float*>(ks),
                       const_cast<float*>(vs), table, starts, lengths, B, rows, pages, page, heads, D, table_cols};
    int rc = check_kv8(a);
    if (rc || B == 0 || rows == 0) return rc;
    rc = check_kv8_rows(dtype, K, ldk, heads * D, rows);
    if (!rc) rc = check_kv8_rows(dtype, V, ldv, heads * D, rows);
    if (rc) return rc;
    if (current_device() < 0) return QG_ERR_CUDA;
    GatherParams p = {};
    kv8_params(a, &p.c, &p.bt);
    p.K = K; p.V = V; p.ldk = ldk; p.ldv = ldv;
    p.k_aligned = rows_aligned(dtype, K, ldk);
    p.v_aligned = rows_aligned(dtype, V, ldv);
    return by_dtype(dtype, [&](auto t) {
        return launch_serialized(k_kv8_gather<decltype(t)>, dim3(static_cast<unsigned>((rows + kGatherRows - 1) / kGatherRows)),
                                 kGatherThreads, 0, 1,
                                 static_cast<cudaStream_t>(stream), p);
    });
}

}  // extern "C"
