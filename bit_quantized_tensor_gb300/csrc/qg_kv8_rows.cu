// Attention over the paged 8-bit cache (kv8_common.cuh): many query rows a sequence, on tcgen05.
//
// The mathematics is that of the kernel for few rows: codes as exact fp16 operands, a page's
// scales outside the products, weights 2^(x + log2 sv - M) in fp16.  With
//   t_j = raw_j c_b + l_b,   c_b = factor sk_b,  l_b = log2 sv_b      (b: j's 16 tokens)
// a weight is one fused multiply-add and one 2^x, like a softmax without scales.
//
// A CTA takes 256 rows (two tiles of 128: the heads that share a key head, times tokens) of a
// sequence and key head, against its tokens 128 at a time:
//   warps 0-3   softmax of tile 0, thread = row (its lane of tensor memory)
//   warps 4-7   softmax of tile 1
//   warps 8-11  codes of K and V from the cache through registers to fp16 in shared memory
//   warp 12     MMA issuer, owner of the tensor memory
// S (128 x 128 fp32) of either tile lies in tensor memory, its weights (fp16) over its first half,
// from where they are the A operand of the product with V; O (128 x D fp32) beside it.  One
// tile's products run while the other's weights are made.  Both K and V lie in shared memory as
// tokens by 64 values (128-byte swizzle), which is K's K-major and V's MN-major form, so they are
// converted alike.  A row's sums are rescaled, in tensor memory, only when its maximum grows by 2^8.
#include <cuda.h>

#include "kv8_attn.cuh"
#include "norm_common.cuh"
#include "qg_gemm_host.h"

namespace qg {

constexpr int kRowsThreads = 13 * 32;
constexpr int kRowsTile = 128;   // rows of a tile, tokens of a step
constexpr int kSiteRowsK = 421, kSiteRowsV = 422, kSiteRowsS = 423, kSiteRowsP = 424, kSiteRowsPv = 425,
              kSiteRowsFree = 426, kSiteRowsQ = 427, kSiteRowsDrain = 428;

template <int D>
struct RowsCfg {
    static constexpr int BLOCKS = D / 64;                  // 128-byte columns of a tile
    static constexpr int TILE_BYTES = 128 * 2 * D;         // 128 rows of fp16
    static constexpr int STAGES = 2;                       // of K and of V
    static constexpr int RING = 2 * TILE_BYTES;            // after the two tiles of Q
    static constexpr int BARS = RING + 2 * STAGES * TILE_BYTES;
    // at least half an SM's, so that no two CTAs meet on one (each takes all tensor memory)
    static constexpr int SMEM = BARS + 256 + 1024 > 117760 ? BARS + 256 + 1024 : 117760;
    static constexpr uint32_t O_COL = 256;                 // S of tile t at 128 t, O at 256 + D t
    static constexpr uint32_t IDESC_S = make_idesc(0, 0, 128, 128);
    static constexpr uint32_t IDESC_O = make_idesc(0, 0, 128, D) | (1u << 16);  // B is MN-major
    static_assert(SMEM <= 232448, "shared memory");
    static_assert(2 * SMEM > 233472, "one CTA an SM");
};

// Shared-memory descriptors: 128-byte swizzle, 1024 bytes between groups of 8 rows; the low word
// has the address and, MN-major, the distance of the next 64 columns.
constexpr uint32_t kTileHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t tile_lo(uint32_t addr, uint32_t next) {
    return ((addr & 0x3FFFFu) >> 4) | ((next >> 4) << 16);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t alo, uint32_t blo, uint32_t idesc, uint32_t accumulate,
                                       uint32_t elected) {
    asm volatile(
        "{\n.reg .pred p, q;\n.reg .b64 da, db;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %5, 0;\n"
        "mov.b64 da, {%1, %6};\nmov.b64 db, {%2, %6};\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}" ::"r"(d),
        "r"(alo), "r"(blo), "r"(idesc), "r"(accumulate), "r"(elected), "r"(kTileHi)
        : "memory");
}
// A from tensor memory.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t blo, uint32_t idesc, uint32_t accumulate,
                                       uint32_t elected) {
    asm volatile(
        "{\n.reg .pred p, q;\n.reg .b64 db;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %5, 0;\n"
        "mov.b64 db, {%2, %6};\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n}" ::"r"(d),
        "r"(a), "r"(blo), "r"(idesc), "r"(accumulate), "r"(elected), "r"(kTileHi)
        : "memory");
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Units of a sequence: key heads times pairs of row tiles.
__device__ __forceinline__ int64_t rows_units(const AttnParams& p, int b) {
    const Kv8Seq s = kv8_seq(p.bt, p.c, b);
    return static_cast<int64_t>(p.c.heads) * ((static_cast<int64_t>(s.n) * p.group + 2 * kRowsTile - 1) / (2 * kRowsTile));
}

template <class T, int D>
__global__ void __launch_bounds__(kRowsThreads, 1) k_kv8_attention_rows(const AttnParams p) {
    using Cfg = RowsCfg<D>;
    constexpr int TILE = kRowsTile;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                     ~static_cast<uintptr_t>(1023));
    __shared__ int64_t mem[kRowsThreads / 32 + 2];
    uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + Cfg::BARS);
    const uint32_t bar0 = smem_u32(bars), smem0 = smem_u32(smem);
    auto k_full = [&](int s) { return bar0 + 8u * s; };
    auto k_free = [&](int s) { return bar0 + 16u + 8u * s; };
    auto v_full = [&](int s) { return bar0 + 32u + 8u * s; };
    auto v_free = [&](int s) { return bar0 + 48u + 8u * s; };
    auto s_full = [&](int t) { return bar0 + 64u + 8u * t; };   // scores of tile t
    auto p_full = [&](int t) { return bar0 + 80u + 8u * t; };   // its weights
    auto pv_done = [&](int t) { return bar0 + 96u + 8u * t; };  // its product with V
    const uint32_t q_full = bar0 + 112u, drain = bar0 + 120u;
    uint32_t* const tmem_holder = reinterpret_cast<uint32_t*>(bars + 16);
    volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(k_full(i), 4);
            mbar_init(k_free(i), 1);
            mbar_init(v_full(i), 4);
            mbar_init(v_free(i), 1);
            mbar_init(s_full(i), 1);
            mbar_init(p_full(i), 4);
            mbar_init(pv_done(i), 1);
        }
        mbar_init(q_full, 8);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    pdl_wait_prior_grid();
    const Kv8Place at = kv8_find<kRowsThreads>(p.bt.B, blockIdx.x, 0, mem, [&](int b) { return rows_units(p, b); });
    if (at.b >= p.bt.B) return;  // more CTAs than units; no tensor memory is held yet
    if (warp == 12) tmem_alloc(smem_u32(tmem_holder), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // not before the tensor memory is held: the next kernel may take its own and then wait for this one
    pdl_launch_dependents();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_holder, 0);

    // the unit: the last rows, which see most, come first
    const Kv8Seq seq = kv8_seq(p.bt, p.c, at.b);
    const int heads = p.c.heads, all_rows = seq.n * p.group;
    const int head = static_cast<int>(at.at % heads);
    const int row0 = ((all_rows + 2 * TILE - 1) / (2 * TILE) - 1 - static_cast<int>(at.at / heads)) * 2 * TILE;
    auto seen_by = [&](int row) {
        const int64_t n = p.causal ? seq.first + row / p.group + 1 : seq.len;
        return row >= all_rows || n < 0 ? 0 : n < seq.len ? static_cast<int>(n) : seq.len;
    };
    // steps of 128 tokens that either tile sees
    int steps[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int first = row0 + t * TILE, last = min(all_rows, first + TILE) - 1;
        steps[t] = first < all_rows ? (seen_by(last) + TILE - 1) / TILE : 0;
    }
    const int most = max(steps[0], steps[1]);
    const int page_log2 = p.c.page_log2;
    const int tokens = max(seen_by(min(all_rows, row0 + TILE) - 1), seen_by(min(all_rows, row0 + 2 * TILE) - 1));
    // page * heads + head of a 16-token block, -1 without a page or behind what is seen
    auto unit_of = [&](int block) {
        if (16 * block >= tokens) return -1;
        const int page = kv8_page(p.c, at.b, (16 * block) >> page_log2);
        return page < 0 ? -1 : page * heads + head;
    };
    const float nan = __uint_as_float(0x7fc00000u);

    if (warp < 8) {
        // ------------------------------------------------ queries, softmax, result of a row
        const int t = warp >> 2, r = threadIdx.x & (TILE - 1), row = row0 + t * TILE + r;
        const uint32_t quad = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t s_at = quad + 128u * t, o_at = quad + Cfg::O_COL + D * t;
        float factor = 0.f;
        {
            const bool in = row < all_rows;
            const T* q = static_cast<const T*>(p.Q) + (seq.row0 + row / p.group) * p.ldq +
                         (head * p.group + row % p.group) * D;
            uint32_t bits = 0;
#pragma unroll 4
            for (int i = 0; i < D / 8; ++i) {
                float f[8];
                load_some<T, 8>(q + 8 * i, in ? 8 : 0, p.q_align == 16, f);
#pragma unroll
                for (int k = 0; k < 8; ++k) bits = max(bits, abs_bits(f[k]));
            }
            const RowPower power = row_power(bits);
            // the factor of a score is not negative: the scale's sign goes into the queries
            const float up = p.scale_log2 < 0.f ? -power.up : power.up;
            factor = power.down * fabsf(p.scale_log2);
            uint8_t* const to = smem + t * Cfg::TILE_BYTES + r * 128;
#pragma unroll 4
            for (int i = 0; i < D / 8; ++i) {
                float f[8];
                load_some<T, 8>(q + 8 * i, in ? 8 : 0, p.q_align == 16, f);
#pragma unroll
                for (int k = 0; k < 8; ++k) f[k] *= up;
                *reinterpret_cast<uint4*>(to + (i >> 3) * 16384 + (((i & 7) ^ (r & 7)) << 4)) =
                    make_uint4(pack2<__half>(f[0], f[1]), pack2<__half>(f[2], f[3]), pack2<__half>(f[4], f[5]),
                               pack2<__half>(f[6], f[7]));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
        }
        const int sees = seen_by(row), mine = steps[t];
        // scales of a step's 8 blocks, one a lane, read a step ahead
        struct Scales {
            float sk, lsv, isv;
        };
        auto fetch = [&](int step) {
            Scales v = {nan, nan, nan};
            const int unit = lane < 8 && step < mine ? unit_of(8 * step + lane) : -1;
            if (unit >= 0) {
                const float sv = p.c.vs[unit];
                v = {p.c.ks[unit], __log2f(sv), __fdividef(1.f, sv)};
            }
            return v;
        };
        Scales next = fetch(0);
        float M = neg_inf(), den = 0.f;
        bool ok = true;
        for (int step = 0; step < mine; ++step) {
            const Scales now = next;
            next = fetch(step + 1);
            if (!__all_sync(0xffffffffu, bounded_wait(s_full(t), step & 1, abort_flag, p.ctl, kSiteRowsS))) {
                ok = false;
                break;
            }
            tc_fence_after();
            const int left = sees - step * TILE;  // of the step's tokens
            const bool whole = __all_sync(0xffffffffu, left >= TILE);
            // loops over 32 tokens are not unrolled: the roles' code has to stay in the instruction cache
            float top = neg_inf();
            if (whole) {
#pragma unroll 1
                for (int ch = 0; ch < 4; ++ch) {
                    uint32_t x[32];
                    tmem_ld_32x32b_x32(s_at + 32 * ch, x);
                    tmem_wait_ld();
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float m0 = __uint_as_float(x[16 * h]), m1 = __uint_as_float(x[16 * h + 1]);
#pragma unroll
                        for (int i = 2; i < 14; i += 4) {
                            m0 = max3(m0, __uint_as_float(x[16 * h + i]), __uint_as_float(x[16 * h + i + 1]));
                            m1 = max3(m1, __uint_as_float(x[16 * h + i + 2]), __uint_as_float(x[16 * h + i + 3]));
                        }
                        m0 = max3(m0, __uint_as_float(x[16 * h + 14]), __uint_as_float(x[16 * h + 15]));
                        const float c = factor * __shfl_sync(0xffffffffu, now.sk, 2 * ch + h);
                        top = fmaxf(top, fmaf(fmaxf(m0, m1), c, __shfl_sync(0xffffffffu, now.lsv, 2 * ch + h)));
                    }
                }
            } else {
#pragma unroll 1
                for (int b = 0; b < 8; ++b) {
                    uint32_t x[16];
                    tmem_ld_32x32b_x16(s_at + 16 * b, x);
                    tmem_wait_ld();
                    const float c = factor * __shfl_sync(0xffffffffu, now.sk, b), l = __shfl_sync(0xffffffffu, now.lsv, b);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (16 * b + i < left) top = fmaxf(top, fmaf(__uint_as_float(x[i]), c, l));
                }
            }
            // O is at rest: this step's scores were issued behind the last step's product with V
            if (__any_sync(0xffffffffu, top > M + kLazy)) {
                const float m = fmaxf(M, top);
                const float f = M == neg_inf() ? 0.f : exp2_fast(M - m);
                M = m;
                den *= f;
                if (step) {
#pragma unroll 1
                    for (int d = 0; d < D; d += 16) {
                        uint32_t x[16];
                        tmem_ld_32x32b_x16(o_at + d, x);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
                        tmem_st_x16(o_at + d, x);
                    }
                }
            }
            const float base = M == neg_inf() ? 0.f : M;
            auto weights = [&](auto all) {
#pragma unroll 1
                for (int ch = 0; ch < 4; ++ch) {
                    uint32_t x[32], w[16];
                    tmem_ld_32x32b_x32(s_at + 32 * ch, x);
                    tmem_wait_ld();
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float c = factor * __shfl_sync(0xffffffffu, now.sk, 2 * ch + h);
                        const float l = __shfl_sync(0xffffffffu, now.lsv, 2 * ch + h) - base;
                        const float isv = __shfl_sync(0xffffffffu, now.isv, 2 * ch + h);
                        const uint64_t cc = two(c, c), ll = two(l, l);
                        uint64_t sum = two(0.f, 0.f);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int k = 16 * h + 2 * i;
                            float2 e = both(fma_two(two(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), cc, ll));
                            if constexpr (!decltype(all)::value) {
                                if (32 * ch + k >= left) e.x = neg_inf();
                                if (32 * ch + k + 1 >= left) e.y = neg_inf();
                            }
                            e.x = exp2_fast(e.x);
                            e.y = exp2_fast(e.y);
                            sum = add_two(sum, two(e.x, e.y));
                            w[8 * h + i] = pack2<__half>(e.x, e.y);
                        }
                        const float2 s2 = both(sum);
                        if (!(s2.x + s2.y == 0.f)) den = fmaf(s2.x + s2.y, isv, den);  // not 0 times a NaN not seen
                    }
                    tmem_st_x16(s_at + 16 * ch, w);  // over scores that have been read
                }
            };
            if (whole)
                weights(std::true_type{});
            else
                weights(std::false_type{});
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full(t));
        }
        if (ok && mine)
            ok = __all_sync(0xffffffffu, bounded_wait(pv_done(t), (mine - 1) & 1, abort_flag, p.ctl, kSiteRowsPv));
        tc_fence_after();
        if (ok) {
            T* out = static_cast<T*>(p.O) + (seq.row0 + row / p.group) * p.ldo + (head * p.group + row % p.group) * D;
            const bool sectors = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
            const float scale = den == 0.f ? 0.f : 1.f / den;
#pragma unroll 1
            for (int d = 0; d < D; d += 16) {
                uint32_t x[16];
                float f[16];
                if (mine) {
                    tmem_ld_32x32b_x16(o_at + d, x);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    f[i] = seq.cut ? nan : !mine || den == 0.f ? 0.f : __uint_as_float(x[i]) * scale;
                if (row < all_rows) {
                    if (sectors)
                        store_sectors<T>(out + d, f);
                    else
                        store_some<T, 16>(out + d, 16, false, f);
                }
            }
        }
        tc_fence_before();
    } else if (warp < 12) {
        // ------------------------------------------------ codes to fp16
        constexpr int CH = D / 16, PASS = 128 / CH;  // 16-byte pieces of a token; tokens a pass
        const int tid = threadIdx.x - 256, chunk = tid % CH, tok0 = tid / CH;
        int unit = lane < 8 ? unit_of(lane) : -1, unit_next = -1;
        uint4 raw[CH];
        // pieces of K or V of a step into registers; zeros where there is no token
        auto load = [&](int step, int units, const int8_t* codes) {
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int tok = tok0 + i * PASS;
                const int at_unit = __shfl_sync(0xffffffffu, units, tok >> 4);
                raw[i] = make_uint4(0, 0, 0, 0);
                if (at_unit >= 0) {
                    const int offset = (step * TILE + tok) & ((1 << page_log2) - 1);
                    raw[i] = *reinterpret_cast<const uint4*>(
                        codes + ((static_cast<int64_t>(at_unit) << page_log2) + offset) * D + 16 * chunk);
                }
            }
        };
        auto store = [&](uint32_t stage_at) {
            uint8_t* const to = smem + stage_at + (chunk >> 2) * 16384;
            const int odd = (chunk >> 2) & 1;  // the second columns' lanes store their halves in turn, not to meet in a bank
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int tok = tok0 + i * PASS, c0 = 2 * (chunk & 3);
                uint32_t h[8];
                s8_to_f16(raw[i].x, h[0], h[1]);
                s8_to_f16(raw[i].y, h[2], h[3]);
                s8_to_f16(raw[i].z, h[4], h[5]);
                s8_to_f16(raw[i].w, h[6], h[7]);
                const uint4 a = make_uint4(h[0], h[1], h[2], h[3]), b = make_uint4(h[4], h[5], h[6], h[7]);
                uint8_t* const at_row = to + tok * 128;
                *reinterpret_cast<uint4*>(at_row + (((c0 + odd) ^ (tok & 7)) << 4)) = odd ? b : a;
                *reinterpret_cast<uint4*>(at_row + (((c0 + 1 - odd) ^ (tok & 7)) << 4)) = odd ? a : b;
            }
            fence_proxy_async_smem();
            __syncwarp();
        };
        if (most) load(0, unit, p.c.kq);
        for (int step = 0; step < most; ++step) {
            const int s = step & 1;
            const uint32_t parity = ((step >> 1) & 1) ^ 1;
            if (lane < 8) unit_next = unit_of(8 * (step + 1) + lane);
            if (!__all_sync(0xffffffffu, bounded_wait(k_free(s), parity, abort_flag, p.ctl, kSiteRowsFree))) break;
            store(Cfg::RING + s * Cfg::TILE_BYTES);
            if (lane == 0) mbar_arrive(k_full(s));
            load(step, unit, p.c.vq);
            if (!__all_sync(0xffffffffu, bounded_wait(v_free(s), parity, abort_flag, p.ctl, kSiteRowsFree))) break;
            store(Cfg::RING + (2 + s) * Cfg::TILE_BYTES);
            if (lane == 0) mbar_arrive(v_full(s));
            unit = unit_next;
            if (step + 1 < most) load(step + 1, unit, p.c.kq);
        }
    } else {
        // ------------------------------------------------ MMA issuer
        const uint32_t elected = elect_lane();
        auto wait = [&](uint32_t bar, uint32_t parity, int site) {
            return __all_sync(0xffffffffu, bounded_wait(bar, parity, abort_flag, p.ctl, site));
        };
        auto commit = [&](uint32_t bar) {
            if (elected) tc_commit(bar);
            __syncwarp();
        };
        // scores of tile t of a step: S = Q K^T
        auto scores = [&](int t, int step) {
            const uint32_t q = smem0 + t * Cfg::TILE_BYTES, k = smem0 + Cfg::RING + (step & 1) * Cfg::TILE_BYTES;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                const uint32_t at_k = (i >> 2) * 16384u + (i & 3) * 32u;
                mma_ss(tmem + 128u * t, tile_lo(q + at_k, 16), tile_lo(k + at_k, 16), Cfg::IDESC_S, i > 0, elected);
            }
            commit(s_full(t));
        };
        auto values = [&](int t, int step) {
            const uint32_t v = smem0 + Cfg::RING + (2 + (step & 1)) * Cfg::TILE_BYTES;
#pragma unroll
            for (int i = 0; i < TILE / 16; ++i)
                mma_ts(tmem + Cfg::O_COL + D * t, tmem + 128u * t + 8u * i, tile_lo(v + 2048u * i, 16384), Cfg::IDESC_O,
                       step > 0 || i > 0, elected);
            commit(pv_done(t));
        };
        bool ok = most == 0 || (wait(q_full, 0, kSiteRowsQ) && wait(k_full(0), 0, kSiteRowsK));
        if (ok && most) {
            tc_fence_after();
            if (steps[0]) scores(0, 0);
            if (steps[1]) scores(1, 0);
            commit(k_free(0));
        }
        for (int step = 0; ok && step < most; ++step) {
            const int s = step & 1;
            const uint32_t parity = (step >> 1) & 1;
            if (!(ok = wait(v_full(s), parity, kSiteRowsV))) break;
            bool k_ready = false;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (ok && step < steps[t]) {
                    if (!(ok = wait(p_full(t), step & 1, kSiteRowsP))) break;
                    tc_fence_after();
                    values(t, step);
                    if (t == 1 || step >= steps[1]) commit(v_free(s));
                }
                if (ok && step + 1 < steps[t]) {
                    if (!k_ready) ok = wait(k_full((step + 1) & 1), ((step + 1) >> 1) & 1, kSiteRowsK);
                    k_ready = true;
                    // the scores go where the weights lie that the product just issued reads
                    if (!ok || !(ok = wait(pv_done(t), step & 1, kSiteRowsPv))) break;
                    tc_fence_after();
                    scores(t, step + 1);
                    if (t == 1 || step + 1 >= steps[1]) commit(k_free((step + 1) & 1));
                }
            }
        }
        commit(drain);  // every MMA issued has completed before anything is released
        bounded_wait(drain, 0, nullptr, p.ctl, kSiteRowsDrain);
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Does a problem of these sizes go to the kernel above?
bool attention_takes_rows(const AttnParams& p) {
    if (p.c.D == 256) return false;
    const int64_t rows = static_cast<int64_t>(p.bt.rows) * p.group;
    return rows >= 64 * static_cast<int64_t>(p.bt.B);
}

template <class T, int D>
static int launch_rows(const AttnParams& p, cudaStream_t s) {
    struct Tag;
    const int rc = raise_smem<Tag>(k_kv8_attention_rows<T, D>);
    if (rc) return rc;
    const int64_t rows = static_cast<int64_t>(p.bt.rows) * p.group;
    const int64_t units = (rows / (2 * kRowsTile) + (p.bt.B < p.bt.rows ? p.bt.B : p.bt.rows)) * p.c.heads;
    if (units > INT32_MAX) return QG_ERR_INVALID_ARG;
    return launch_serialized(k_kv8_attention_rows<T, D>, dim3(static_cast<unsigned>(units)), kRowsThreads,
                             RowsCfg<D>::SMEM, 1, s, p);
}

int attention_rows(int dtype, const AttnParams& p, cudaStream_t s) {
    if (dtype == QG_F16) return p.c.D == 64 ? launch_rows<__half, 64>(p, s) : launch_rows<__half, 128>(p, s);
    return p.c.D == 64 ? launch_rows<__nv_bfloat16, 64>(p, s) : launch_rows<__nv_bfloat16, 128>(p, s);
}

#define QG_ROWS_BUDGET(T, NAME, D)                                                           \
    QG_BLOCK_KERNEL_BUDGET("k_kv8_attention_rows<" NAME "," #D ">",                          \
                           (reinterpret_cast<const void*>(k_kv8_attention_rows<T, D>)),      \
                           kRowsThreads, RowsCfg<D>::SMEM, 512, 1, 1)
QG_ROWS_BUDGET(__half, "f16", 64);
QG_ROWS_BUDGET(__half, "f16", 128);
QG_ROWS_BUDGET(__nv_bfloat16, "bf16", 64);
QG_ROWS_BUDGET(__nv_bfloat16, "bf16", 128);

}  // namespace qg
