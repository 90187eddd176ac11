// Attention over the paged 8-bit cache (kv8_common.cuh): few query rows a sequence.
//
//   x_j = scale log2(e) sk_j (q . kq_j)                      exponent of token j
//   O = sum_j 2^x_j sv_j vq_j / sum_j 2^x_j
//
// The codes go to the tensor cores as exact fp16 numbers, so a page's scales have to
// stay outside: sk is a factor of the product's result, and sv goes into the exponent,
//   w_j = 2^(x_j + log2 sv_j - M + 9),   O = sum w_j vq_j / sum (w_j / sv_j),
// with M + 6 a running upper bound of x_j + log2 sv_j, so that w_j, rounded to fp16 for the
// second product, is at most 2^15 whatever the pages' scales are.  (Where that leaves w_j
// hardly anything, its term of the denominator is 2^(x_j - M + 9).)  Sums, M and the
// denominator are fp32.  Queries go in as fp16 times a power of two of their row, which
// is exact for bf16 too but for values 2^-28 of the row's largest.
#include <cuda.h>

#include "kv8_attn.cuh"
#include "kv8_host.h"
#include "qg_gemm_host.h"

namespace qg {

// One warp takes 32 tokens a step, for 8 or 16 rows (NB = 1, 2): the heads that share a key
// head, times a sequence's query rows.  Tokens are the rows of the products' results and
// query rows their 8 columns (S^T = K Q^T, O^T = V^T P^T), so that 4 or 8 heads a key head
// waste little; the weights change sides in registers (movmatrix).  All (sequence, key
// head, rows) units' tiles of 128 tokens lie on one axis that the CTAs cut into equal
// pieces, wherever the units' borders are, so a batch of any lengths loads all SMs alike;
// a unit that several CTAs have parts of is joined by a second kernel from their fp32 sums.
//
// The cache's bytes are what this cannot do without, and turning them into fp16 is most of
// what it executes, so the rest is kept small: each warp has a ring of its own that TMA
// fills (a box for 16 or 32 tokens, swizzled so that no lanes meet in a bank), and no
// barrier but the end of a unit; the running maximum is looked at once for 32 tokens and
// the sums are rescaled only when it has grown by 2^6.
//
// Measured, 32 heads of 128 values on 8 key heads: one token each for 64 sequences of up to 8192
// 118.6 us, 5.6 TB/s (83% of a copy); one token over 131071 62 us, 4.3 TB/s, where the join, which a
// copy does not need, and the start of a lone round of CTAs show.
constexpr int kAttnWarps = 4, kAttnThreads = 32 * kAttnWarps;
constexpr int kAttnStep = 32;                       // tokens of a warp's step
constexpr int kAttnTile = kAttnStep * kAttnWarps;
constexpr int kAttnStages = 2;
constexpr int kSiteAttnK = 411, kSiteAttnV = 412;

// Box of 16 or 32 tokens of a page and head, 128 bytes (or D) of each.  Issued by a whole
// warp under an elected lane's predicate, which keeps its operands in uniform registers.
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, int d, int token, int unit, uint32_t bar,
                                         uint32_t elected) {
    asm volatile(
        "{\n.reg .pred q;\nsetp.ne.b32 q, %6, 0;\n"
        "@q cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];\n}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(d), "r"(token), "r"(unit), "r"(bar), "r"(elected)
        : "memory");
}
// An 8 x 8 matrix of 16-bit values, two a lane (row lane / 4), transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
    return d;
}

// Units and tiles of a sequence.
struct AttnSeq {
    Kv8Seq s;
    int rows, row_tiles, tiles;
    __device__ __forceinline__ int64_t work(int heads) const { return static_cast<int64_t>(heads) * row_tiles * tiles; }
};
template <int NB>
__device__ __forceinline__ AttnSeq attn_seq(const AttnParams& p, int b) {
    AttnSeq a;
    a.s = kv8_seq(p.bt, p.c, b);
    a.rows = a.s.n * p.group;
    if (a.rows >= p.from) a.rows = 0;  // the other kernel's
    a.row_tiles = (a.rows + 8 * NB - 1) / (8 * NB);
    a.tiles = max(1, (a.s.len + kAttnTile - 1) / kAttnTile);
    return a;
}

// Where a CTA's piece of the axis starts.
struct AttnUnit {
    int b, head, row_tile;
    int64_t tile;
};
template <int NB>
__device__ __forceinline__ AttnUnit attn_unit(const AttnParams& p, const Kv8Place& at) {
    AttnUnit u = {at.b, 0, 0, 0};
    if (at.b >= p.bt.B) return u;
    const AttnSeq a = attn_seq<NB>(p, at.b);
    const int64_t per_head = static_cast<int64_t>(a.row_tiles) * a.tiles;
    u.head = static_cast<int>(at.at / per_head);
    const int64_t rest = at.at - u.head * per_head;
    u.row_tile = static_cast<int>(rest / a.tiles);
    u.tile = rest % a.tiles;
    return u;
}

// The token of a box's 8 (or the second 8) that is column n of a product, so that the
// lanes that read together, two tokens by four 16-byte pieces of K and four tokens by two
// pieces (D = 64: four half pieces) of V, lie in different banks under TMA's swizzle.
__device__ __forceinline__ constexpr int token_of(int n) {
    return (((n >> 2) & 1) * 4 + ((n >> 1) & 1) * 3) ^ ((n & 1) * 5);
}

template <int D, int NB_>
struct AttnCfg {
    static constexpr int NB = NB_, ROWS = 8 * NB;
    static constexpr int W = D < 128 ? D : 128;         // bytes of a box's row
    static constexpr int BOXES = D / W;                 // boxes across a head
    static constexpr int HALF_BYTES = 16 * W;           // 16 tokens of a box
    static constexpr int KV_BYTES = 2 * BOXES * HALF_BYTES;  // K, or V, of a step
    static constexpr int WARP_BYTES = 2 * kAttnStages * KV_BYTES;
    static constexpr int STRIDE = D + 2;                // floats of a row of partial sums: O, M, denominator
    static constexpr int PART = ROWS * STRIDE;
    static constexpr int SMEM = kAttnWarps * WARP_BYTES + 1024;
    static constexpr int PER_SM = D == 64 ? 4 : D == 128 ? 3 : 1;
    static_assert(kAttnWarps * PART * 4 <= SMEM - 1024, "partial sums reuse the rings");
    // address in a box of 16-byte piece `chunk` of token t
    __device__ __forceinline__ static int place(int t, int chunk) {
        return t * W + ((chunk ^ (W == 128 ? t & 7 : (t >> 1) & 3)) << 4);
    }
};

// Two values of a row of the result: 0 for a row that sees nothing, NaN for a sequence that is
// longer than its table and for a row whose scores are all -inf (a query with an infinity; its
// softmax is 0 / 0).  With any finite score the total is not 0.
template <class T>
__device__ __forceinline__ void store_out(const AttnParams& p, const AttnSeq& a, int head, int row, int d, int D,
                                          float2 sum, float total) {
    T* out = static_cast<T*>(p.O) + (a.s.row0 + row / p.group) * p.ldo + (head * p.group + row % p.group) * D + d;
    float f = kDenUnit / total;
    if (total == 0.f) {  // (a branch: as a choice it cost the kernel's loop 1 to 3%)
        const bool sees = a.s.len > 0 && (!p.causal || a.s.first + row / p.group >= 0);
        sum.x = sum.y = 0.f;
        f = sees ? __uint_as_float(0x7fc00000u) : 0.f;
    }
    if (a.s.cut) f = __uint_as_float(0x7fc00000u);
    out[0] = from_f32<T>(sum.x * f);
    out[1] = from_f32<T>(sum.y * f);
}

template <class T, int D, int NB>
__global__ void __launch_bounds__(kAttnThreads, AttnCfg<D, NB>::PER_SM)
    k_kv8_attention(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const AttnParams p) {
    using Cfg = AttnCfg<D, NB>;
    constexpr int KS = D / 16;          // MMA steps of k . q
    constexpr int DT = D / 16;          // 16-value tiles of O^T
    constexpr int PER = Cfg::W / 8;     // values of a token that a lane holds of a box of V
    constexpr int ROWS = Cfg::ROWS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                     ~static_cast<uintptr_t>(1023));
    __shared__ int64_t mem[kAttnWarps + 2];
    __shared__ __align__(8) uint64_t bars[kAttnWarps][2 * kAttnStages];
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    uint8_t* const ring = smem + warp * Cfg::WARP_BYTES;
    const uint32_t ring_u32 = smem_u32(ring), bar0 = smem_u32(&bars[warp][0]);
    const uint32_t elected = elect_lane();
    auto k_bar = [&](int s) { return bar0 + 16u * s; };
    auto v_bar = [&](int s) { return bar0 + 16u * s + 8u; };
    if (elected) {
        for (int s = 0; s < kAttnStages; ++s) {
            mbar_init(k_bar(s), 1);
            mbar_init(v_bar(s), 1);
        }
        fence_mbar_init();
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    __syncwarp();
    pdl_wait_prior_grid();
    fence_proxy_async_global();  // the cache may have been written just before, with ordinary stores
    const Kv8Place at = kv8_find<kAttnThreads>(p.bt.B, blockIdx.x, p.ctas, mem,
                                               [&](int b) { return attn_seq<NB>(p, b).work(p.c.heads); });
    int64_t w0 = at.total * blockIdx.x / p.ctas;
    const int64_t w1 = at.total * (blockIdx.x + 1) / p.ctas;
    AttnUnit u = attn_unit<NB>(p, at);
    const int page_log2 = p.c.page_log2;
    const bool wide = page_log2 > 4;  // a step's tokens lie in one page: boxes of 32
    uint32_t filled = 0;  // steps whose copies this warp has issued: their stage and phase
    bool ok = true;

    while (w0 < w1 && u.b < p.bt.B) {
        const AttnSeq a = attn_seq<NB>(p, u.b);
        if (a.rows == 0) {  // a sequence without rows has no place on the axis
            u = {u.b + 1, 0, 0, 0};
            continue;
        }
        const int64_t end = min(static_cast<int64_t>(a.tiles), u.tile + (w1 - w0));
        // tokens that a row of the sequence sees
        auto seen_by = [&](int row) {
            const int64_t n = p.causal ? a.s.first + row / p.group + 1 : a.s.len;
            return row >= a.rows || n < 0 ? 0 : n < a.s.len ? static_cast<int>(n) : a.s.len;
        };
        const int row0 = u.row_tile * ROWS;
        const int most = seen_by(min(a.rows, row0 + ROWS) - 1), least = seen_by(row0);
        // this lane's columns of the products: rows 8 n + 2 c + m of the unit
        int sees[NB][2];
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int m = 0; m < 2; ++m) sees[n][m] = seen_by(row0 + 8 * n + 2 * c + m);

        // this warp's steps of 32 tokens of tiles u.tile .. end that anyone sees
        const int t0 = static_cast<int>(u.tile) * kAttnTile + kAttnStep * warp;
        const int t1 = min(most, static_cast<int>(end) * kAttnTile);
        const int steps = t1 > t0 ? (t1 - t0 + kAttnTile - 1) / kAttnTile : 0;
        // pages of 16 steps' halves, one a lane, and what their scales come to: of this batch of
        // steps and of the next
        struct Half {
            int unit;          // page * heads + head, -1: no page
            float sk, lsv, isv;
        };
        auto fetch = [&](int batch) {
            const int token = t0 + (batch * 16 + (lane >> 1)) * kAttnTile + 16 * (lane & 1);
            Half h = {-1, __uint_as_float(0x7fc00000u), 0.f, 0.f};
            if (token < t1) {
                const int page = kv8_page(p.c, u.b, token >> page_log2);
                float sv = h.sk;
                if (page >= 0) {
                    h.unit = page * p.c.heads + u.head;
                    h.sk = p.c.ks[h.unit];
                    sv = p.c.vs[h.unit];
                }
                h.lsv = page_log2_of(sv);
                h.isv = exp2_fast(kDenPower - h.lsv);
            }
            return h;
        };
        Half now = fetch(0), next = now;
        if (steps > 16) next = fetch(1);
        // copies of K, or V, of a step; `unit` is that of its batch.  Steps are counted over all
        // units that the warp works on: stage and phase of a step
        const uint32_t base = filled;
        auto stage = [&](int step) { return static_cast<int>((base + step) % kAttnStages); };
        auto phase = [&](int step) { return ((base + step) / kAttnStages) & 1u; };
        auto load = [&](int step, int unit, bool value) {
            const int j = 2 * (step & 15), s = stage(step), token = t0 + step * kAttnTile, mask = (1 << page_log2) - 1;
            const int u0 = max(__shfl_sync(0xffffffffu, unit, j), 0);
            const uint32_t bar = value ? v_bar(s) : k_bar(s);
            const uint32_t dst = ring_u32 + (2 * s + (value ? 1 : 0)) * Cfg::KV_BYTES;
            const CUtensorMap* map = value ? &tmV : &tmK;
            const bool both_in = wide || token + 16 < t1;
            if (elected) mbar_arrive_expect_tx(bar, both_in ? Cfg::KV_BYTES : Cfg::KV_BYTES / 2);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < Cfg::BOXES; ++i)
                load_box(dst + 2 * i * Cfg::HALF_BYTES, map, i * Cfg::W, token & mask, u0, bar, elected);
            if (!wide && both_in) {
                const int u1 = max(__shfl_sync(0xffffffffu, unit, j + 1), 0);
#pragma unroll
                for (int i = 0; i < Cfg::BOXES; ++i)
                    load_box(dst + (2 * i + 1) * Cfg::HALF_BYTES, map, i * Cfg::W, (token + 16) & mask, u1, bar, elected);
            }
        };
        const int ready = ok ? steps : 0;
        for (int i = 0; i < kAttnStages && i < ready; ++i) {
            load(i, now.unit, false);
            load(i, now.unit, true);
        }

        // queries: for MMA step k lane c of row g holds the four values that its 32-bit word of a
        // token's codes has in that step
        uint32_t qf[NB][KS][2];
        float factor[NB][2];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            const int row = row0 + 8 * n + g;
            const T* q = static_cast<const T*>(p.Q) + (a.s.row0 + row / p.group) * p.ldq +
                         (u.head * p.group + row % p.group) * D + c * 16;
            uint32_t bits = 0;
            uint2 raw[KS];
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                raw[k] = make_uint2(0u, 0u);
                const T* at_k = q + (k / 4) * 64 + (k % 4) * 4;
                if (row < a.rows) {
                    if (p.q_align >= 8) {
                        raw[k] = *reinterpret_cast<const uint2*>(at_k);
                    } else {
                        const uint16_t* h = reinterpret_cast<const uint16_t*>(at_k);
                        raw[k] = make_uint2(h[0] | static_cast<uint32_t>(h[1]) << 16, h[2] | static_cast<uint32_t>(h[3]) << 16);
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const float2 x = unpack2<T>(raw[k].x), y = unpack2<T>(raw[k].y);
                bits = max(max(max(bits, abs_bits(x.x)), max(abs_bits(x.y), abs_bits(y.x))), abs_bits(y.y));
            }
            bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, 1));
            bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, 2));
            const RowPower power = row_power(bits);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const float2 x = unpack2<T>(raw[k].x), y = unpack2<T>(raw[k].y);
                qf[n][k][0] = pack2<__half>(x.x * power.up, x.y * power.up);
                qf[n][k][1] = pack2<__half>(y.x * power.up, y.y * power.up);
            }
            const float down = power.down * p.scale_log2;
            factor[n][0] = __shfl_sync(0xffffffffu, down, 8 * c);
            factor[n][1] = __shfl_sync(0xffffffffu, down, 8 * c + 4);
        }

        float o[DT][NB][4], M[NB][2], den[NB][2];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                M[n][m] = neg_inf();
                den[n][m] = 0.f;
            }
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[d][n][i] = 0.f;
        }

        for (int step = 0; step < ready; ++step) {
            if ((step & 15) == 0 && step) {
                now = next;
                if (step + 16 < ready) next = fetch(step / 16 + 1);
            }
            const int s = stage(step);
            if (!__all_sync(0xffffffffu, bounded_wait(k_bar(s), phase(step), nullptr, p.ctl, kSiteAttnK))) {
                ok = false;
                break;
            }
            // scores of 2 x 16 tokens (rows token_of(g) and 8 more of each 16) by the unit's rows
            const uint8_t* st = ring + 2 * s * Cfg::KV_BYTES;
            float x[2][NB][4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[h][n][i] = 0.f;
#pragma unroll
            for (int k = 0; k < KS; k += 4) {
                const int chunk = (k / 4) * 4 + c;  // of the head's 16-byte pieces
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint8_t* box = st + (2 * (chunk / (Cfg::W / 16)) + h) * Cfg::HALF_BYTES;
                    const uint4 lo = *reinterpret_cast<const uint4*>(box + Cfg::place(token_of(g), chunk % (Cfg::W / 16)));
                    const uint4 hi = *reinterpret_cast<const uint4*>(box + Cfg::place(8 + token_of(g), chunk % (Cfg::W / 16)));
                    const uint32_t lw[4] = {lo.x, lo.y, lo.z, lo.w}, hw[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        uint32_t a0, a1, a2, a3;
                        s8_to_f16(lw[m], a0, a2);
                        s8_to_f16(hw[m], a1, a3);
#pragma unroll
                        for (int n = 0; n < NB; ++n)
                            mma_f16(x[h][n], a0, a1, a2, a3, qf[n][k + m][0], qf[n][k + m][1]);
                    }
                }
            }
            __syncwarp();
            const int ahead = (step + kAttnStages) >> 4 == step >> 4 ? now.unit : next.unit;
            if (step + kAttnStages < ready) load(step + kAttnStages, ahead, false);

            const int j = 2 * (step & 15);
            float lsv[2], isv[2], top[NB][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float sk = __shfl_sync(0xffffffffu, now.sk, j + h);
                lsv[h] = __shfl_sync(0xffffffffu, now.lsv, j + h);
                isv[h] = __shfl_sync(0xffffffffu, now.isv, j + h);
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    const float f0 = factor[n][0] * sk, f1 = factor[n][1] * sk;
                    x[h][n][0] = fmaf(x[h][n][0], f0, lsv[h]);
                    x[h][n][1] = fmaf(x[h][n][1], f1, lsv[h]);
                    x[h][n][2] = fmaf(x[h][n][2], f0, lsv[h]);
                    x[h][n][3] = fmaf(x[h][n][3], f1, lsv[h]);
                }
            }
            const int tok = t0 + step * kAttnTile;
            if (tok + kAttnStep > least) {  // a step at the end of what some row sees
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int n = 0; n < NB; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (tok + 16 * h + token_of(g) + 8 * (i >> 1) >= sees[n][i & 1]) x[h][n][i] = neg_inf();
            }
            bool moves = false;
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    float v = fmaxf(fmaxf(x[0][n][m], x[0][n][m + 2]), fmaxf(x[1][n][m], x[1][n][m + 2]));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                    top[n][m] = v;
                    moves |= v > M[n][m] + kLazy;  // M is -inf at first
                }
            if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        const float v = fmaxf(M[n][m], top[n][m]);
                        const float half = M[n][m] == neg_inf() ? 0.f : exp2_fast(0.5f * (M[n][m] - v)), f = half * half;
                        M[n][m] = v;
                        den[n][m] = den[n][m] * half * half;
#pragma unroll
                        for (int d = 0; d < DT; ++d) {
                            o[d][n][m] *= f;
                            o[d][n][m + 2] *= f;
                        }
                    }
            }
            // weights, in fp16 and from the products' rows to their columns
            uint32_t pf[2][NB][2];
            bool low = false;
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                const float m0 = weight_base(M[n][0]), m1 = weight_base(M[n][1]);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float e0 = exp2_fast(x[h][n][0] - m0), e1 = exp2_fast(x[h][n][1] - m1);
                    const float e2 = exp2_fast(x[h][n][2] - m0), e3 = exp2_fast(x[h][n][3] - m1);
                    const float s0 = e0 + e2, s1 = e1 + e3;
                    // not the low ones, nor 0 times a NaN of tokens that are not seen
                    if (!(s0 < kLowWeight)) den[n][0] = fmaf(s0, isv[h], den[n][0]);
                    if (!(s1 < kLowWeight)) den[n][1] = fmaf(s1, isv[h], den[n][1]);
                    low |= s0 < kLowWeight || s1 < kLowWeight;
                    pf[h][n][0] = transposed(pack2<__half>(e0, e1));
                    pf[h][n][1] = transposed(pack2<__half>(e2, e3));
                }
            }
            if (__any_sync(0xffffffffu, low)) {
                // tokens of small scales next to large ones: 2^x, whose size they keep in the denominator
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        const float base = weight_base(M[n][m]);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float x0 = x[h][n][m], x2 = x[h][n][m + 2];
                            const bool less = exp2_fast(x0 - base) + exp2_fast(x2 - base) < kLowWeight;
                            if (less && x0 > neg_inf()) den[n][m] += exp2_fast(x0 - base + (kDenPower - lsv[h]));
                            if (less && x2 > neg_inf()) den[n][m] += exp2_fast(x2 - base + (kDenPower - lsv[h]));
                        }
                    }
                __syncwarp();
            }
            if (!__all_sync(0xffffffffu, bounded_wait(v_bar(s), phase(step), nullptr, p.ctl, kSiteAttnV))) {
                ok = false;
                break;
            }
            // O^T += V^T w: row g of a box's tiles are values g PER .. of its row, two a tile; lane c's
            // tokens are those of columns 2 c, 2 c + 1 of either 8, whose bytes are brought together
            st += Cfg::KV_BYTES;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int i = 0; i < Cfg::BOXES; ++i) {
                    const uint8_t* box = st + (2 * i + h) * Cfg::HALF_BYTES;
                    uint32_t vw[4][PER / 4];
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const int token = 8 * (t >> 1) + token_of(2 * c + (t & 1));
                        if constexpr (PER == 8) {
                            const uint2 w = *reinterpret_cast<const uint2*>(box + Cfg::place(token, g >> 1) + 8 * (g & 1));
                            vw[t][0] = w.x;
                            vw[t][1] = w.y;
                        } else {
                            const uint4 w = *reinterpret_cast<const uint4*>(box + Cfg::place(token, g));
                            vw[t][0] = w.x;
                            vw[t][1] = w.y;
                            vw[t][2] = w.z;
                            vw[t][3] = w.w;
                        }
                    }
#pragma unroll
                    for (int k = 0; k < PER / 4; ++k) {
                        // bytes of token pairs side by side, then as fp16 pairs
                        uint32_t b[4][2];
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const uint32_t lo = __byte_perm(vw[2 * r][k], vw[2 * r + 1][k], 0x5140);
                            const uint32_t hi = __byte_perm(vw[2 * r][k], vw[2 * r + 1][k], 0x7362);
                            s8_to_f16(lo, b[0][r], b[1][r]);
                            s8_to_f16(hi, b[2][r], b[3][r]);
                        }
                        const int tile = (i * PER + 4 * k) / 2;
#pragma unroll
                        for (int n = 0; n < NB; ++n) {
                            mma_f16(o[tile][n], b[0][0], b[1][0], b[0][1], b[1][1], pf[h][n][0], pf[h][n][1]);
                            mma_f16(o[tile + 1][n], b[2][0], b[3][0], b[2][1], b[3][1], pf[h][n][0], pf[h][n][1]);
                        }
                    }
                }
            }
            __syncwarp();
            if (step + kAttnStages < ready) load(step + kAttnStages, ahead, true);
        }
        filled += static_cast<uint32_t>(ready);

        // the warps' sums go where the rings were, and become the unit's or a part's
        __syncthreads();
        float* mine = reinterpret_cast<float*>(smem) + warp * Cfg::PART;
#pragma unroll
        for (int n = 0; n < NB; ++n) {
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                float v = den[n][m];
                v += __shfl_xor_sync(0xffffffffu, v, 4);
                v += __shfl_xor_sync(0xffffffffu, v, 8);
                v += __shfl_xor_sync(0xffffffffu, v, 16);
                float* r = mine + (8 * n + 2 * c + m) * Cfg::STRIDE;
#pragma unroll
                for (int d = 0; d < DT; ++d)
                    *reinterpret_cast<float2*>(r + (2 * d / PER) * Cfg::W + g * PER + 2 * d % PER) =
                        make_float2(o[d][n][m], o[d][n][m + 2]);
                if (g == 0) *reinterpret_cast<float2*>(r + D) = make_float2(M[n][m], v);
            }
        }
        __syncthreads();
        const bool whole = u.tile == 0 && end == a.tiles;
        const int rows = min(ROWS, a.rows - row0);
        float* part = p.part + (static_cast<int64_t>(blockIdx.x) * 2 + (u.tile == 0 ? 1 : 0)) * Cfg::PART;
        for (int i = threadIdx.x; i < rows * (D / 2); i += kAttnThreads) {
            const int r = i / (D / 2), d = 2 * (i % (D / 2));
            const float* from = reinterpret_cast<const float*>(smem) + r * Cfg::STRIDE;
            float2 md[kAttnWarps];
            float m = neg_inf(), total = 0.f;
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) {
                md[w] = *reinterpret_cast<const float2*>(from + w * Cfg::PART + D);
                m = fmaxf(m, md[w].x);
            }
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) {
                const float half = md[w].x == neg_inf() ? 0.f : exp2_fast(0.5f * (md[w].x - m)), e = half * half;
                const float2 v = *reinterpret_cast<const float2*>(from + w * Cfg::PART + d);
                sum.x = fmaf(v.x, e, sum.x);
                sum.y = fmaf(v.y, e, sum.y);
                total = fmaf(md[w].y * half, half, total);
            }
            if (whole) {
                store_out<T>(p, a, u.head, row0 + r, d, D, sum, total);
            } else {
                *reinterpret_cast<float2*>(part + r * Cfg::STRIDE + d) = sum;
                if (d == 0) *reinterpret_cast<float2*>(part + r * Cfg::STRIDE + D) = make_float2(m, total);
            }
        }
        fence_proxy_async_smem();  // the rings, read and written here, are filled by TMA again
        __syncthreads();
        w0 += end - u.tile;
        u.tile = 0;
        if (end == a.tiles && ++u.row_tile == a.row_tiles) {
            u.row_tile = 0;
            if (++u.head == p.c.heads) {
                u.head = 0;
                ++u.b;
            }
        }
    }
    if (!ok && elected) {
        // copies may still be in flight: give them a fixed time to land
        const uint64_t start = global_timer_ns();
        while (global_timer_ns() - start < 1000000) {
        }
    }
    pdl_launch_dependents();
}

// Joins the parts of a unit that CTA borders cut: CTA k takes the unit that border k
// (the start of piece k) cuts, if no earlier border cuts it too.  Only rows that exist are
// joined; the parts are spread over the threads, since a long sequence alone has 50 of them
// a unit and each is a load from the L2 away.
constexpr int kJoinThreads = 256;
constexpr int kJoinParts = 64;  // parts whose weights are held at a time

template <class T, int D, int NB>
__global__ void __launch_bounds__(kJoinThreads) k_kv8_attention_join(const AttnParams p) {
    using Cfg = AttnCfg<D, NB>;
    constexpr int ROWS = Cfg::ROWS;
    constexpr int LANES = D / 2;                      // threads across a row, two values each
    constexpr int SLICES = kJoinThreads / LANES;      // parts, or rows, at a time
    __shared__ int64_t mem[kJoinThreads / 32 + 2];
    __shared__ float weight[kJoinParts][ROWS];
    __shared__ float top[ROWS], total[ROWS];
    __shared__ float2 sums[SLICES][LANES];
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const int k = blockIdx.x + 1;
    const Kv8Place at =
        kv8_find<kJoinThreads>(p.bt.B, k, p.ctas, mem, [&](int b) { return attn_seq<NB>(p, b).work(p.c.heads); });
    const AttnUnit u = attn_unit<NB>(p, at);
    if (u.b >= p.bt.B || u.tile == 0) return;
    const AttnSeq a = attn_seq<NB>(p, u.b);
    const int64_t wk = at.total * k / p.ctas, u0 = wk - u.tile, u1 = u0 + a.tiles;
    auto border = [&](int i) { return at.total * i / p.ctas; };
    if (border(k - 1) > u0) return;
    // parts of pieces k - 1 .. last; a piece without tiles (fewer tiles than pieces) has none
    int last = static_cast<int>((u1 * p.ctas - 1) / at.total);
    while (last > k && border(last) >= u1) --last;
    while (last + 1 < p.ctas && border(last + 1) < u1) ++last;
    const bool dense = at.total >= p.ctas;
    auto part = [&](int cta) {
        return p.part + (static_cast<int64_t>(cta) * 2 + (cta < k ? 1 : 0)) * Cfg::PART;
    };
    const int rows = min(ROWS, a.rows - u.row_tile * ROWS), count = last - k + 2;
    // a row's largest M over its parts: 16 threads a row, those of the rows that exist
    {
        const int r = threadIdx.x / 16, j0 = threadIdx.x % 16;
        float m = neg_inf();
        for (int j = j0; j < count && r < rows; j += 16)
            if (dense || border(k + j) > border(k - 1 + j)) m = fmaxf(m, part(k - 1 + j)[r * Cfg::STRIDE + D]);
#pragma unroll
        for (int o = 8; o > 0; o /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (j0 == 0 && r < ROWS) {
            top[r] = m;
            total[r] = 0.f;
        }
    }
    const int slice = threadIdx.x / LANES, lane = threadIdx.x % LANES;
    // rows and slices of parts share the CTA's slices: one row at a time, or all slices a row
    float2 o[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) o[r] = make_float2(0.f, 0.f);
    for (int j0 = 0; j0 < count; j0 += kJoinParts) {
        const int n = min(kJoinParts, count - j0);
        __syncthreads();
        // thread (r, i): weights of parts i, i + 16, ... of row r, and their denominators
        const int r = threadIdx.x / 16, i0 = threadIdx.x % 16;
        float den = 0.f;
        for (int i = i0; i < n && r < rows; i += 16) {
            const int j = j0 + i;
            float e = 0.f;
            if (dense || border(k + j) > border(k - 1 + j)) {
                const float* f = part(k - 1 + j) + r * Cfg::STRIDE;
                const float half = f[D] == neg_inf() ? 0.f : exp2_fast(0.5f * (f[D] - top[r]));
                e = half * half;
                den = fmaf(f[D + 1] * half, half, den);
            }
            weight[i][r] = e;
        }
#pragma unroll
        for (int o2 = 8; o2 > 0; o2 /= 2) den += __shfl_xor_sync(0xffffffffu, den, o2);
        if (i0 == 0 && r < ROWS) total[r] += den;
        __syncthreads();
        for (int i = slice; i < n; i += SLICES) {
            if (!dense && border(k + j0 + i) == border(k - 1 + j0 + i)) continue;
            const float* f = part(k - 1 + j0 + i) + 2 * lane;
            float2 v[ROWS];  // all rows' loads ahead of their use
#pragma unroll
            for (int q = 0; q < ROWS; ++q)
                if (q < rows) v[q] = *reinterpret_cast<const float2*>(f + q * Cfg::STRIDE);
#pragma unroll
            for (int q = 0; q < ROWS; ++q)
                if (q < rows) {
                    o[q].x = fmaf(v[q].x, weight[i][q], o[q].x);
                    o[q].y = fmaf(v[q].y, weight[i][q], o[q].y);
                }
        }
    }
#pragma unroll
    for (int q = 0; q < ROWS; ++q) {
        if (q >= rows) break;
        __syncthreads();
        sums[slice][lane] = o[q];
        __syncthreads();
        if (slice == 0) {
            float2 v = sums[0][lane];
#pragma unroll
            for (int i = 1; i < SLICES; ++i) {
                v.x += sums[i][lane].x;
                v.y += sums[i][lane].y;
            }
            store_out<T>(p, a, u.head, u.row_tile * ROWS + q, 2 * lane, D, v, total[q]);
        }
    }
}

constexpr int kAttnCtas = 152 * 4;  // the most pieces (four CTAs an SM)

size_t kv8_attention_workspace(int64_t, int64_t, int64_t D) {
    const size_t few = static_cast<size_t>(kAttnCtas) * 2 * 16 * static_cast<size_t>(D + 2) * sizeof(float);
    const size_t many = D == 256 ? 0 : attention_rows_workspace(D);
    return few > many ? few : many;
}

// The cache's codes as pages * heads blocks of `page` rows of D bytes, boxes of 16 or 32 rows.
template <int D>
static int code_map(CUtensorMap* map, const int8_t* codes, const Kv8Cache& c) {
    constexpr int W = D < 128 ? D : 128;
    return make_tmap_3d_bytes(map, codes, D, 1 << c.page_log2, static_cast<int64_t>(c.pages) * c.heads, W,
                              c.page_log2 > 4 ? 32 : 16, W == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

template <class T, int D, int NB>
static int launch_attention(AttnParams p, int dev, cudaStream_t s) {
    struct Tag;
    int rc = raise_smem<Tag>(k_kv8_attention<T, D, NB>);
    if (rc) return rc;
    CUtensorMap k, v;
    rc = code_map<D>(&k, p.c.kq, p.c);
    if (!rc) rc = code_map<D>(&v, p.c.vq, p.c);
    if (rc) return rc;
    p.ctas = num_sms(dev) * AttnCfg<D, NB>::PER_SM;
    if (p.ctas > kAttnCtas) p.ctas = kAttnCtas;
    rc = launch_serialized(k_kv8_attention<T, D, NB>, dim3(static_cast<unsigned>(p.ctas)), kAttnThreads,
                           AttnCfg<D, NB>::SMEM, 1, s, k, v, p);
    if (rc || p.ctas == 1) return rc;
    return launch_serialized(k_kv8_attention_join<T, D, NB>, dim3(static_cast<unsigned>(p.ctas - 1)), kJoinThreads, 0, 1,
                             s, p);
}

// 8 rows a unit where that is all that a sequence has of a key head on average, else 16.  Next to prompts
// that go to the other kernel the rest may have fewer: 1024 tokens next to 63 single ones of 4 heads a key
// head would take 272 us with 8 (282), but 64 sequences of 8 tokens each 392 (248).
template <class T, int D>
static int attention_by_rows(const AttnParams& p, int dev, cudaStream_t s) {
    const int64_t rows = (static_cast<int64_t>(p.bt.rows) + p.bt.B - 1) / p.bt.B * p.group;
    return rows <= 8 ? launch_attention<T, D, 1>(p, dev, s) : launch_attention<T, D, 2>(p, dev, s);
}

template <class T>
static int attention_by_size(const AttnParams& p, int dev, cudaStream_t s) {
    if (p.c.D == 64) return attention_by_rows<T, 64>(p, dev, s);
    if (p.c.D == 128) return attention_by_rows<T, 128>(p, dev, s);
    return attention_by_rows<T, 256>(p, dev, s);
}

#define QG_ATTN_BUDGETS_NB(T, NAME, D, NB)                                                                           \
    QG_BLOCK_KERNEL_BUDGET("k_kv8_attention<" NAME "," #D "," #NB ">",                                               \
                           (reinterpret_cast<const void*>(k_kv8_attention<T, D, NB>)), kAttnThreads,                 \
                           (AttnCfg<D, NB>::SMEM), 0, 1, (AttnCfg<D, NB>::PER_SM));                                  \
    QG_BLOCK_KERNEL_BUDGET("k_kv8_attention_join<" NAME "," #D "," #NB ">",                                          \
                           (reinterpret_cast<const void*>(k_kv8_attention_join<T, D, NB>)), kJoinThreads, 0, 0, 1, 1)
#define QG_ATTN_BUDGETS(T, NAME, D)    \
    QG_ATTN_BUDGETS_NB(T, NAME, D, 1); \
    QG_ATTN_BUDGETS_NB(T, NAME, D, 2)
QG_ATTN_BUDGETS(__half, "f16", 64);
QG_ATTN_BUDGETS(__half, "f16", 128);
QG_ATTN_BUDGETS(__half, "f16", 256);
QG_ATTN_BUDGETS(__nv_bfloat16, "bf16", 64);
QG_ATTN_BUDGETS(__nv_bfloat16, "bf16", 128);
QG_ATTN_BUDGETS(__nv_bfloat16, "bf16", 256);

}  // namespace qg

using namespace qg;

extern "C" int kv8_attention(int dtype, int64_t B, int64_t rows, int64_t q_heads, int64_t heads, int64_t D,
                             const void* Q, int64_t ldq, const int8_t* kq, const int8_t* vq, const float* ks,
                             const float* vs, int64_t pages, int64_t page, const int32_t* table, int64_t table_cols,
                             const int32_t* starts, const int32_t* lengths, float scale, int causal, void* O,
                             int64_t ldo, void* ws, size_t ws_bytes, void* stream) {
    const NvtxRange nvtx_range("kv8_attention");
    if (dtype != QG_F16 && dtype != QG_BF16) return QG_ERR_UNSUPPORTED;
    const Kv8Args a = {const_cast<int8_t*>(kq), const_cast<int8_t*>(vq), const_cast<float*>(ks),
                       const_cast<float*>(vs), table, starts, lengths, B, rows, pages, page, heads, D, table_cols};
    int rc = check_kv8(a);
    if (rc) return rc;
    const float scale_log2 = scale * 1.44269504088896340736f;
    if (q_heads < 1 || q_heads % heads || q_heads > 65536 || rows * (q_heads / heads) > INT32_MAX - 256 ||
        !(scale_log2 - scale_log2 == 0.f))
        return QG_ERR_INVALID_ARG;
    if (B == 0 || rows == 0) return QG_OK;
    rc = check_kv8_rows(dtype, Q, ldq, q_heads * D, rows);
    if (!rc) rc = check_kv8_rows(dtype, O, ldo, q_heads * D, rows);
    if (rc) return rc;
    if (!ws || ws_bytes < kv8_attention_workspace(rows, q_heads, D)) return QG_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(ws) % 256) return QG_ERR_MISALIGNED;
    const int dev = current_device();
    if (dev < 0) return QG_ERR_CUDA;
    AttnParams p = {};
    kv8_params(a, &p.c, &p.bt);
    p.Q = Q; p.ldq = ldq; p.O = O; p.ldo = ldo;
    p.causal = causal != 0;
    const uintptr_t places = reinterpret_cast<uintptr_t>(Q) | static_cast<uintptr_t>(2 * ldq);
    p.q_align = places % 16 == 0 ? 16 : places % 8 == 0 ? 8 : 2;
    p.group = static_cast<int>(q_heads / heads);
    p.scale_log2 = scale_log2;
    p.part = static_cast<float*>(ws);
    p.ctl = host_ctl(dev);
    if (!p.ctl.status) return QG_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    p.from = attention_rows_from(p);
    if (p.from <= p.bt.rows * static_cast<int64_t>(p.group)) {
        rc = attention_rows(dtype, p, dev, s);
        if (rc || p.from == 1) return rc;
    }
    return dtype == QG_F16 ? attention_by_size<__half>(p, dev, s) : attention_by_size<__nv_bfloat16>(p, dev, s);
}
