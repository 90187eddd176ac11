// Attention over the paged 8-bit cache (kv8_common.cuh): few query rows a sequence.
//
//   x_j = scale log2(e) sk_j (q . kq_j)                      exponent of token j
//   O = sum_j 2^x_j sv_j vq_j / sum_j 2^x_j
//
// The codes go to the tensor cores as exact fp16 numbers, so a page's scales have to
// stay outside: sk is a factor of the product's result, and sv goes into the exponent,
//   w_j = 2^(x_j + log2 sv_j - M),   O = sum w_j vq_j / sum (w_j / sv_j),
// with M a running upper bound of x_j + log2 sv_j, so that w_j, rounded to fp16 for the
// second product, is at most 2^8 whatever the pages' scales are.  Sums, M and the
// denominator are fp32.  Queries go in as fp16 times a power of two of their row, which
// is exact for bf16 too but for values 2^-28 of the row's largest.
#include "kv8_common.cuh"
#include "kv8_host.h"

namespace qg {

// One warp takes 16 tokens a step, for 16 rows: the heads that share a key head, times a
// sequence's query rows.  All (sequence, key head, 16 rows) units' tiles of 64 tokens lie
// on one axis that the CTAs cut into equal pieces, wherever the units' borders are, so a
// batch of any lengths loads all SMs alike; a unit that several CTAs have parts of is
// joined by a second kernel from their fp32 sums.
constexpr int kAttnWarps = 4, kAttnThreads = 32 * kAttnWarps;
constexpr int kAttnRows = 16;
constexpr int kAttnTile = 16 * kAttnWarps;
constexpr int kAttnStages = 4;
constexpr float kLazy = 8.f;  // log2 of how far M may lag behind

struct AttnParams {
    Kv8Cache c;
    Kv8Batch bt;
    const void* Q;
    int64_t ldq;
    bool q_bf16, causal;
    int group;          // query heads a key head
    float scale_log2;   // scale * log2(e)
    void* O;
    int64_t ldo;
    float* part;        // 2 partial sums a CTA: kAttnRows x (D + 2)
    int ctas;
};

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float neg_inf() { return __uint_as_float(0xff800000u); }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Units and tiles of a sequence.
struct AttnSeq {
    Kv8Seq s;
    int rows, row_tiles, tiles;
    __device__ __forceinline__ int64_t work(int heads) const { return static_cast<int64_t>(heads) * row_tiles * tiles; }
};
__device__ __forceinline__ AttnSeq attn_seq(const AttnParams& p, int b) {
    AttnSeq a;
    a.s = kv8_seq(p.bt, p.c, b);
    a.rows = a.s.n * p.group;
    a.row_tiles = (a.rows + kAttnRows - 1) / kAttnRows;
    a.tiles = max(1, (a.s.len + kAttnTile - 1) / kAttnTile);
    return a;
}

// Where a CTA's piece of the axis starts.
struct AttnUnit {
    int b, head, row_tile;
    int64_t tile;
};
__device__ __forceinline__ AttnUnit attn_unit(const AttnParams& p, const Kv8Place& at) {
    AttnUnit u = {at.b, 0, 0, 0};
    if (at.b >= p.bt.B) return u;
    const AttnSeq a = attn_seq(p, at.b);
    const int64_t per_head = static_cast<int64_t>(a.row_tiles) * a.tiles;
    u.head = static_cast<int>(at.at / per_head);
    const int64_t rest = at.at - u.head * per_head;
    u.row_tile = static_cast<int>(rest / a.tiles);
    u.tile = rest % a.tiles;
    return u;
}

// Place of 16-byte piece `chunk` of token `t` of a warp's 16 in its stage: rows of D bytes,
// pieces exchanged so that neither K's reads (two tokens by four pieces) nor V's (four even
// tokens by two pieces, or by four halves) meet in a bank.
template <int D>
__device__ __forceinline__ int kv_place(int t, int chunk) {
    if constexpr (D == 64) {
        const int half = (t ^ (t >> 2)) & 1;
        return (t >> 1) * 128 + half * 64 + ((chunk ^ (t & 2)) << 4);
    } else {
        return t * D + ((chunk ^ (t & 6) ^ ((t & 1) << 2)) << 4);
    }
}

template <int D>
struct AttnCfg {
    static constexpr int CHUNKS = D / 16;               // 16-byte pieces of a token
    static constexpr int KV_BYTES = 16 * D;             // a warp's tokens of K, or V
    static constexpr int STAGE_BYTES = 2 * KV_BYTES + 16;  // and the two scales
    static constexpr int WARP_BYTES = kAttnStages * STAGE_BYTES;
    static constexpr int STRIDE = D + 2;                // floats of a row of partial sums: O, M, denominator
    static constexpr int SMEM = kAttnWarps * WARP_BYTES > kAttnWarps * kAttnRows * STRIDE * 4
                                    ? kAttnWarps * WARP_BYTES
                                    : kAttnWarps * kAttnRows * STRIDE * 4;
};

// 2^14 .. 2^15 over a row's largest magnitude (as bits), a power of two, and 1 over it.
struct RowPower {
    float up, down;
};
__device__ __forceinline__ RowPower row_power(uint32_t amax_bits) {
    int e = 268 - static_cast<int>(amax_bits >> 23);
    e = min(e, 253);
    return {__uint_as_float(static_cast<uint32_t>(e) << 23), __uint_as_float(static_cast<uint32_t>(254 - e) << 23)};
}

template <class T, int D>
__global__ void __launch_bounds__(kAttnThreads) k_kv8_attention(const AttnParams p) {
    using Cfg = AttnCfg<D>;
    constexpr int KS = D / 16;   // MMA steps of q . k
    constexpr int NT = D / 8;    // 8-column tiles of O
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int64_t mem[kAttnWarps + 2];
    pdl_wait_prior_grid();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const Kv8Place at = kv8_find<kAttnThreads>(p.bt.B, blockIdx.x, p.ctas, mem,
                                               [&](int b) { return attn_seq(p, b).work(p.c.heads); });
    int64_t w0 = at.total * blockIdx.x / p.ctas;
    const int64_t w1 = at.total * (blockIdx.x + 1) / p.ctas;
    AttnUnit u = attn_unit(p, at);
    uint8_t* const ring = smem + warp * Cfg::WARP_BYTES;
    const uint32_t ring_u32 = smem_u32(ring);
    const int page_log2 = p.c.page_log2;
    const int64_t page_bytes = static_cast<int64_t>(p.c.heads) * D << page_log2;

    while (w0 < w1 && u.b < p.bt.B) {
        const AttnSeq a = attn_seq(p, u.b);
        if (a.rows == 0) {  // a sequence without rows has no place on the axis
            u = {u.b + 1, 0, 0, 0};
            continue;
        }
        const int64_t end = min(static_cast<int64_t>(a.tiles), u.tile + (w1 - w0));
        // the two rows of this thread, g and g + 8 of the unit's 16
        int row[2], sees[2];
        const T* q[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            row[i] = u.row_tile * kAttnRows + g + 8 * i;
            const int token = row[i] / p.group;
            sees[i] = 0;
            q[i] = nullptr;
            if (row[i] < a.rows) {
                const int64_t upto = p.causal ? a.s.first + token + 1 : a.s.len;
                sees[i] = upto < 0 ? 0 : upto < a.s.len ? static_cast<int>(upto) : a.s.len;
                q[i] = static_cast<const T*>(p.Q) + (a.s.row0 + token) * p.ldq +
                       (u.head * p.group + row[i] % p.group) * D;
            }
        }
        // what any row of the unit sees, the same in all threads
        const int last_row = min(a.rows, (u.row_tile + 1) * kAttnRows) - 1;
        const int64_t most64 = p.causal ? a.s.first + last_row / p.group + 1 : a.s.len;
        const int most = most64 < 0 ? 0 : most64 < a.s.len ? static_cast<int>(most64) : a.s.len;

        // this warp's 16 tokens of tiles u.tile .. end that anyone sees
        const int t0 = static_cast<int>(u.tile) * kAttnTile + 16 * warp;
        const int t1 = min(most, static_cast<int>(end) * kAttnTile);
        const int steps = t1 > t0 ? (t1 - t0 + kAttnTile - 1) / kAttnTile : 0;
        int page_of = -1;  // of step (base + lane)
        int page_base = 0;
        auto fetch_pages = [&](int base) {
            page_base = base;
            const int step = base + lane;
            page_of = step < steps ? kv8_page(p.c, u.b, (t0 + step * kAttnTile) >> page_log2) : -1;
        };
        auto issue = [&](int step) {
            if (step < steps) {
                if (step >= page_base + 32) fetch_pages(step);
                const int number = __shfl_sync(0xffffffffu, page_of, step - page_base);
                const uint32_t st = ring_u32 + (step % kAttnStages) * Cfg::STAGE_BYTES;
                const int offset = (t0 + step * kAttnTile) & ((1 << page_log2) - 1);
                const int64_t from = (number < 0 ? 0 : number) * page_bytes +
                                     ((static_cast<int64_t>(u.head) << page_log2) + offset) * D;
#pragma unroll
                for (int i = lane; i < 16 * Cfg::CHUNKS; i += 32) {
                    const int t = i / Cfg::CHUNKS, chunk = i % Cfg::CHUNKS;
                    cp_async16(st + kv_place<D>(t, chunk), p.c.kq + from + t * D + 16 * chunk);
                    cp_async16(st + Cfg::KV_BYTES + kv_place<D>(t, chunk), p.c.vq + from + t * D + 16 * chunk);
                }
                if (number >= 0) {
                    const int64_t unit = static_cast<int64_t>(number) * p.c.heads + u.head;
                    if (lane < 2) cp_async4(st + 2 * Cfg::KV_BYTES + 4 * lane, (lane ? p.c.vs : p.c.ks) + unit);
                } else if (lane < 2) {
                    reinterpret_cast<uint32_t*>(ring + (step % kAttnStages) * Cfg::STAGE_BYTES + 2 * Cfg::KV_BYTES)[lane] =
                        0x7fc00000u;
                }
            }
            cp_async_commit();
        };
        fetch_pages(0);
#pragma unroll
        for (int i = 0; i < kAttnStages - 1; ++i) issue(i);

        // queries: lane c holds, for MMA step k, the four values that its 32-bit word of a
        // token's codes has in that step
        uint32_t qf[KS][4];
        float row_factor[2];
        {
            uint32_t bits[2] = {0u, 0u};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    const int d = (k / 4) * 64 + c * 16 + (k % 4) * 4;
#pragma unroll
                    for (int m = 0; m < 4; ++m)
                        if (q[i]) bits[i] = max(bits[i], abs_bits(to_f32<T>(q[i][d + m])));
                }
                bits[i] = max(bits[i], __shfl_xor_sync(0xffffffffu, bits[i], 1));
                bits[i] = max(bits[i], __shfl_xor_sync(0xffffffffu, bits[i], 2));
                const RowPower power = row_power(bits[i]);
                row_factor[i] = power.down * p.scale_log2;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    const int d = (k / 4) * 64 + c * 16 + (k % 4) * 4;
                    float f[4];
#pragma unroll
                    for (int m = 0; m < 4; ++m) f[m] = q[i] ? to_f32<T>(q[i][d + m]) * power.up : 0.f;
                    qf[k][i] = pack2<__half>(f[0], f[1]);
                    qf[k][i + 2] = pack2<__half>(f[2], f[3]);
                }
            }
        }

        float o[NT][4], M[2] = {neg_inf(), neg_inf()}, den[2] = {0.f, 0.f};
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][i] = 0.f;

        for (int step = 0; step < steps; ++step) {
            cp_async_wait<kAttnStages - 2>();
            __syncwarp();
            issue(step + kAttnStages - 1);
            const uint8_t* st = ring + (step % kAttnStages) * Cfg::STAGE_BYTES;
            const float sk = reinterpret_cast<const float*>(st + 2 * Cfg::KV_BYTES)[0];
            const float sv = reinterpret_cast<const float*>(st + 2 * Cfg::KV_BYTES)[1];
            // scores of 16 rows by 2 x 8 tokens
            float x[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
#pragma unroll
                for (int i = 0; i < 4; ++i) x[n][i] = 0.f;
#pragma unroll
                for (int k = 0; k < KS; k += 4) {
                    const uint4 w = *reinterpret_cast<const uint4*>(st + kv_place<D>(8 * n + g, (k / 4) * 4 + c));
                    const uint32_t word[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        uint32_t b0, b1;
                        s8_to_f16(word[m], b0, b1);
                        mma_f16(x[n], qf[k + m][0], qf[k + m][1], qf[k + m][2], qf[k + m][3], b0, b1);
                    }
                }
            }
            const int tok = t0 + step * kAttnTile + 2 * c;  // of x[0][0]; x[n][i] is 8 n + i % 2 on
            const float lsv = __log2f(sv), isv = __fdividef(1.f, sv);
            float top[2] = {neg_inf(), neg_inf()};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float f = row_factor[i] * sk;
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        float& v = x[n][2 * i + m];
                        v = tok + 8 * n + m < sees[i] ? fmaf(v, f, lsv) : neg_inf();
                        top[i] = fmaxf(top[i], v);
                    }
                top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
                top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
            }
            const bool moves = top[0] > M[0] + kLazy || top[1] > M[1] + kLazy || (M[0] == neg_inf() && top[0] > M[0]) ||
                               (M[1] == neg_inf() && top[1] > M[1]);
            if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float m = fmaxf(M[i], top[i]);
                    const float f = M[i] == neg_inf() ? 0.f : exp2_fast(M[i] - m);
                    M[i] = m;
                    den[i] *= f;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        o[n][2 * i] *= f;
                        o[n][2 * i + 1] *= f;
                    }
                }
            }
            uint32_t pf[4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float m = M[i] == neg_inf() ? 0.f : M[i];
                float sum = 0.f;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float e0 = exp2_fast(x[n][2 * i] - m), e1 = exp2_fast(x[n][2 * i + 1] - m);
                    sum += e0 + e1;
                    pf[2 * n + i] = pack2<__half>(e0, e1);
                }
                if (!(sum == 0.f)) den[i] = fmaf(sum, isv, den[i]);  // not 0 times a NaN of tokens that it does not see
            }
            // O += w . V: column g of tile n is value g D / 8 + n of a head; lane c's tokens are 2 c,
            // 2 c + 1, 2 c + 8 and 2 c + 9, whose bytes are brought together
            constexpr int PER = D / 8;  // values of a lane a token
            const uint8_t* sv8 = st + Cfg::KV_BYTES;
            uint32_t vw[4][PER / 4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int token = 2 * c + (t & 1) + 8 * (t >> 1);
                if constexpr (D == 64) {
                    const uint2 w = *reinterpret_cast<const uint2*>(sv8 + kv_place<D>(token, g >> 1) + 8 * (g & 1));
                    vw[t][0] = w.x;
                    vw[t][1] = w.y;
                } else {
#pragma unroll
                    for (int k = 0; k < PER / 16; ++k) {
                        const uint4 w = *reinterpret_cast<const uint4*>(sv8 + kv_place<D>(token, (PER / 16) * g + k));
                        vw[t][4 * k] = w.x;
                        vw[t][4 * k + 1] = w.y;
                        vw[t][4 * k + 2] = w.z;
                        vw[t][4 * k + 3] = w.w;
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < PER / 4; ++k) {
                // bytes of token pairs side by side, then as fp16 pairs
                uint32_t b[4][2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t lo = __byte_perm(vw[2 * h][k], vw[2 * h + 1][k], 0x5140);
                    const uint32_t hi = __byte_perm(vw[2 * h][k], vw[2 * h + 1][k], 0x7362);
                    s8_to_f16(lo, b[0][h], b[1][h]);
                    s8_to_f16(hi, b[2][h], b[3][h]);
                }
#pragma unroll
                for (int m = 0; m < 4; ++m) mma_f16(o[4 * k + m], pf[0], pf[1], pf[2], pf[3], b[m][0], b[m][1]);
            }
        }
        cp_async_wait<0>();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            den[i] += __shfl_xor_sync(0xffffffffu, den[i], 1);
            den[i] += __shfl_xor_sync(0xffffffffu, den[i], 2);
        }
        __syncthreads();  // the rings are free: partial sums of the warps go there
        float* mine = reinterpret_cast<float*>(smem) + warp * kAttnRows * Cfg::STRIDE;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float* r = mine + (g + 8 * i) * Cfg::STRIDE;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                // columns 2 c and 2 c + 1 of tile n: lanes' values (2 c) D / 8 + n
                r[(2 * c) * (D / 8) + n] = o[n][2 * i];
                r[(2 * c + 1) * (D / 8) + n] = o[n][2 * i + 1];
            }
            if (c == 0) {
                r[D] = M[i];
                r[D + 1] = den[i];
            }
        }
        __syncthreads();
        const bool whole = u.tile == 0 && end == a.tiles;
        float* part = p.part + (static_cast<int64_t>(blockIdx.x) * 2 + (u.tile == 0 ? 1 : 0)) * kAttnRows * Cfg::STRIDE;
        for (int i = threadIdx.x; i < kAttnRows * D; i += kAttnThreads) {
            const int r = i / D, d = i % D;
            const float* from = reinterpret_cast<const float*>(smem) + r * Cfg::STRIDE;
            float m = neg_inf(), sum = 0.f, total = 0.f;
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) m = fmaxf(m, from[w * kAttnRows * Cfg::STRIDE + D]);
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) {
                const float* f = from + w * kAttnRows * Cfg::STRIDE;
                const float e = f[D] == neg_inf() ? 0.f : exp2_fast(f[D] - m);
                sum = fmaf(f[d], e, sum);
                total = fmaf(f[D + 1], e, total);
            }
            if (whole) {
                const int rr = u.row_tile * kAttnRows + r;
                if (rr < a.rows) {
                    const float v = a.s.cut ? __uint_as_float(0x7fc00000u) : total == 0.f ? 0.f : sum / total;
                    static_cast<T*>(p.O)[(a.s.row0 + rr / p.group) * p.ldo + (u.head * p.group + rr % p.group) * D + d] =
                        from_f32<T>(v);
                }
            } else {
                part[r * Cfg::STRIDE + d] = sum;
                if (d == 0) {
                    part[r * Cfg::STRIDE + D] = m;
                    part[r * Cfg::STRIDE + D + 1] = total;
                }
            }
        }
        __syncthreads();  // the rings may be filled again
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
    pdl_launch_dependents();
}

// Joins the parts of a unit that CTA borders cut: CTA k takes the unit that border k
// (the start of piece k) cuts, if no earlier border cuts it too.  Only rows that exist are
// joined; the parts are spread over the threads, since a long sequence alone has 50 of them
// a unit and each is a load from the L2 away.
constexpr int kJoinThreads = 256;
constexpr int kJoinParts = 64;  // parts whose weights are held at a time

template <class T, int D>
__global__ void __launch_bounds__(kJoinThreads) k_kv8_attention_join(const AttnParams p) {
    using Cfg = AttnCfg<D>;
    constexpr int LANES = D / 2;                      // threads across a row, two values each
    constexpr int SLICES = kJoinThreads / LANES;      // parts, or rows, at a time
    __shared__ int64_t mem[kJoinThreads / 32 + 2];
    __shared__ float weight[kJoinParts][kAttnRows];
    __shared__ float top[kAttnRows], total[kAttnRows];
    __shared__ float2 sums[SLICES][LANES];
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const int k = blockIdx.x + 1;
    const Kv8Place at =
        kv8_find<kJoinThreads>(p.bt.B, k, p.ctas, mem, [&](int b) { return attn_seq(p, b).work(p.c.heads); });
    const AttnUnit u = attn_unit(p, at);
    if (u.b >= p.bt.B || u.tile == 0) return;
    const AttnSeq a = attn_seq(p, u.b);
    const int64_t wk = at.total * k / p.ctas, u0 = wk - u.tile, u1 = u0 + a.tiles;
    auto border = [&](int i) { return at.total * i / p.ctas; };
    if (border(k - 1) > u0) return;
    // parts of pieces k - 1 .. last; a piece without tiles (fewer tiles than pieces) has none
    int last = static_cast<int>((u1 * p.ctas - 1) / at.total);
    while (last > k && border(last) >= u1) --last;
    while (last + 1 < p.ctas && border(last + 1) < u1) ++last;
    const bool dense = at.total >= p.ctas;
    auto part = [&](int cta) {
        return p.part + (static_cast<int64_t>(cta) * 2 + (cta < k ? 1 : 0)) * kAttnRows * Cfg::STRIDE;
    };
    const int rows = min(kAttnRows, a.rows - u.row_tile * kAttnRows), count = last - k + 2;
    // a row's largest M over its parts: 16 threads a row
    {
        const int r = threadIdx.x / 16, j0 = threadIdx.x % 16;
        float m = neg_inf();
        for (int j = j0; j < count; j += 16)
            if (dense || border(k + j) > border(k - 1 + j)) m = fmaxf(m, part(k - 1 + j)[r * Cfg::STRIDE + D]);
#pragma unroll
        for (int o = 8; o > 0; o /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (j0 == 0) {
            top[r] = m;
            total[r] = 0.f;
        }
    }
    const int slice = threadIdx.x / LANES, lane = threadIdx.x % LANES;
    // rows and slices of parts share the CTA's slices: one row at a time, or all slices a row
    float2 o[kAttnRows];
#pragma unroll
    for (int r = 0; r < kAttnRows; ++r) o[r] = make_float2(0.f, 0.f);
    for (int j0 = 0; j0 < count; j0 += kJoinParts) {
        const int n = min(kJoinParts, count - j0);
        __syncthreads();
        // thread (r, i): weights of parts i, i + 16, ... of row r, and their denominators
        const int r = threadIdx.x / 16, i0 = threadIdx.x % 16;
        float den = 0.f;
        for (int i = i0; i < n; i += 16) {
            const int j = j0 + i;
            float e = 0.f;
            if (dense || border(k + j) > border(k - 1 + j)) {
                const float* f = part(k - 1 + j) + r * Cfg::STRIDE;
                e = f[D] == neg_inf() ? 0.f : exp2_fast(f[D] - top[r]);
                den = fmaf(f[D + 1], e, den);
            }
            weight[i][r] = e;
        }
#pragma unroll
        for (int o2 = 8; o2 > 0; o2 /= 2) den += __shfl_xor_sync(0xffffffffu, den, o2);
        if (i0 == 0) total[r] += den;
        __syncthreads();
        for (int i = slice; i < n; i += SLICES) {
            if (!dense && border(k + j0 + i) == border(k - 1 + j0 + i)) continue;
            const float* f = part(k - 1 + j0 + i) + 2 * lane;
            float2 v[kAttnRows];  // all rows' loads ahead of their use
#pragma unroll
            for (int q = 0; q < kAttnRows; ++q)
                if (q < rows) v[q] = *reinterpret_cast<const float2*>(f + q * Cfg::STRIDE);
#pragma unroll
            for (int q = 0; q < kAttnRows; ++q)
                if (q < rows) {
                    o[q].x = fmaf(v[q].x, weight[i][q], o[q].x);
                    o[q].y = fmaf(v[q].y, weight[i][q], o[q].y);
                }
        }
    }
#pragma unroll
    for (int q = 0; q < kAttnRows; ++q) {
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
            const int rr = u.row_tile * kAttnRows + q;
            const float t = total[q], nan = __uint_as_float(0x7fc00000u);
            T* out = static_cast<T*>(p.O) + (a.s.row0 + rr / p.group) * p.ldo +
                     (u.head * p.group + rr % p.group) * D + 2 * lane;
            out[0] = from_f32<T>(a.s.cut ? nan : t == 0.f ? 0.f : v.x / t);
            out[1] = from_f32<T>(a.s.cut ? nan : t == 0.f ? 0.f : v.y / t);
        }
    }
}

constexpr int kAttnCtas = 152 * 3;  // the most pieces (three CTAs an SM)

size_t kv8_attention_workspace(int64_t, int64_t, int64_t D) {
    return static_cast<size_t>(kAttnCtas) * 2 * kAttnRows * static_cast<size_t>(D + 2) * sizeof(float);
}

template <class T, int D>
static int launch_attention(AttnParams p, int dev, cudaStream_t s) {
    struct Tag;
    int rc = raise_smem<Tag>(k_kv8_attention<T, D>);
    if (rc) return rc;
    const int per_sm = D == 256 ? 1 : 3;
    p.ctas = num_sms(dev) * per_sm;
    if (p.ctas > kAttnCtas) p.ctas = kAttnCtas;
    rc = launch_serialized(k_kv8_attention<T, D>, dim3(static_cast<unsigned>(p.ctas)), kAttnThreads, AttnCfg<D>::SMEM, 1,
                           s, p);
    if (rc || p.ctas == 1) return rc;
    return launch_serialized(k_kv8_attention_join<T, D>, dim3(static_cast<unsigned>(p.ctas - 1)), kJoinThreads, 0, 1, s,
                             p);
}

template <class T>
static int attention_by_size(const AttnParams& p, int dev, cudaStream_t s) {
    if (p.c.D == 64) return launch_attention<T, 64>(p, dev, s);
    if (p.c.D == 128) return launch_attention<T, 128>(p, dev, s);
    return launch_attention<T, 256>(p, dev, s);
}

#define QG_ATTN_BUDGETS(T, NAME, D, PER)                                                                          \
    QG_BLOCK_KERNEL_BUDGET("k_kv8_attention<" NAME "," #D ">", (reinterpret_cast<const void*>(k_kv8_attention<T, D>)), \
                           kAttnThreads, AttnCfg<D>::SMEM, 0, 1, PER);                                            \
    QG_BLOCK_KERNEL_BUDGET("k_kv8_attention_join<" NAME "," #D ">",                                               \
                           (reinterpret_cast<const void*>(k_kv8_attention_join<T, D>)), kJoinThreads, 0, 0, 1, 1)
QG_ATTN_BUDGETS(__half, "f16", 64, 3);
QG_ATTN_BUDGETS(__half, "f16", 128, 3);
QG_ATTN_BUDGETS(__half, "f16", 256, 1);
QG_ATTN_BUDGETS(__nv_bfloat16, "bf16", 64, 3);
QG_ATTN_BUDGETS(__nv_bfloat16, "bf16", 128, 3);
QG_ATTN_BUDGETS(__nv_bfloat16, "bf16", 256, 1);

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
    if (q_heads < 1 || q_heads % heads || q_heads > 65536 || rows * (q_heads / heads) > INT32_MAX - 128 ||
        !(scale - scale == 0.f))
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
    p.group = static_cast<int>(q_heads / heads);
    p.scale_log2 = scale * 1.44269504088896340736f;
    p.part = static_cast<float*>(ws);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == QG_F16 ? attention_by_size<__half>(p, dev, s) : attention_by_size<__nv_bfloat16>(p, dev, s);
}
