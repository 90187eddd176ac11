// RMS norm of every head of Q and K and the rotation by position, forward and
// backward, one pass over the data each.
//
//   rstd = 1 / sqrt(sum(x^2) / D + eps),  z = x rstd g
//   y_a = z_a cos - z_b sin,  y_b = z_b cos + z_a sin    for R / 2 pairs (a, b)
//   y = z for the other D - R values of a head
// Pair i is (i, i + R / 2) or, PAIRS, (2 i, 2 i + 1); its cos and sin are values i and
// R / 2 + i of the table's row of the token's position.  Backward:
//   dz = the rotation by the negative angle of dy,  xh = x rstd,  e = dz g
//   dx = rstd (e - xh sum(e xh) / D),  dg = sum over tokens and heads of dz xh
//
// Bound by the bytes of x and y (and dy).  A few lanes hold a head, each 16 bytes of
// either side of its pairs, so that the rotation needs no exchange, and a lane keeps its
// place in the head over all heads of a token: cos, sin and g stay in registers.
#include "norm_common.cuh"

namespace qg {

constexpr int kRopeThreads = 128, kRopeWarps = kRopeThreads / 32;
constexpr int kRopeUnroll = 2;       // heads in flight a group of lanes
constexpr int64_t kRopeMaxD = 1024;
constexpr int kRopeMaxParts = 1024;  // rows of partial sums of either gain

// Q or K.
struct RopeJob {
    const void *X, *dY, *gain;
    void *Y;            // dX backward
    float* rstd;
    float* dgain;
    int64_t ldx, lddy, ldy;
    int heads;
};

struct RopeParams {
    RopeJob job[2];
    int blocks[2];       // CTAs of either job, Q's first
    int tokens, D, R;
    int lanes, rotating;             // lanes that hold a head, that rotate
    int group, group_log, step;      // lanes set aside for a head, a power of two; heads a warp
    int heads_per, splits[2];        // a warp takes heads_per heads of a token: parts of either job's
    uint64_t split_inv[2];           // floor(2^64 / splits) + 1, by which an item's token is found
    bool gain_f32;
    const int32_t* positions;
    const float* table;
    int table_rows;
    float eps;
    float* partial;      // backward: kRopeMaxParts x D for Q, then the same for K
};

__device__ __forceinline__ float group_sum(float v, int group) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (o < group) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Row of the table for a token; null outside the table.
__device__ __forceinline__ const float* table_row(const RopeParams& p, int token) {
    const int pos = p.positions ? p.positions[token] : token;
    return pos >= 0 && pos < p.table_rows ? p.table + static_cast<int64_t>(pos) * p.R : nullptr;
}

// Token of an item, the part of its heads in `part`.  Exact for items below 2^64 / splits.
__device__ __forceinline__ int token_of(const RopeParams& p, bool second, int64_t item, int& part) {
    const int splits = p.splits[second];
    const int token = static_cast<int>(splits == 1 ? item : __umul64hi(item, p.split_inv[second]));
    part = static_cast<int>(item) - token * splits;
    return token;
}

// What a lane holds of every head.
template <class T>
struct RopeLane {
    static constexpr int E = 16 / static_cast<int>(sizeof(T));  // values of a 16-byte piece
    int sub, l;       // which head of the warp's, which lane of it
    bool on, turns;
    int a, b;         // its two pieces' places in a head
    template <bool PAIRS>
    __device__ __forceinline__ void init(const RopeParams& p) {
        const int lane = threadIdx.x & 31;
        sub = lane >> p.group_log;
        l = lane & (p.group - 1);
        on = l < p.lanes;
        turns = l < p.rotating;
        a = PAIRS || !turns ? 2 * E * l : E * l;
        b = PAIRS || !turns ? a + E : p.R / 2 + E * l;
        if (!on) a = b = 0;
    }
    // cos and sin of its E pairs: (1, 0) where it does not rotate, NaN without a row
    __device__ __forceinline__ void angles(const RopeParams& p, const float* row, float (&c)[E], float (&s)[E]) const {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            c[i] = 1.f;
            s[i] = 0.f;
        }
        if (!on || !turns) return;
        if (row && ((p.R / 2) % 4 == 0) && aligned(p.table)) {
            load_vec<float, E>(row + E * l, c);
            load_vec<float, E>(row + p.R / 2 + E * l, s);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                c[i] = row ? row[E * l + i] : __uint_as_float(0x7fc00000u);
                s[i] = row ? row[p.R / 2 + E * l + i] : __uint_as_float(0x7fc00000u);
            }
        }
    }
    __device__ __forceinline__ static bool aligned(const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; }
    // its gains, piece a then piece b
    __device__ __forceinline__ void gains(const RopeParams& p, const void* gain, float (&g)[2 * E]) const {
        float ga[E], gb[E];
#pragma unroll
        for (int i = 0; i < E; ++i) ga[i] = gb[i] = 1.f;
        if (on && gain) {
            const bool vec = aligned(gain);
            if (p.gain_f32) {
                load_some<float, E>(static_cast<const float*>(gain) + a, E, vec, ga);
                load_some<float, E>(static_cast<const float*>(gain) + b, E, vec, gb);
            } else {
                load_some<T, E>(static_cast<const T*>(gain) + a, E, vec, ga);
                load_some<T, E>(static_cast<const T*>(gain) + b, E, vec, gb);
            }
        }
#pragma unroll
        for (int i = 0; i < E; ++i) {
            g[i] = ga[i];
            g[E + i] = gb[i];
        }
    }
};

// Pair i of 2 E values held in two pieces.
template <bool PAIRS, int E>
__device__ __forceinline__ constexpr int first_of(int i) { return PAIRS ? 2 * i : i; }
template <bool PAIRS, int E>
__device__ __forceinline__ constexpr int second_of(int i) { return PAIRS ? 2 * i + 1 : E + i; }

// The first and the second values of a lane's pairs, two pairs a register pair.
template <bool PAIRS, int E>
__device__ __forceinline__ void split_pairs(const float (&v)[2 * E], uint64_t (&a)[E / 2], uint64_t (&b)[E / 2]) {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
        a[i] = two(v[first_of<PAIRS, E>(2 * i)], v[first_of<PAIRS, E>(2 * i + 1)]);
        b[i] = two(v[second_of<PAIRS, E>(2 * i)], v[second_of<PAIRS, E>(2 * i + 1)]);
    }
}
template <bool PAIRS, int E>
__device__ __forceinline__ void join_pairs(const uint64_t (&a)[E / 2], const uint64_t (&b)[E / 2], float (&v)[2 * E]) {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
        const float2 x = both(a[i]), y = both(b[i]);
        v[first_of<PAIRS, E>(2 * i)] = x.x;
        v[first_of<PAIRS, E>(2 * i + 1)] = x.y;
        v[second_of<PAIRS, E>(2 * i)] = y.x;
        v[second_of<PAIRS, E>(2 * i + 1)] = y.y;
    }
}

template <class T>
__device__ __forceinline__ void widen(uint4 w, float* f) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            f[i] = __uint_as_float(v[i]);
        } else {
            const float2 x = unpack2<T>(v[i]);
            f[2 * i] = x.x;
            f[2 * i + 1] = x.y;
        }
    }
}
template <class T>
__device__ __forceinline__ uint4 narrow(const float* f) {
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4)
            v[i] = __float_as_uint(f[i]);
        else
            v[i] = pack2<T>(f[2 * i], f[2 * i + 1]);
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
}

// A warp takes heads_per heads of a token, U steps of as many as its lanes hold at most;
// their loads go out ahead of those of the gains and the table.  The hardware deals the
// CTAs out, which evens out what a loop over tokens left uneven.
//
// Measured: 8192 tokens of 40 heads of 128 bf16 values 35.7 us, 4.8 TB/s (71% of a copy).  A warp's
// life is the loads' latency and some 400 instructions, which the 28 warps that fit do not cover
// altogether; with four heads in flight a group of lanes instead of two there are fewer (38.6), and
// with 64 registers for 32 warps the loop spills.
template <class T, bool PAIRS>
__global__ void __launch_bounds__(kRopeThreads, 7) k_qk_norm_rope(const RopeParams p) {
    constexpr int E = RopeLane<T>::E, U = kRopeUnroll;
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const bool second = static_cast<int>(blockIdx.x) >= p.blocks[0];
    const RopeJob& j = p.job[second];
    const int64_t item = static_cast<int64_t>(blockIdx.x - (second ? p.blocks[0] : 0)) * kRopeWarps + (threadIdx.x >> 5);
    if (item >= static_cast<int64_t>(p.tokens) * p.splits[second]) return;
    int h0;
    const int token = token_of(p, second, item, h0);
    h0 *= p.heads_per;
    const int h1 = min(j.heads, h0 + p.heads_per);
    RopeLane<T> lane;
    lane.template init<PAIRS>(p);
    const int step = p.step, h = h0 + lane.sub;
    const T* x = static_cast<const T*>(j.X) + token * j.ldx;
    T* y = static_cast<T*>(j.Y) + token * j.ldy;
    uint4 wa[U], wb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        wa[u] = wb[u] = make_uint4(0, 0, 0, 0);
        if (lane.on && h + u * step < h1) {
            const T* at = x + (h + u * step) * p.D;
            wa[u] = *reinterpret_cast<const uint4*>(at + lane.a);
            wb[u] = *reinterpret_cast<const uint4*>(at + lane.b);
        }
    }
    // y_a = x_a (g_a cos) - x_b (g_b sin), y_b = x_b (g_b cos) + x_a (g_a sin), both times rstd
    uint64_t ac[E / 2], bs[E / 2], bc[E / 2], as[E / 2];
    {
        float c[E], s[E], g[2 * E];
        lane.angles(p, p.R ? table_row(p, token) : nullptr, c, s);
        lane.gains(p, j.gain, g);
        uint64_t ga[E / 2], gb[E / 2];
        split_pairs<PAIRS, E>(g, ga, gb);
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            const uint64_t cc = two(c[2 * i], c[2 * i + 1]), ss = two(s[2 * i], s[2 * i + 1]);
            ac[i] = mul_two(ga[i], cc);
            bc[i] = mul_two(gb[i], cc);
            as[i] = mul_two(ga[i], ss);
            bs[i] = mul_two(gb[i], two(-s[2 * i], -s[2 * i + 1]));
        }
    }
    const float inv_d = 1.f / static_cast<float>(p.D);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (h0 + u * step >= h1) break;  // the same for the whole warp
        float v[2 * E];
        widen<T>(wa[u], v);
        widen<T>(wb[u], v + E);
        uint64_t a[E / 2], b[E / 2], sq = two(0.f, 0.f);
        split_pairs<PAIRS, E>(v, a, b);
#pragma unroll
        for (int i = 0; i < E / 2; ++i) sq = fma_two(b[i], b[i], fma_two(a[i], a[i], sq));
        const float2 half = both(sq);
        const float rstd = rsqrtf(fmaf(group_sum(half.x + half.y, p.group), inv_d, p.eps));
        const uint64_t r2 = two(rstd, rstd);
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            const uint64_t za = mul_two(a[i], r2), zb = mul_two(b[i], r2);
            a[i] = fma_two(za, ac[i], mul_two(zb, bs[i]));
            b[i] = fma_two(zb, bc[i], mul_two(za, as[i]));
        }
        join_pairs<PAIRS, E>(a, b, v);
        const int head = h + u * step;
        if (lane.on && head < h1) {
            T* at = y + head * p.D;
            *reinterpret_cast<uint4*>(at + lane.a) = narrow<T>(v);
            *reinterpret_cast<uint4*>(at + lane.b) = narrow<T>(v + E);
            if (j.rstd && lane.l == 0) j.rstd[static_cast<int64_t>(token) * j.heads + head] = rstd;
        }
    }
}

// The gains' gradients stay in registers while a warp walks over its items, so the grid is what
// fits at once.  Measured: 8192 tokens of 40 heads of 128 bf16 values 49.5 us with the sum over
// the CTAs, 5.2 TB/s (77% of a copy); bound by latency with 16 warps an SM of 128 registers (four
// heads in flight spill: 74 us).
template <class T, bool PAIRS>
__global__ void __launch_bounds__(kRopeThreads, 4) k_qk_norm_rope_backward(const RopeParams p) {
    constexpr int E = RopeLane<T>::E, U = kRopeUnroll;
    __shared__ float sums[kRopeWarps][32][2 * E + 1];
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const bool second = static_cast<int>(blockIdx.x) >= p.blocks[0];
    const RopeJob& j = p.job[second];
    const int block = blockIdx.x - (second ? p.blocks[0] : 0), blocks = p.blocks[second];
    RopeLane<T> lane;
    lane.template init<PAIRS>(p);
    uint64_t ga[E / 2], gb[E / 2], dga[E / 2], dgb[E / 2];
    {
        float g[2 * E];
        lane.gains(p, j.gain, g);
        split_pairs<PAIRS, E>(g, ga, gb);
    }
#pragma unroll
    for (int i = 0; i < E / 2; ++i) dga[i] = dgb[i] = two(0.f, 0.f);
    const int step = p.step;
    const float inv_d = 1.f / static_cast<float>(p.D);
    const int64_t items = static_cast<int64_t>(p.tokens) * p.splits[second];
    for (int64_t item = block * kRopeWarps + (threadIdx.x >> 5); item < items; item += blocks * kRopeWarps) {
        int part;
        const int token = token_of(p, second, item, part), h0 = part * p.heads_per, h1 = min(j.heads, h0 + p.heads_per);
        const T* x = static_cast<const T*>(j.X) + token * j.ldx;
        const T* dy = static_cast<const T*>(j.dY) + token * j.lddy;
        T* dx = static_cast<T*>(j.Y) + token * j.ldy;
        const float* rs = j.rstd + static_cast<int64_t>(token) * j.heads;
        const int h = h0 + lane.sub;
        uint4 xa[U], xb[U], ya[U], yb[U];
        float r[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            xa[u] = xb[u] = ya[u] = yb[u] = make_uint4(0, 0, 0, 0);
            r[u] = 0.f;
            const int head = h + u * step;
            if (lane.on && head < h1) {
                xa[u] = *reinterpret_cast<const uint4*>(x + head * p.D + lane.a);
                xb[u] = *reinterpret_cast<const uint4*>(x + head * p.D + lane.b);
                ya[u] = *reinterpret_cast<const uint4*>(dy + head * p.D + lane.a);
                yb[u] = *reinterpret_cast<const uint4*>(dy + head * p.D + lane.b);
                r[u] = rs[head];
            }
        }
        float c[E], s[E];
        lane.angles(p, p.R ? table_row(p, token) : nullptr, c, s);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (h0 + u * step >= h1) break;
            // values of heads or lanes that are not there are 0, and so is what they add
            float v[2 * E], d[2 * E];
            widen<T>(xa[u], v);
            widen<T>(xb[u], v + E);
            widen<T>(ya[u], d);
            widen<T>(yb[u], d + E);
            uint64_t ha[E / 2], hb[E / 2], da[E / 2], db[E / 2], dot2 = two(0.f, 0.f);
            split_pairs<PAIRS, E>(v, ha, hb);
            split_pairs<PAIRS, E>(d, da, db);
            const uint64_t r2 = two(r[u], r[u]);
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                const uint64_t cc = two(c[2 * i], c[2 * i + 1]), ss = two(s[2 * i], s[2 * i + 1]);
                const uint64_t ns = two(-s[2 * i], -s[2 * i + 1]);
                const uint64_t za = fma_two(da[i], cc, mul_two(db[i], ss)), zb = fma_two(db[i], cc, mul_two(da[i], ns));
                ha[i] = mul_two(ha[i], r2);
                hb[i] = mul_two(hb[i], r2);
                dga[i] = fma_two(za, ha[i], dga[i]);
                dgb[i] = fma_two(zb, hb[i], dgb[i]);
                da[i] = mul_two(za, ga[i]);
                db[i] = mul_two(zb, gb[i]);
                dot2 = fma_two(db[i], hb[i], fma_two(da[i], ha[i], dot2));
            }
            const float2 half = both(dot2);
            const float dot = -group_sum(half.x + half.y, p.group) * inv_d;
            const int head = h + u * step;
            if (lane.on && head < h1) {
                const uint64_t dot_two = two(dot, dot);
#pragma unroll
                for (int i = 0; i < E / 2; ++i) {
                    da[i] = mul_two(r2, fma_two(ha[i], dot_two, da[i]));
                    db[i] = mul_two(r2, fma_two(hb[i], dot_two, db[i]));
                }
                join_pairs<PAIRS, E>(da, db, d);
                *reinterpret_cast<uint4*>(dx + head * p.D + lane.a) = narrow<T>(d);
                *reinterpret_cast<uint4*>(dx + head * p.D + lane.b) = narrow<T>(d + E);
            }
        }
    }
    // the CTA's sums, in the order of warps and heads
    {
        float dg[2 * E];
        join_pairs<PAIRS, E>(dga, dgb, dg);
#pragma unroll
        for (int i = 0; i < 2 * E; ++i) sums[threadIdx.x >> 5][threadIdx.x & 31][i] = dg[i];
    }
    __syncthreads();
    float* out = p.partial + (static_cast<int64_t>(second ? kRopeMaxParts : 0) + block) * p.D;
    for (int i = threadIdx.x; i < p.lanes * 2 * E; i += kRopeThreads) {
        const int l = i / (2 * E), v = i % (2 * E);
        float sum = 0.f;
        for (int w = 0; w < kRopeWarps; ++w)
            for (int h = 0; h < step; ++h) sum += sums[w][h * p.group + l][v];
        const bool turns = l < p.rotating;
        const int a = PAIRS || !turns ? 2 * E * l : E * l;
        out[v < E ? a + v : (PAIRS || !turns ? a + v : p.R / 2 + E * l + v - E)] = sum;
    }
}

// Heads whose pieces are not 16 bytes at 16-byte places: a warp takes a head, a lane
// every 32nd pair and every 32nd of the values that do not rotate; read twice.  Measured: 8192 tokens of
// 40 heads of 90 bf16 values 245 us, backward 437, where pieces would take some 26 and 36.
template <bool PAIRS>
__device__ __forceinline__ int slot_first(const RopeParams& p, int i) {  // i in [0, R / 2 + (D - R))
    return i >= p.R / 2 ? p.R / 2 + i : PAIRS ? 2 * i : i;
}
template <bool PAIRS>
__device__ __forceinline__ int slot_second(const RopeParams& p, int i) { return PAIRS ? 2 * i + 1 : p.R / 2 + i; }

template <class T, bool PAIRS, bool BACKWARD>
__global__ void __launch_bounds__(kRopeThreads) k_qk_norm_rope_any(const RopeParams p) {
    extern __shared__ float gain_sums[];  // BACKWARD: warps x D
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const bool second = static_cast<int>(blockIdx.x) >= p.blocks[0];
    const RopeJob& j = p.job[second];
    const int block = blockIdx.x - (second ? p.blocks[0] : 0), blocks = p.blocks[second];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int half = p.R / 2, slots = half + p.D - p.R;
    float* dg = gain_sums + warp * p.D;
    if constexpr (BACKWARD)
        for (int i = lane; i < slots; i += 32) {
            dg[slot_first<PAIRS>(p, i)] = 0.f;
            if (i < half) dg[slot_second<PAIRS>(p, i)] = 0.f;
        }
    const float nan = __uint_as_float(0x7fc00000u);
    const int64_t items = static_cast<int64_t>(p.tokens) * j.heads;
    for (int64_t item = block * kRopeWarps + warp; item < items; item += blocks * kRopeWarps) {
        const int token = static_cast<int>(item / j.heads), head = static_cast<int>(item % j.heads);
        const float* row = p.R ? table_row(p, token) : nullptr;
        const T* x = static_cast<const T*>(j.X) + token * j.ldx + head * p.D;
        const T* dy = BACKWARD ? static_cast<const T*>(j.dY) + token * j.lddy + head * p.D : nullptr;
        T* y = static_cast<T*>(j.Y) + token * j.ldy + head * p.D;
        auto gain = [&](int i) { return j.gain ? weight_at<T>(j.gain, p.gain_f32, i) : 1.f; };
        float sum = 0.f, rstd = BACKWARD ? j.rstd[item] : 0.f;
        for (int i = lane; i < slots; i += 32) {
            const int ia = slot_first<PAIRS>(p, i), ib = i < half ? slot_second<PAIRS>(p, i) : -1;
            const float xa = to_f32<T>(x[ia]), xb = ib >= 0 ? to_f32<T>(x[ib]) : 0.f;
            if constexpr (!BACKWARD) {
                sum = fmaf(xa, xa, fmaf(xb, xb, sum));
            } else {
                float da = to_f32<T>(dy[ia]), db = 0.f;
                if (ib >= 0) {
                    const float c = row ? row[i] : nan, s = row ? row[half + i] : nan, d0 = da, d1 = to_f32<T>(dy[ib]);
                    da = fmaf(d0, c, d1 * s);
                    db = fmaf(d1, c, -(d0 * s));
                    dg[ib] = fmaf(db, xb * rstd, dg[ib]);
                    sum = fmaf(db * gain(ib), xb * rstd, sum);
                }
                dg[ia] = fmaf(da, xa * rstd, dg[ia]);
                sum = fmaf(da * gain(ia), xa * rstd, sum);
            }
        }
        sum = warp_sum(sum);
        const float mean = sum / static_cast<float>(p.D);
        if constexpr (!BACKWARD) {
            rstd = rsqrtf(mean + p.eps);
            if (j.rstd && lane == 0) j.rstd[item] = rstd;
        }
        for (int i = lane; i < slots; i += 32) {
            const int ia = slot_first<PAIRS>(p, i), ib = i < half ? slot_second<PAIRS>(p, i) : -1;
            const float c = ib < 0 ? 1.f : row ? row[i] : nan, s = ib < 0 ? 0.f : row ? row[half + i] : nan;
            const float xa = to_f32<T>(x[ia]) * rstd, xb = ib >= 0 ? to_f32<T>(x[ib]) * rstd : 0.f;
            if constexpr (!BACKWARD) {
                const float za = xa * gain(ia), zb = ib >= 0 ? xb * gain(ib) : 0.f;
                y[ia] = from_f32<T>(fmaf(za, c, -(zb * s)));
                if (ib >= 0) y[ib] = from_f32<T>(fmaf(zb, c, za * s));
            } else {
                const float d0 = to_f32<T>(dy[ia]), d1 = ib >= 0 ? to_f32<T>(dy[ib]) : 0.f;
                const float da = fmaf(d0, c, d1 * s), db = fmaf(d1, c, -(d0 * s));
                y[ia] = from_f32<T>(rstd * fmaf(-xa, mean, da * gain(ia)));
                if (ib >= 0) y[ib] = from_f32<T>(rstd * fmaf(-xb, mean, db * gain(ib)));
            }
        }
    }
    if constexpr (BACKWARD) {
        __syncthreads();
        float* out = p.partial + (static_cast<int64_t>(second ? kRopeMaxParts : 0) + block) * p.D;
        for (int i = threadIdx.x; i < p.D; i += kRopeThreads) {
            float v = 0.f;
            for (int w = 0; w < kRopeWarps; ++w) v += gain_sums[w * p.D + i];
            out[i] = v;
        }
    }
}

// The gains' gradients: 32 columns a CTA, 32 slices of the rows each, added in order.
__global__ void __launch_bounds__(1024) k_rope_gains(const float* partial, int parts_q, int parts_k, int D, float* dgq,
                                                     float* dgk) {
    __shared__ float red[32][33];
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const bool second = blockIdx.y == 1;
    float* out = second ? dgk : dgq;
    if (!out) return;
    const float* src = partial + (second ? static_cast<int64_t>(kRopeMaxParts) * D : 0);
    const int parts = second ? parts_k : parts_q;
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), slice = threadIdx.x >> 5;
    float v = 0.f;
    if (col < D) {
#pragma unroll 8
        for (int i = slice; i < parts; i += 32) v += src[static_cast<int64_t>(i) * D + col];
    }
    red[slice][threadIdx.x & 31] = v;
    __syncthreads();
    if (slice == 0 && col < D) {
        v = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) v += red[i][threadIdx.x];
        out[col] = v;
    }
}

size_t rope_backward_workspace(int64_t D) { return 2 * sizeof(float) * kRopeMaxParts * static_cast<size_t>(D); }

// ------------------------------------------------------------ launches

static bool pieces_fit(const RopeJob& j, int64_t elem, bool backward) {
    if (!j.heads) return true;
    auto ok = [&](const void* q, int64_t ld) { return aligned16(q) && ld * elem % 16 == 0; };
    return ok(j.X, j.ldx) && ok(j.Y, j.ldy) && (!backward || ok(j.dY, j.lddy));
}

template <class T, bool PAIRS, bool BACKWARD>
static int launch_rope(RopeParams p, int dev, cudaStream_t s, int* parts) {
    const int64_t elem = sizeof(T);
    const int E = 16 / static_cast<int>(elem);
    const int heads = p.job[0].heads + p.job[1].heads;
    const bool pieces = p.D * elem % 16 == 0 && (p.D - p.R) % (2 * E) == 0 && p.R % (2 * E) == 0 && p.D / (2 * E) <= 32 &&
                        pieces_fit(p.job[0], elem, BACKWARD) && pieces_fit(p.job[1], elem, BACKWARD);
    const int64_t most = BACKWARD ? kRopeMaxParts : int64_t(1) << 20;
    // CTAs of a job that walks over its items: enough for them, at most its share of `full`
    const int64_t full = static_cast<int64_t>(num_sms(dev)) * (BACKWARD ? 4 : 8);
    auto share = [&](int i, int64_t items) -> int {
        if (!p.job[i].heads) return 0;
        const int64_t want = (items + kRopeWarps - 1) / kRopeWarps;
        int64_t part = full * p.job[i].heads / heads;
        part = part < 1 ? 1 : part > most ? most : part;
        return static_cast<int>(want < part ? want : part);
    };
    if (pieces) {
        p.lanes = p.D / (2 * E);
        p.rotating = p.R / (2 * E);
        p.group = 1;
        while (p.group < p.lanes) p.group *= 2, ++p.group_log;
        const int step = p.step = 32 / p.group;
        // heads of a token that a warp takes: as many as it has in flight, fewer where that
        // would leave SMs without warps
        p.heads_per = kRopeUnroll * step;
        while (p.heads_per > step && static_cast<int64_t>(p.tokens) * heads / p.heads_per < 4 * kRopeWarps * num_sms(dev))
            p.heads_per /= 2;
        for (int i = 0; i < 2; ++i) {
            p.splits[i] = (p.job[i].heads + p.heads_per - 1) / p.heads_per;
            p.split_inv[i] = p.splits[i] > 1 ? ~0ull / p.splits[i] + 1 : 0;
            const int64_t items = static_cast<int64_t>(p.tokens) * p.splits[i];
            parts[i] = p.blocks[i] = BACKWARD ? share(i, items) : static_cast<int>((items + kRopeWarps - 1) / kRopeWarps);
        }
        const dim3 grid(static_cast<unsigned>(p.blocks[0] + p.blocks[1]));
        if constexpr (BACKWARD)
            return launch_serialized(k_qk_norm_rope_backward<T, PAIRS>, grid, kRopeThreads, 0, 1, s, p);
        else
            return launch_serialized(k_qk_norm_rope<T, PAIRS>, grid, kRopeThreads, 0, 1, s, p);
    }
    for (int i = 0; i < 2; ++i) parts[i] = p.blocks[i] = share(i, static_cast<int64_t>(p.tokens) * p.job[i].heads);
    return launch_serialized(k_qk_norm_rope_any<T, PAIRS, BACKWARD>,
                             dim3(static_cast<unsigned>(p.blocks[0] + p.blocks[1])), kRopeThreads,
                             BACKWARD ? kRopeWarps * p.D * sizeof(float) : 0, 1, s, p);
}

template <bool BACKWARD>
static int rope_by_type(int dtype, int style, const RopeParams& p, int dev, cudaStream_t s, int* parts) {
    return by_dtype(dtype, [&](auto t) {
        return style ? launch_rope<decltype(t), true, BACKWARD>(p, dev, s, parts)
                     : launch_rope<decltype(t), false, BACKWARD>(p, dev, s, parts);
    });
}

static int check_rope(int dtype, int wdtype, int style, int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t R,
                      const int32_t* positions, const float* table, int64_t table_rows, const void* gq, const void* gk) {
    if (!dtype_ok(dtype) || (wdtype != dtype && wdtype != QG_F32)) return QG_ERR_UNSUPPORTED;
    if (style != QG_ROPE_HALF && style != QG_ROPE_PAIRS) return QG_ERR_UNSUPPORTED;
    if (T < 0 || T > (1 << 27) || Hq < 0 || Hk < 0 || Hq > 65536 || Hk > 65536 || D < 1 || R < 0 || R > D || R % 2)
        return QG_ERR_INVALID_ARG;
    if (D > kRopeMaxD) return QG_ERR_UNSUPPORTED;
    if (R && T && (!table || table_rows < 1 || table_rows > (int64_t(1) << 30))) return QG_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(positions) % 4 || reinterpret_cast<uintptr_t>(table) % 4) return QG_ERR_MISALIGNED;
    return check_weight(gq, wdtype) ? check_weight(gq, wdtype) : check_weight(gk, wdtype);
}

// Rows of H heads of D values, `ld` apart.
static int check_heads(int dtype, int64_t T, int64_t H, int64_t D, const void* X, int64_t ld) {
    if (H == 0) return QG_OK;
    if (!X || (T > 1 && ld < H * D)) return QG_ERR_INVALID_ARG;
    return reinterpret_cast<uintptr_t>(X) % dtype_bytes(dtype) ? QG_ERR_MISALIGNED : QG_OK;
}

static RopeParams rope_params(int64_t T, int64_t D, int64_t R, int wdtype, const int32_t* positions,
                              const float* table, int64_t table_rows, float eps) {
    RopeParams p = {};
    p.tokens = static_cast<int>(T);
    p.D = static_cast<int>(D);
    p.R = static_cast<int>(R);
    p.gain_f32 = wdtype == QG_F32;
    p.positions = positions;
    p.table = table;
    p.table_rows = static_cast<int>(table_rows);
    p.eps = eps;
    return p;
}

#define QG_ROPE_BUDGETS(T, NAME, PAIRS)                                                                             \
    QG_BLOCK_KERNEL_BUDGET("k_qk_norm_rope<" NAME "," #PAIRS ">",                                                   \
                           (reinterpret_cast<const void*>(k_qk_norm_rope<T, PAIRS>)), kRopeThreads, 0, 0, 1, 4);     \
    QG_BLOCK_KERNEL_BUDGET("k_qk_norm_rope_backward<" NAME "," #PAIRS ">",                                          \
                           (reinterpret_cast<const void*>(k_qk_norm_rope_backward<T, PAIRS>)), kRopeThreads, 0, 0,   \
                           1, 3);                                                                                   \
    QG_BLOCK_KERNEL_BUDGET("k_qk_norm_rope_any<" NAME "," #PAIRS ",false>",                                         \
                           (reinterpret_cast<const void*>(k_qk_norm_rope_any<T, PAIRS, false>)), kRopeThreads, 0, 0, \
                           1, 1);                                                                                   \
    QG_BLOCK_KERNEL_BUDGET("k_qk_norm_rope_any<" NAME "," #PAIRS ",true>",                                          \
                           (reinterpret_cast<const void*>(k_qk_norm_rope_any<T, PAIRS, true>)), kRopeThreads,        \
                           kRopeWarps * static_cast<int>(kRopeMaxD) * 4, 0, 1, 1)
QG_ROPE_BUDGETS(__half, "f16", false);
QG_ROPE_BUDGETS(__half, "f16", true);
QG_ROPE_BUDGETS(__nv_bfloat16, "bf16", false);
QG_ROPE_BUDGETS(__nv_bfloat16, "bf16", true);
QG_ROPE_BUDGETS(float, "f32", false);
QG_ROPE_BUDGETS(float, "f32", true);
QG_BLOCK_KERNEL_BUDGET("k_rope_gains", reinterpret_cast<const void*>(k_rope_gains), 1024, 0, 0, 1, 1);

}  // namespace qg

using namespace qg;

extern "C" {

int qk_norm_rope(int dtype, int style, int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t R, const void* Q,
                 int64_t ldq, const void* K, int64_t ldk, const void* gq, const void* gk, int wdtype,
                 const int32_t* positions, const float* table, int64_t table_rows, float eps, void* Yq, int64_t ldyq,
                 void* Yk, int64_t ldyk, float* rq, float* rk, void* stream) {
    const NvtxRange nvtx_range("qk_norm_rope");
    int rc = check_rope(dtype, wdtype, style, T, Hq, Hk, D, R, positions, table, table_rows, gq, gk);
    if (rc) return rc;
    if (!(eps >= 0.f)) return QG_ERR_INVALID_ARG;
    if (T == 0 || Hq + Hk == 0) return QG_OK;
    rc = check_heads(dtype, T, Hq, D, Q, ldq);
    if (!rc) rc = check_heads(dtype, T, Hk, D, K, ldk);
    if (!rc) rc = check_heads(dtype, T, Hq, D, Yq, ldyq);
    if (!rc) rc = check_heads(dtype, T, Hk, D, Yk, ldyk);
    if (!rc) rc = check_f32(rq);
    if (!rc) rc = check_f32(rk);
    if (rc) return rc;
    const int dev = current_device();
    if (dev < 0) return QG_ERR_CUDA;
    RopeParams p = rope_params(T, D, R, wdtype, positions, table, table_rows, eps);
    p.job[0] = {Q, nullptr, gq, Yq, rq, nullptr, ldq, 0, ldyq, static_cast<int>(Hq)};
    p.job[1] = {K, nullptr, gk, Yk, rk, nullptr, ldk, 0, ldyk, static_cast<int>(Hk)};
    int parts[2];
    return rope_by_type<false>(dtype, style, p, dev, static_cast<cudaStream_t>(stream), parts);
}

int qk_norm_rope_backward(int dtype, int style, int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t R,
                          const void* dYq, int64_t lddyq, const void* dYk, int64_t lddyk, const void* Q, int64_t ldq,
                          const void* K, int64_t ldk, const void* gq, const void* gk, int wdtype,
                          const int32_t* positions, const float* table, int64_t table_rows, const float* rq,
                          const float* rk, void* dQ, int64_t lddq, void* dK, int64_t lddk, float* dgq, float* dgk,
                          void* ws, size_t ws_bytes, void* stream) {
    const NvtxRange nvtx_range("qk_norm_rope_backward");
    int rc = check_rope(dtype, wdtype, style, T, Hq, Hk, D, R, positions, table, table_rows, gq, gk);
    if (rc) return rc;
    if (Hq + Hk == 0 && !dgq && !dgk) return QG_OK;
    if ((Hq && !dgq) || (Hk && !dgk)) return QG_ERR_INVALID_ARG;
    rc = check_f32(dgq);
    if (!rc) rc = check_f32(dgk);
    if (T > 0) {
        if ((Hq && !rq) || (Hk && !rk)) return QG_ERR_INVALID_ARG;
        if (!rc) rc = check_heads(dtype, T, Hq, D, Q, ldq);
        if (!rc) rc = check_heads(dtype, T, Hk, D, K, ldk);
        if (!rc) rc = check_heads(dtype, T, Hq, D, dYq, lddyq);
        if (!rc) rc = check_heads(dtype, T, Hk, D, dYk, lddyk);
        if (!rc) rc = check_heads(dtype, T, Hq, D, dQ, lddq);
        if (!rc) rc = check_heads(dtype, T, Hk, D, dK, lddk);
        if (!rc) rc = check_f32(rq);
        if (!rc) rc = check_f32(rk);
    }
    if (rc) return rc;
    if (!ws || ws_bytes < rope_backward_workspace(D)) return QG_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(ws) % 16) return QG_ERR_MISALIGNED;
    const int dev = current_device();
    if (dev < 0) return QG_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    RopeParams p = rope_params(T, D, R, wdtype, positions, table, table_rows, 0.f);
    p.job[0] = {Q, dYq, gq, dQ, const_cast<float*>(rq), dgq, ldq, lddyq, lddq, static_cast<int>(Hq)};
    p.job[1] = {K, dYk, gk, dK, const_cast<float*>(rk), dgk, ldk, lddyk, lddk, static_cast<int>(Hk)};
    p.partial = static_cast<float*>(ws);
    int parts[2] = {0, 0};  // none without tokens or heads: the gains' gradients are 0
    if (T > 0 && Hq + Hk > 0) {
        rc = rope_by_type<true>(dtype, style, p, dev, s, parts);
        if (rc) return rc;
    }
    return launch_serialized(k_rope_gains, dim3(static_cast<unsigned>((D + 31) / 32), 2), 1024, 0, 1, s,
                             static_cast<const float*>(p.partial), parts[0], parts[1], static_cast<int>(D),
                             dgq, dgk);
}

}  // extern "C"
