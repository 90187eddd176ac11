// Microscaled 4-bit quantizers: along the rows (fp4_quantize), along rows and
// columns in one pass (fp4_quantize_both), the tensor scale they may use
// (fp4_tensor_scale), and the way back to values (fp4_dequantize).  Formats,
// layout and the rounding rules: fp4_common.cuh.
#include "fp4_common.cuh"
#include "qg_ptx.cuh"

namespace qg {

// ------------------------------------------------------- along the rows
//
// One thread quantizes a block at a time: its 16 or 32 values come in 16-byte
// loads, the maximum and the codes stay in its registers, and the scale bytes
// of the four blocks of a scale tile's row go out as one word through two
// shuffles.  2^log_tx threads lie along a row (at least 4), the others of the
// CTA on further rows; a thread walks down the rows with the same column, so
// that addresses only advance.  Memory (2 or 4 bytes in, 0.56 or 0.53 out per
// value) would allow 13 us for 4096 x 8192 bf16; from cold caches it takes 20.9 us
// (86 MB, 4.1 TB/s): a thread loads, waits and computes in turn, waits for loads are
// the largest stall, and 44 % of an SM's warps do not cover them (DRAM 43 % busy).
// Few instructions a value still count: maxima are found on packed words, the
// factors of the 128 scale bytes lie in a table, and divisions are left to the few
// scales next to a rounding boundary.
constexpr int kQuantThreads = 256;

template <int FMT, class T>
__global__ void __launch_bounds__(kQuantThreads)
    k_fp4_quantize(int64_t M, int64_t rows, int64_t K, int log_tx, const T* X, int64_t ldx,
                   const float* tscale, uint8_t* __restrict__ Xq, uint8_t* __restrict__ Xs) {
    constexpr int B = fp4_block(FMT);
    __shared__ float factors[128];
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const TensorScale ts = tensor_scale(FMT == kNv ? tscale : nullptr);
    if constexpr (FMT == kNv) {
        fill_factors(factors, ts.ts);
        __syncthreads();
    }
    const int tx = 1 << log_tx, ty = kQuantThreads >> log_tx;
    const int64_t tiles = fp4_col_tiles(FMT, K), ld = fp4_codes_ld(K);
    const int64_t blk = static_cast<int64_t>(blockIdx.y) * tx + (threadIdx.x & (tx - 1));
    if (blk >= 4 * tiles) return;  // tx >= 4: groups of 4 lanes leave together
    const int64_t k0 = blk * B;
    const bool some = k0 < K, codes_here = k0 < 2 * ld;
    const int n = static_cast<int>(min(K - k0, int64_t(B)));
    const uint32_t quad = 0xfu << (threadIdx.x & 28);
    const int64_t step = static_cast<int64_t>(gridDim.x) * ty;
    int64_t row = static_cast<int64_t>(blockIdx.x) * ty + (threadIdx.x >> log_tx);
    const T* x = X + row * ldx + k0;
    uint8_t* q = Xq + row * ld + k0 / 2;
    uint8_t* const s0 = Xs + (blk >> 2) * 512;
    // U rows' blocks are on their way before the first is quantized
    constexpr int W = B * static_cast<int>(sizeof(T)) / 4, U = 32 / W;
    for (; row < rows; row += U * step) {
        uint32_t w[U][W];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (some && row + u * step < M) {
                load_words<T, B>(x, n, true, w[u]);
            } else {
#pragma unroll
                for (int i = 0; i < W; ++i) w[u][i] = 0;  // also a block behind K
            }
            x += step * ldx;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t here = row + u * step;
            if (U > 1 && here >= rows) break;  // groups of 4 lanes alike
            uint32_t byte = 0;
            if (here < M && codes_here) {
                uint32_t codes[B / 8];
                byte = quantize_words<FMT, T>(w[u], ts, factors, codes);
                if constexpr (B == 16)
                    *reinterpret_cast<uint2*>(q) = make_uint2(codes[0], codes[1]);
                else
                    *reinterpret_cast<uint4*>(q) = make_uint4(codes[0], codes[1], codes[2], codes[3]);
            }
            q += step * ld;
            uint32_t word = byte << (8 * (threadIdx.x & 3));
            word |= __shfl_xor_sync(quad, word, 1);
            word |= __shfl_xor_sync(quad, word, 2);
            const uint32_t r = static_cast<uint32_t>(here) & 127u;
            if ((threadIdx.x & 3) == 0)
                *reinterpret_cast<uint32_t*>(s0 + (here >> 7) * tiles * 512 + (r & 31u) * 16 + (r >> 5) * 4) = word;
        }
    }
}

// Rows whose addresses are not 16-byte aligned: a warp takes eight blocks of
// four rows.  Its loads are of one value a lane, neighbours in neighbouring lanes
// and all on their way at once; shared memory (rows of an odd number of words,
// so no two lanes meet in a bank) hands each thread a block to quantize as above.
// Read value by value a block a thread, 777 x 1333 fp32 took 7 us; with one value
// a lane to the end, its maxima and codes put together with eight shuffles, 9 us;
// this way 3.1 us.
template <int FMT, class T>
__global__ void __launch_bounds__(kQuantThreads)
    k_fp4_quantize_lanes(int64_t M, int64_t rows, int64_t K, const T* X, int64_t ldx,
                         const float* tscale, uint8_t* __restrict__ Xq, uint8_t* __restrict__ Xs) {
    constexpr int B = fp4_block(FMT), COLS = 8 * B, LOADS = COLS / 32;
    __shared__ float staged[kQuantThreads][B + 1];
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const TensorScale ts = tensor_scale(FMT == kNv ? tscale : nullptr);
    const int lane = threadIdx.x & 31;
    float (*const mine)[B + 1] = staged + (threadIdx.x & ~31);
    const int64_t tiles = fp4_col_tiles(FMT, K), ld = fp4_codes_ld(K);
    const int64_t groups = (tiles + 1) / 2;  // of eight blocks along a row
    const int64_t units = groups * ((rows + 3) / 4);
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kQuantThreads / 32);
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * (kQuantThreads / 32) + (threadIdx.x >> 5); i < units; i += warps) {
        const int64_t row0 = i / groups * 4, k0 = i % groups * COLS;
        float v[4][LOADS];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const T* const x = X + (row0 + r) * ldx;
#pragma unroll
            for (int j = 0; j < LOADS; ++j) {
                const int64_t k = k0 + 32 * j + lane;
                v[r][j] = row0 + r < M && k < K ? to_f32<T>(x[k]) : 0.f;
            }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int j = 0; j < LOADS; ++j) {
                const int c = 32 * j + lane;
                mine[8 * r + c / B][c % B] = v[r][j];
            }
        __syncwarp();
        float x[B];
#pragma unroll
        for (int c = 0; c < B; ++c) x[c] = mine[lane][c];
        __syncwarp();  // read before the next blocks overwrite it
        uint32_t codes[B / 8];
        uint32_t word = quantize_block<FMT>(x, ts, codes) << (8 * (lane & 3));
        const int64_t row = row0 + (lane >> 3), k = k0 + (lane & 7) * B;
        if (row < M && k < 2 * ld) {
            uint8_t* const q = Xq + row * ld + k / 2;
            if constexpr (B == 16)
                *reinterpret_cast<uint2*>(q) = make_uint2(codes[0], codes[1]);
            else
                *reinterpret_cast<uint4*>(q) = make_uint4(codes[0], codes[1], codes[2], codes[3]);
        }
        word |= __shfl_xor_sync(0xffffffffu, word, 1);
        word |= __shfl_xor_sync(0xffffffffu, word, 2);
        if ((lane & 3) == 0 && row < rows && k < tiles * (4 * B))
            *reinterpret_cast<uint32_t*>(Xs + fp4_scale_offset(row, k / B, tiles)) = word;
    }
}

// ------------------------------------------------------- rows and columns
//
// A CTA takes a tile of 128 x 128 values once and quantizes it along both axes:
// X (blocks along a row) and X^T (blocks along a column), as a training step
// needs an operand once for each of its two products.  Rows are quantized from
// the registers of the load, columns from shared memory, two of a 16-bit type
// at a time.  Codes of X^T and all scales are put together in shared memory
// and leave in 16-byte pieces.  The tile also gives the column sums (the bias
// gradient).  Memory (2 or 4 bytes in, 1.12 or 1.06 out per value) would allow
// 15.7 us for 8192 x 4096 bf16; it takes 27 to 29 us (mx 25): each value is quantized
// twice, the tile crosses shared memory once each way, and a CTA loads, waits and
// computes in turn.
constexpr int kBothThreads = 256;
constexpr int kTile = 128;

template <int FMT, class T>
struct BothSmem {
    static constexpr int B = fp4_block(FMT), NB = kTile / B;   // blocks along an axis of the tile
    // words a row of the tile: odd, so that a warp along a row and one down a
    // column both meet distinct banks
    static constexpr int PITCH = kTile * static_cast<int>(sizeof(T)) / 4 + 1;
    static constexpr int SCALES = NB / 4 * 512;                // of one direction
    static constexpr int CODES_PITCH = kTile / 2 + 16;         // bytes a row of X^T's codes
    static constexpr int TILE_BYTES = (kTile * PITCH * 4 + 15) / 16 * 16;
    static constexpr int BYTES = TILE_BYTES + kTile * CODES_PITCH + 2 * SCALES + NB * kTile * 4 + 512;
};

template <int FMT, class T>
__global__ void __launch_bounds__(kBothThreads)
    k_fp4_quantize_both(uint32_t first_tile, int64_t M, int64_t K, const T* X, int64_t ldx, bool aligned,
                        const float* tscale, uint8_t* __restrict__ Xq, uint8_t* __restrict__ Xs,
                        uint8_t* __restrict__ Tq, uint8_t* __restrict__ Ts, float* __restrict__ partial) {
    using S = BothSmem<FMT, T>;
    constexpr int B = S::B, NB = S::NB, PITCH = S::PITCH, W = B * static_cast<int>(sizeof(T)) / 4;
    extern __shared__ __align__(16) uint8_t both_smem[];
    uint32_t* const tile = reinterpret_cast<uint32_t*>(both_smem);
    uint8_t* const tcodes = both_smem + S::TILE_BYTES;
    uint8_t* const rscales = tcodes + kTile * S::CODES_PITCH;
    uint8_t* const tscales = rscales + S::SCALES;
    float* const sums = reinterpret_cast<float*>(tscales + S::SCALES);  // [NB][kTile]
    float* const factors = sums + NB * kTile;
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const uint32_t tile_m = first_tile + blockIdx.y;
    const int64_t m0 = static_cast<int64_t>(tile_m) * kTile, k0 = static_cast<int64_t>(blockIdx.x) * kTile;
    const TensorScale ts = tensor_scale(FMT == kNv ? tscale : nullptr);
    if constexpr (FMT == kNv) {
        fill_factors(factors, ts.ts);
        __syncthreads();
    }
    const int64_t ldq = fp4_codes_ld(K), ldt = fp4_codes_ld(M);
    // place of (row, block) in this tile's scale tiles
    auto scale_at = [](int r, int b) { return (b >> 2) * 512 + (r & 31) * 16 + (r >> 5) * 4 + (b & 3); };

    // the tile, zero outside X, and the blocks along its rows.  Aligned rows are
    // loaded a block a thread (U at a time, before the first is quantized);
    // others into the tile first, one value a lane and 16 rows of a warp in flight
    constexpr int ITERS = kTile * NB / kBothThreads, U = 32 / W < ITERS ? 32 / W : ITERS;
    if (!aligned) {
        T* const values = reinterpret_cast<T*>(tile);
        constexpr int PER_WARP = kTile / (kBothThreads / 32), LANE_PITCH = PITCH * 4 / static_cast<int>(sizeof(T));
        const int lane = threadIdx.x & 31, first = (threadIdx.x >> 5) * PER_WARP;
#pragma unroll 1
        for (int c = lane; c < kTile; c += 32) {
            T v[PER_WARP];
#pragma unroll
            for (int j = 0; j < PER_WARP; ++j)
                v[j] = m0 + first + j < M && k0 + c < K ? X[(m0 + first + j) * ldx + k0 + c] : from_f32<T>(0.f);
#pragma unroll
            for (int j = 0; j < PER_WARP; ++j) values[(first + j) * LANE_PITCH + c] = v[j];
        }
        __syncthreads();
    }
#pragma unroll 1
    for (int i0 = 0; i0 < ITERS; i0 += U) {
        uint32_t w[U][W];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = (i0 + u) * kBothThreads + threadIdx.x, m = i / NB, b = i % NB;
            const int64_t k = k0 + b * B;
            if (!aligned) {
#pragma unroll
                for (int j = 0; j < W; ++j) w[u][j] = tile[m * PITCH + b * W + j];
            } else if (m0 + m < M && k < K) {
                load_words<T, B>(X + (m0 + m) * ldx + k, static_cast<int>(min(K - k, int64_t(B))), true, w[u]);
            } else {
#pragma unroll
                for (int j = 0; j < W; ++j) w[u][j] = 0;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = (i0 + u) * kBothThreads + threadIdx.x, m = i / NB, b = i % NB;
            const int64_t k = k0 + b * B;
            if (aligned) {
#pragma unroll
                for (int j = 0; j < W; ++j) tile[m * PITCH + b * W + j] = w[u][j];
            }
            if (Xq) {
                uint32_t codes[B / 8];
                rscales[scale_at(m, b)] = static_cast<uint8_t>(quantize_words<FMT, T>(w[u], ts, factors, codes));
                if (m0 + m < M && k < 2 * ldq) {
                    uint8_t* q = Xq + (m0 + m) * ldq + k / 2;
                    if constexpr (B == 16)
                        *reinterpret_cast<uint2*>(q) = make_uint2(codes[0], codes[1]);
                    else
                        *reinterpret_cast<uint4*>(q) = make_uint4(codes[0], codes[1], codes[2], codes[3]);
                }
            }
        }
    }
    __syncthreads();

    // blocks along the columns: 32-bit words, that is one or two columns a thread
    constexpr int PER = 4 / static_cast<int>(sizeof(T)), COLS = kTile / PER;
    for (int i = threadIdx.x; i < COLS * NB; i += kBothThreads) {
        const int c = i % COLS, b = i / COLS;  // a warp's lanes on neighbouring words
        uint32_t v[B];
#pragma unroll
        for (int j = 0; j < B; ++j) v[j] = tile[(b * B + j) * PITCH + c];
#pragma unroll
        for (int h = 0; h < PER; ++h) {
            uint32_t w[W], codes[B / 8];
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < W; ++j) {
                if constexpr (PER == 1) {
                    w[j] = v[j];
                    sum += __uint_as_float(w[j]);
                } else {
                    w[j] = __byte_perm(v[2 * j], v[2 * j + 1], h ? 0x7632 : 0x5410);
                    const float2 f = unpack2<typename std::conditional<PER == 1, __half, T>::type>(w[j]);
                    sum += f.x + f.y;
                }
            }
            const int k = PER * c + h;
            if (Tq) {
                tscales[scale_at(k, b)] = static_cast<uint8_t>(quantize_words<FMT, T>(w, ts, factors, codes));
                uint8_t* q = tcodes + k * S::CODES_PITCH + b * (B / 2);
                if constexpr (B == 16)
                    *reinterpret_cast<uint2*>(q) = make_uint2(codes[0], codes[1]);
                else
                    *reinterpret_cast<uint4*>(q) = make_uint4(codes[0], codes[1], codes[2], codes[3]);
            }
            if (partial) sums[b * kTile + k] = sum;
        }
    }
    __syncthreads();

    if (Tq) {
        // rows of 64 bytes, four threads each; ldt is a multiple of 16 bytes
#pragma unroll
        for (int i = threadIdx.x; i < kTile * 4; i += kBothThreads) {
            const int k = i / 4, piece = i % 4;
            const int64_t at = m0 / 2 + 16 * piece;
            if (k0 + k < K && at < ldt)
                *reinterpret_cast<uint4*>(Tq + (k0 + k) * ldt + at) =
                    *reinterpret_cast<const uint4*>(tcodes + k * S::CODES_PITCH + 16 * piece);
        }
    }
    // whole scale tiles; values outside X were 0, so their scales are
    constexpr int PIECES = S::SCALES / 16;
    for (int i = threadIdx.x; i < 2 * PIECES; i += kBothThreads) {
        const bool t = i >= PIECES;
        const int j = t ? i - PIECES : i;
        uint8_t* const out = t ? Ts : Xs;
        const int64_t tiles = fp4_col_tiles(FMT, t ? M : K);
        const int64_t col = (t ? m0 : k0) / (4 * B) + j / 32;
        if (out && col < tiles)
            *reinterpret_cast<uint4*>(out + ((t ? k0 : m0) / 128 * tiles + col) * 512 + j % 32 * 16) =
                *reinterpret_cast<const uint4*>((t ? tscales : rscales) + 16 * j);
    }
    if (partial && threadIdx.x < kTile && k0 + threadIdx.x < K) {
        float sum = sums[threadIdx.x];
#pragma unroll
        for (int b = 1; b < NB; ++b) sum += sums[b * kTile + threadIdx.x];
        partial[tile_m * K + k0 + threadIdx.x] = sum;
    }
}

// ------------------------------------------------------- tensor scale
//
// ts = max(fl(amax fl(1 / 2688)), 2^-100) over the finite values, 1 where all are 0:
// 2688 = 6 * 448, so the largest value of the tensor lands on the largest
// code times the largest block scale.  Each CTA leaves its maximum in the
// workspace and one more warp joins them (a maximum does not depend on the
// order); bound by reading X once (8192 x 4096 bf16: 15.6 us, 4.3 TB/s).
constexpr int kAmaxThreads = 512;
constexpr int kAmaxMaxCtas = 1024;

__device__ __forceinline__ uint32_t finite_abs_bits(float v) {
    const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
    return b >= 0x7f800000u ? 0u : b;
}

template <class T>
__global__ void __launch_bounds__(kAmaxThreads)
    k_fp4_amax(int64_t M, int64_t K, const T* X, int64_t ldx, bool aligned,
               uint32_t* __restrict__ part) {
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const int64_t per_row = (K + V - 1) / V, step = static_cast<int64_t>(gridDim.x) * kAmaxThreads;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kAmaxThreads + threadIdx.x;
    // one pass over the thread's share, four loads in flight; without `finite`
    // infinities and NaN count as what their bits are, above all else
    auto share = [&](auto finite) {
        uint32_t m = 0;
        for (int64_t row = blockIdx.y; row < M; row += gridDim.y) {
            const T* const x = X + row * ldx;
            for (int64_t i = first; i < per_row; i += 4 * step) {
                uint32_t w[4][4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int64_t k = (i + u * step) * V;
                    load_words<T, V>(x + k, static_cast<int>(max(int64_t(0), min(K - k, int64_t(V)))), aligned, w[u]);
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if constexpr (sizeof(T) == 4) {
                            const uint32_t v = w[u][j] & 0x7fffffffu;
                            m = max(m, decltype(finite)::value ? finite_abs_bits(__uint_as_float(v)) : v);
                        } else if constexpr (decltype(finite)::value) {
                            const float2 f = unpack2<T>(w[u][j]);
                            m = max(m, max(finite_abs_bits(f.x), finite_abs_bits(f.y)));
                        } else {
                            m = __vmaxu2(m, w[u][j] & 0x7fff7fffu);
                        }
                    }
                }
            }
        }
        if constexpr (sizeof(T) == 2 && !decltype(finite)::value) m = packed_amax_bits<T>(m);
        return m;
    };
    uint32_t m = share(std::false_type{});
    if (m >= 0x7f800000u) m = share(std::true_type{});
    m = __reduce_max_sync(0xffffffffu, m);
    __shared__ uint32_t wm[kAmaxThreads / 32];
    if ((threadIdx.x & 31) == 0) wm[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x < 32) {
        m = threadIdx.x < kAmaxThreads / 32 ? wm[threadIdx.x] : 0u;
        m = __reduce_max_sync(0xffffffffu, m);
        if (threadIdx.x == 0) part[blockIdx.y * gridDim.x + blockIdx.x] = m;
    }
}

__global__ void __launch_bounds__(32) k_fp4_scale_join(const uint32_t* part, int parts,
                                                       float* __restrict__ scale) {
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    uint32_t m = 0;
    for (int i = threadIdx.x; i < parts; i += 32) m = max(m, part[i]);
    m = __reduce_max_sync(0xffffffffu, m);
    if (threadIdx.x == 0)
        *scale = m ? fmaxf(__fmul_rn(__uint_as_float(m), 1.f / 2688.f), 0x1p-100f) : 1.f;
}

// ------------------------------------------------------- back to values

// One thread takes 16 values a step and walks down the rows, as above; its two
// 16-byte stores are one of 32 bytes where rows are aligned to that.  Bound by
// memory (0.56 or 0.53 bytes in, 2 or 4 out per value): 4096 x 8192 to bf16 in
// 16.8 us (5.1 TB/s).
constexpr int kDequantThreads = 256;

template <int FMT, class T>
__global__ void __launch_bounds__(kDequantThreads)
    k_fp4_dequantize(int64_t M, int64_t K, int log_tx, const uint8_t* Xq, const uint8_t* Xs,
                     const float* tscale, T* __restrict__ Y, int64_t ldy, bool sectors) {
    constexpr int B = fp4_block(FMT);
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const int tx = 1 << log_tx, ty = kDequantThreads >> log_tx;
    const int64_t k = (static_cast<int64_t>(blockIdx.y) * tx + (threadIdx.x & (tx - 1))) * 16;
    if (k >= K) return;
    const float ts = FMT == kNv && tscale ? *tscale : 1.f;
    const int n = static_cast<int>(min(K - k, int64_t(16)));
    const int64_t step = static_cast<int64_t>(gridDim.x) * ty, ld = fp4_codes_ld(K);
    const int64_t tiles = fp4_col_tiles(FMT, K), blk = k / B;
    int64_t row = static_cast<int64_t>(blockIdx.x) * ty + (threadIdx.x >> log_tx);
    const uint8_t* q = Xq + row * ld + k / 2;
    const uint8_t* const s0 = Xs + (blk >> 2) * 512 + (blk & 3);
    T* y = Y + row * ldy + k;
#pragma unroll 2
    for (; row < M; row += step, q += step * ld, y += step * ldy) {
        const uint2 c = *reinterpret_cast<const uint2*>(q);
        const uint32_t r = static_cast<uint32_t>(row) & 127u;
        const uint32_t byte = s0[(row >> 7) * tiles * 512 + (r & 31u) * 16 + (r >> 5) * 4];
        const float d = __fmul_rn(scale_value<FMT>(byte), ts);
        float lo[8], hi[8], x[16];
        e2m1x8_values(c.x, lo);
        e2m1x8_values(c.y, hi);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = __fmul_rn(lo[i], d);
            x[8 + i] = __fmul_rn(hi[i], d);
        }
        if (sectors && n == 16)
            store_sectors(y, x);
        else
            store_some<T, 16>(y, n, true, x);
    }
}

// The same into rows that are not 16-byte aligned: a warp takes 128 values of
// four rows, each thread makes 16 of them, and shared memory turns them so that
// a store is of one value a lane, neighbours in neighbouring lanes.  (One value a
// lane to the end, each with its own code and scale read: 6.7 us for 777 x 1333
// into fp32, against 2.7 us.)
template <int FMT, class T>
__global__ void __launch_bounds__(kDequantThreads)
    k_fp4_dequantize_lanes(int64_t M, int64_t K, const uint8_t* Xq, const uint8_t* Xs,
                           const float* tscale, T* __restrict__ Y, int64_t ldy) {
    constexpr int B = fp4_block(FMT);
    __shared__ float staged[kDequantThreads][17];
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const float ts = FMT == kNv && tscale ? *tscale : 1.f;
    const int lane = threadIdx.x & 31;
    float (*const mine)[17] = staged + (threadIdx.x & ~31);
    const int64_t tiles = fp4_col_tiles(FMT, K), ld = fp4_codes_ld(K);
    const int64_t groups = (K + 127) / 128, units = groups * ((M + 3) / 4);
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kDequantThreads / 32);
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * (kDequantThreads / 32) + (threadIdx.x >> 5); i < units; i += warps) {
        const int64_t row0 = i / groups * 4, k0 = i % groups * 128;
        const int64_t row = row0 + (lane >> 3), k = k0 + (lane & 7) * 16;
        if (row < M && k < K) {
            const uint2 c = *reinterpret_cast<const uint2*>(Xq + row * ld + k / 2);
            const float d = __fmul_rn(scale_value<FMT>(Xs[fp4_scale_offset(row, k / B, tiles)]), ts);
            float lo[8], hi[8];
            e2m1x8_values(c.x, lo);
            e2m1x8_values(c.y, hi);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                mine[lane][j] = __fmul_rn(lo[j], d);
                mine[lane][8 + j] = __fmul_rn(hi[j], d);
            }
        }
        __syncwarp();
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            T* const y = Y + (row0 + r) * ldy;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = 32 * j + lane;
                if (row0 + r < M && k0 + c < K) y[k0 + c] = from_f32<T>(mine[8 * r + c / 16][c % 16]);
            }
        }
        __syncwarp();  // read before the next values overwrite it
    }
}

// ------------------------------------------------------- host side

static bool rows_aligned(const void* p, int64_t ld, size_t elem, int64_t rows) {
    return aligned16(p) && (rows <= 1 || (static_cast<size_t>(ld) * elem) % 16 == 0);
}

// Cut of a kernel whose threads walk down the rows: 2^log_tx threads along a
// row, grid.y over the row, and in grid.x CTAs for `per_sm` an SM: whole rounds of
// those that are resident at once, and never one more.  The quantizer's four are
// so busy that two rounds do (4096 x 8192 bf16: 20.9 us; 22.0 with two CTAs above
// them, 22.2 with a round and a half); the way back, whose rounds are of loads and
// stores alone, gains from more (eight 19.3 us, twelve 17.4, sixteen 16.8).
struct Walk {
    int log_tx;
    dim3 grid;
};
static Walk walk(int64_t rows, int64_t per_row, int threads, int per_sm) {
    Walk w;
    w.log_tx = 2;
    while (w.log_tx < 8 && (int64_t(1) << w.log_tx) < per_row) ++w.log_tx;
    const int64_t ty = threads >> w.log_tx;
    const int64_t gy = (per_row + (int64_t(1) << w.log_tx) - 1) >> w.log_tx;
    const int64_t share = int64_t(per_sm) * num_sms(current_device()) / gy, most = share > 1 ? share : 1;
    const int64_t gx = (rows + ty - 1) / ty;
    w.grid = dim3(static_cast<unsigned>(gx < most ? gx : most), static_cast<unsigned>(gy));
    return w;
}

// Cut of a kernel whose warps take units of four rows: six CTAs an SM.
static dim3 unit_grid(int64_t rows, int64_t groups, int threads) {
    const int64_t ctas = (groups * ((rows + 3) / 4) + threads / 32 - 1) / (threads / 32);
    const int64_t most = 6 * num_sms(current_device());
    return dim3(static_cast<unsigned>(ctas < most ? ctas : most));
}

int fp4_quantize_run(int fmt, int dtype, int64_t M, int64_t K, const void* X, int64_t ldx, const float* ts,
                     uint8_t* Xq, uint8_t* Xs, bool zero_pad, cudaStream_t s) {
    const int64_t rows = zero_pad ? (M + 127) / 128 * 128 : M;
    const int64_t per_row = 4 * fp4_col_tiles(fmt, K);
    if (rows == 0 || per_row == 0) return QG_OK;
    const Walk w = walk(rows, per_row, kQuantThreads, 8);
    return by_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        const bool al = rows_aligned(X, ldx, sizeof(T), M);
        if (!al) {
            auto* f = fmt == kNv ? k_fp4_quantize_lanes<kNv, T> : k_fp4_quantize_lanes<kMx, T>;
            return launch_serialized(f, unit_grid(rows, (per_row + 7) / 8, kQuantThreads), kQuantThreads, 0, 1, s,
                                     M, rows, K, static_cast<const T*>(X), ldx, ts, Xq, Xs);
        }
        auto* f = fmt == kNv ? k_fp4_quantize<kNv, T> : k_fp4_quantize<kMx, T>;
        return launch_serialized(f, w.grid, kQuantThreads, 0, 1, s, M, rows, K, w.log_tx, static_cast<const T*>(X), ldx,
                                 ts, Xq, Xs);
    });
}

template <int FMT, class T>
static int launch_both(dim3 grid, uint32_t first_tile, int64_t M, int64_t K, const void* X, int64_t ldx, const float* ts,
                       uint8_t* Xq, uint8_t* Xs, uint8_t* Tq, uint8_t* Ts, float* partial, cudaStream_t s) {
    constexpr int SMEM = BothSmem<FMT, T>::BYTES;
    auto* f = k_fp4_quantize_both<FMT, T>;
    struct Flags {};
    const int rc = raise_smem<Flags>(f);
    if (rc) return rc;
    return launch_serialized(f, grid, kBothThreads, SMEM, 1, s, first_tile, M, K, static_cast<const T*>(X), ldx,
                             rows_aligned(X, ldx, sizeof(T), M), ts, Xq, Xs, Tq, Ts, partial);
}

int fp4_quantize_both_run(int fmt, int dtype, int64_t M, int64_t K, const void* X, int64_t ldx, const float* ts,
                          uint8_t* Xq, uint8_t* Xs, uint8_t* Tq, uint8_t* Ts, float* colsum, float* partial,
                          cudaStream_t s) {
    const int64_t tiles_k = (K + kTile - 1) / kTile, tiles_m = (M + kTile - 1) / kTile;
    int rc = QG_OK;
    // as many tiles of rows a launch as a grid's y counts
    for (int64_t first = 0; !rc && tiles_k && first < tiles_m; first += kMaxGridY) {
        const int64_t gy = tiles_m - first < kMaxGridY ? tiles_m - first : kMaxGridY;
        const dim3 grid(static_cast<unsigned>(tiles_k), static_cast<unsigned>(gy));
        const uint32_t at = static_cast<uint32_t>(first);
        rc = by_dtype(dtype, [&](auto t) {
            using T = decltype(t);
            float* const part = colsum ? partial : nullptr;
            return fmt == kNv ? launch_both<kNv, T>(grid, at, M, K, X, ldx, ts, Xq, Xs, Tq, Ts, part, s)
                              : launch_both<kMx, T>(grid, at, M, K, X, ldx, ts, Xq, Xs, Tq, Ts, part, s);
        });
    }
    if (rc || !colsum) return rc;
    return sum_partials_run(partial, tiles_m, K, colsum, s);
}

// CTAs along a row and over the rows: the two an SM that are resident at once (8192 x
// 4096 bf16: 15.6 us; 16.7 with 512 CTAs on 152 SMs), each thread with 4 loads.
static dim3 amax_grid(int64_t M, int64_t K, size_t elem) {
    const int64_t pieces = (K * static_cast<int64_t>(elem) + 15) / 16;
    int64_t x = (pieces + 4 * kAmaxThreads - 1) / (4 * kAmaxThreads);
    const int64_t two = 2 * num_sms(current_device()), most = two < kAmaxMaxCtas ? two : kAmaxMaxCtas;
    x = x < 1 ? 1 : x > most ? most : x;
    int64_t y = most / x;
    y = M < 1 ? 1 : y > M ? M : y;
    return dim3(static_cast<unsigned>(x), static_cast<unsigned>(y));
}

#define QG_FP4_BUDGETS(T, NAME)                                                                              \
    QG_BLOCK_KERNEL_BUDGET("k_fp4_quantize_lanes<nv," NAME ">", reinterpret_cast<const void*>(k_fp4_quantize_lanes<kNv, T>), \
                           kQuantThreads, 0, 0, 1, 4);                                                       \
    QG_BLOCK_KERNEL_BUDGET("k_fp4_quantize_lanes<mx," NAME ">", reinterpret_cast<const void*>(k_fp4_quantize_lanes<kMx, T>), \
                           kQuantThreads, 0, 0, 1, 4);                                                       \
    QG_BLOCK_KERNEL_BUDGET("k_fp4_quantize<nv," NAME ">", reinterpret_cast<const void*>(k_fp4_quantize<kNv, T>), \
                           kQuantThreads, 0, 0, 1, 2);                                                       \
    QG_BLOCK_KERNEL_BUDGET("k_fp4_quantize<mx," NAME ">", reinterpret_cast<const void*>(k_fp4_quantize<kMx, T>), \
                           kQuantThreads, 0, 0, 1, 4);                                                       \
    QG_BLOCK_KERNEL_BUDGET("k_fp4_quantize_both<nv," NAME ">",                                               \
                           reinterpret_cast<const void*>(k_fp4_quantize_both<kNv, T>), kBothThreads,         \
                           (BothSmem<kNv, T>::BYTES), 0, 1, 2);                                              \
    QG_BLOCK_KERNEL_BUDGET("k_fp4_quantize_both<mx," NAME ">",                                               \
                           reinterpret_cast<const void*>(k_fp4_quantize_both<kMx, T>), kBothThreads,         \
                           (BothSmem<kMx, T>::BYTES), 0, 1, 2);                                              \
    QG_BLOCK_KERNEL_BUDGET("k_fp4_amax<" NAME ">", reinterpret_cast<const void*>(k_fp4_amax<T>), kAmaxThreads, \
                           0, 0, 1, 2);                                                                      \
    QG_BLOCK_KERNEL_BUDGET("k_fp4_dequantize_lanes<nv," NAME ">", reinterpret_cast<const void*>(k_fp4_dequantize_lanes<kNv, T>), \
                           kDequantThreads, 0, 0, 1, 4);                                                       \
    QG_BLOCK_KERNEL_BUDGET("k_fp4_dequantize_lanes<mx," NAME ">", reinterpret_cast<const void*>(k_fp4_dequantize_lanes<kMx, T>), \
                           kDequantThreads, 0, 0, 1, 4);                                                       \
    QG_BLOCK_KERNEL_BUDGET("k_fp4_dequantize<nv," NAME ">",                                                  \
                           reinterpret_cast<const void*>(k_fp4_dequantize<kNv, T>), kDequantThreads, 0, 0, 1, 4); \
    QG_BLOCK_KERNEL_BUDGET("k_fp4_dequantize<mx," NAME ">",                                                  \
                           reinterpret_cast<const void*>(k_fp4_dequantize<kMx, T>), kDequantThreads, 0, 0, 1, 4)
QG_FP4_BUDGETS(__half, "f16");
QG_FP4_BUDGETS(__nv_bfloat16, "bf16");
QG_FP4_BUDGETS(float, "f32");
QG_BLOCK_KERNEL_BUDGET("k_fp4_scale_join", reinterpret_cast<const void*>(k_fp4_scale_join), 32, 0, 0, 1, 1);

}  // namespace qg

using namespace qg;

constexpr int64_t kMaxCols = int64_t(1) << 27;  // grid.y covers a row

// Checks shared by the calls that read a rows x K matrix of floating type.
static int check_matrix(int fmt, int dtype, int64_t M, int64_t K, const void* X, int64_t ldx) {
    if (!fmt_ok(fmt) || !dtype_ok(dtype)) return QG_ERR_UNSUPPORTED;
    if (M < 0 || K < 0 || M > INT32_MAX || K > kMaxCols) return QG_ERR_INVALID_ARG;
    if (M && K && !X) return QG_ERR_INVALID_ARG;
    if (M > 1 && ldx < K) return QG_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(X) % dtype_bytes(dtype)) return QG_ERR_MISALIGNED;
    return QG_OK;
}

static int check_scale(int fmt, const float* ts) {
    if (ts && fmt == kMx) return QG_ERR_UNSUPPORTED;  // the power-of-two format has no tensor scale
    if (reinterpret_cast<uintptr_t>(ts) % 4) return QG_ERR_MISALIGNED;
    return QG_OK;
}

extern "C" {

int64_t qg_fp4_codes_ld(int64_t K) { return K > 0 ? fp4_codes_ld(K) : 0; }

size_t qg_fp4_scale_bytes(int fmt, int64_t rows, int64_t K) {
    if (!fmt_ok(fmt) || rows <= 0 || K <= 0) return 0;
    return static_cast<size_t>(fp4_scale_bytes(fmt, rows, K));
}

int fp4_tensor_scale(int dtype, int64_t M, int64_t K, const void* X, int64_t ldx, float* scale, void* ws,
                     size_t ws_bytes, void* stream) {
    const NvtxRange nvtx_range("fp4_tensor_scale");
    int rc = check_matrix(kNv, dtype, M, K, X, ldx);
    if (rc) return rc;
    if (!scale) return QG_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(scale) % 4) return QG_ERR_MISALIGNED;
    if (!ws || ws_bytes < qg_workspace_size(QG_OP_FP4_TENSOR_SCALE, 1, 1, 1)) return QG_ERR_WORKSPACE;
    if (!aligned16(ws)) return QG_ERR_MISALIGNED;
    if (current_device() < 0) return QG_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int64_t m = M, k = K;
    if (ldx == K || M <= 1) {  // rows end to end: one long row
        k = M * K;
        m = k ? 1 : 0;
    }
    const dim3 grid = amax_grid(m, k, dtype_bytes(dtype));
    const int ctas = static_cast<int>(grid.x * grid.y);
    uint32_t* part = static_cast<uint32_t*>(ws);
    rc = by_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        return launch_serialized(k_fp4_amax<T>, grid, kAmaxThreads, 0, 1, s, m, k,
                                 static_cast<const T*>(X), ldx, rows_aligned(X, ldx, sizeof(T), m), part);
    });
    if (rc) return rc;
    return launch_serialized(k_fp4_scale_join, dim3(1), 32, 0, 1, s, part, ctas, scale);
}

int fp4_quantize(int fmt, int dtype, int64_t M, int64_t K, const void* X, int64_t ldx, const float* tscale,
                 uint8_t* Xq, uint8_t* Xs, void* stream) {
    const NvtxRange nvtx_range("fp4_quantize");
    int rc = check_matrix(fmt, dtype, M, K, X, ldx);
    if (!rc) rc = check_scale(fmt, tscale);
    if (rc) return rc;
    if (M == 0 || K == 0) return QG_OK;
    if (!Xq || !Xs) return QG_ERR_INVALID_ARG;
    if (!aligned16(Xq) || !aligned16(Xs)) return QG_ERR_MISALIGNED;
    if (current_device() < 0) return QG_ERR_CUDA;
    return fp4_quantize_run(fmt, dtype, M, K, X, ldx, tscale, Xq, Xs, true, static_cast<cudaStream_t>(stream));
}

int fp4_quantize_both(int fmt, int dtype, int64_t M, int64_t K, const void* X, int64_t ldx, const float* tscale,
                      uint8_t* Xq, uint8_t* Xs, uint8_t* Tq, uint8_t* Ts, void* stream) {
    const NvtxRange nvtx_range("fp4_quantize_both");
    int rc = check_matrix(fmt, dtype, M, K, X, ldx);
    if (!rc) rc = check_scale(fmt, tscale);
    if (rc) return rc;
    if ((Xq == nullptr) != (Xs == nullptr)) return QG_ERR_INVALID_ARG;
    if (M == 0 || K == 0) return QG_OK;
    if (!Tq || !Ts) return QG_ERR_INVALID_ARG;
    if (!aligned16(Xq) || !aligned16(Xs) || !aligned16(Tq) || !aligned16(Ts)) return QG_ERR_MISALIGNED;
    if (current_device() < 0) return QG_ERR_CUDA;
    return fp4_quantize_both_run(fmt, dtype, M, K, X, ldx, tscale, Xq, Xs, Tq, Ts, nullptr, nullptr,
                                 static_cast<cudaStream_t>(stream));
}

int fp4_dequantize(int fmt, int dtype, int64_t M, int64_t K, const uint8_t* Xq, const uint8_t* Xs,
                   const float* tscale, void* Y, int64_t ldy, void* stream) {
    const NvtxRange nvtx_range("fp4_dequantize");
    int rc = check_matrix(fmt, dtype, M, K, Y, ldy);
    if (!rc) rc = check_scale(fmt, tscale);
    if (rc) return rc;
    if (M == 0 || K == 0) return QG_OK;
    if (!Xq || !Xs) return QG_ERR_INVALID_ARG;
    if (!aligned16(Xq) || !aligned16(Xs)) return QG_ERR_MISALIGNED;
    if (current_device() < 0) return QG_ERR_CUDA;
    const Walk w = walk(M, (K + 15) / 16, kDequantThreads, 16);
    return by_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        auto* f = fmt == kNv ? k_fp4_dequantize<kNv, T> : k_fp4_dequantize<kMx, T>;
        if (!rows_aligned(Y, ldy, sizeof(T), M)) {
            auto* g = fmt == kNv ? k_fp4_dequantize_lanes<kNv, T> : k_fp4_dequantize_lanes<kMx, T>;
            return launch_serialized(g, unit_grid(M, (K + 127) / 128, kDequantThreads), kDequantThreads, 0, 1,
                                     static_cast<cudaStream_t>(stream), M, K, Xq, Xs, tscale, static_cast<T*>(Y), ldy);
        }
        const bool sectors = (reinterpret_cast<uintptr_t>(Y) & 31u) == 0 &&
                             (M <= 1 || static_cast<size_t>(ldy) * sizeof(T) % 32 == 0);
        return launch_serialized(f, w.grid, kDequantThreads, 0, 1, static_cast<cudaStream_t>(stream), M, K, w.log_tx, Xq,
                                 Xs, tscale, static_cast<T*>(Y), ldy, sectors);
    });
}

}  // extern "C"
