// Pieces that both kernels of the attention over the 8-bit cache use.
#pragma once
#include "kv8_common.cuh"

namespace qg {

// A weight is 2^(x + log2 sv - M + kWeightPower): the row's largest is 2^9 to 2^15 as its running
// maximum M lags by up to kLazy, as far up in fp16's range as that allows.  What is 2^-23 of the
// largest has all of fp16's bits, what is below 2^-34 of it is rounded away: a hundred thousand such
// tokens are 2^-17 of the result at most, and 2^-8 if weights were 2^(x + log2 sv - M).  A lag of 4
// and a power of 11 gain two bits more and cost a batch with a prompt 6% (300 to 320 us), since
// some row of 32 is rescaled in more of the steps; a lag of 8 gains no time over 6.
constexpr float kLazy = 6.f, kWeightPower = 9.f;

struct AttnParams {
    Kv8Cache c;
    Kv8Batch bt;
    const void* Q;
    int64_t ldq;
    bool causal;
    int q_align;        // 16 or 8 where all heads of Q start at such addresses, else 2
    int group;          // query heads a key head
    float scale_log2;   // scale * log2(e)
    void* O;
    int64_t ldo;
    float* part;        // 2 partial sums a CTA: rows x (D + 2)
    int ctas;
    int splits;         // many rows: CTAs a unit
    int from;           // sequences of so many rows and more go to the kernel for many rows
    Ctl ctl;
};

// The kernel for many rows (qg_kv8_rows.cu), and whether it takes a problem.
int attention_rows_from(const AttnParams& p);
int attention_rows(int dtype, const AttnParams& p, int dev, cudaStream_t s);
size_t attention_rows_workspace(int64_t D);

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Below this sum of a block's weights its part of the denominator is summed without log2 sv.
// Weights lost to underflow next to a larger sum are 2^-26 of it at most.
constexpr float kLowWeight = 0x1p-100f;
// Denominators are kept times 2^20 over 2^-M, 2^kDenPower over the weights.  With a page's scale from
// 2^-64 to 2^121 their terms are then between 2^-101 and 2^90; as M moves they are multiplied by
// 2^(d / 2) twice, since 2^d alone may be below fp32's range where the result is not.
constexpr float kDenPower = 20.f - kWeightPower, kDenUnit = 1 << static_cast<int>(kDenPower);
// log2 of a page's scale; zeros of a page that nothing was written to count like the smallest.
__device__ __forceinline__ float page_log2_of(float s) { return s <= kPageScaleFloor ? -64.f : __log2f(s); }
__device__ __forceinline__ float neg_inf() { return __uint_as_float(0xff800000u); }
// What is subtracted from an exponent for its weight; any number where nothing has been seen (M = -inf).
__device__ __forceinline__ float weight_base(float M) { return M == neg_inf() ? 0.f : M - kWeightPower; }

__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t e;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(e));
    return e;
}

// 2^14 .. 2^15 over a row's largest magnitude (as bits), a power of two, and 1 over it.
struct RowPower {
    float up, down;
};
__device__ __forceinline__ RowPower row_power(uint32_t amax_bits) {
    int e = 268 - static_cast<int>(amax_bits >> 23);
    e = min(e, 253);
    return {__uint_as_float(static_cast<uint32_t>(e) << 23), __uint_as_float(static_cast<uint32_t>(254 - e) << 23)};
}

}  // namespace qg
