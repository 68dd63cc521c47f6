// tq_paged_rows.cuh -- what the tensor-core kernels of paged attention share: the
// lazy softmax reference's constants, tiles whose rows are of very unlike sizes,
// and the rows that a column sees.
#pragma once
#include "tq_common.cuh"
#include "tq_paged.cuh"
#include "tq_tcgen05.cuh"

namespace tq {
namespace {

constexpr float wTau = 8.0f, wUp = 6.0f;  // lazy raise of R; weights are 2^(s - R + wUp)
// A product of the operand tiles is below 2^(15 + 14) D <= 2^36, so with a factor
// up to this the scores are below 2^24, where R's last bit is 1.
constexpr float wFar = 1.0f / 4096;

struct __align__(8) RowMeta {  // of a row of a tile whose rows are of very unlike sizes
    float kf, e;               // as the tile's
};
// A tile gets them where its largest row is larger than its smallest (not zero)
// by more than this: two f16 terms of a key 2^-16 of the tile's largest still keep
// 2^-22 of it (the low term's last bit is 2^-38 of the largest), one of a value
// 2^-24 of it 2^-12.
constexpr float wSpreadK = 65536.0f, wSpreadV = 16777216.0f;

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ uint32_t bf16x2_max(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// The rows of a tile that a column sees: its first `vis`, or those of a mask.
struct CausalRows {
    int vis;
    __device__ __forceinline__ uint32_t from(int c) const  // of rows c .. c + 31, as bits
    {
        const int n = vis - c;
        return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
    }
};

struct TreeRows {
    const uint32_t *mask;
    int j0, n;  // the tile's first row among the new ones, new tokens
    __device__ __forceinline__ uint32_t from(int c) const { return paged_tree_bits(mask, j0 + c, n); }
};

// A tile whose rows have exponents of their own (their sizes are very unlike, so
// that one exponent would leave some of them too few of f16's bits): this
// column's true base-2 scores, value exponents added, in place of the products.
// The thread goes on with those as with any tile's; the weights' sum, whose terms
// need each row's value exponent, is taken here at the reference R that it will
// choose.  Out of line: rare, and its registers are not the common path's.
// Rows c0 .. c1 - 1 of the tile.
template <typename Rows>
__device__ __noinline__ float mixed_tile(uint32_t t_s, const RowMeta *rm, float ie, Rows rows, float R, int c0, int c1)
{
    float mx = -INFINITY, sum = 0.0f;
#pragma unroll 1
    for (int c = c0; c < c1; c += 16) {
        uint32_t x[16];
        tc_ld16(t_s + c, x);
        tc_wait_ld();
        tc_pin(x);
        const uint32_t seen = rows.from(c);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const RowMeta r = rm[c + j];
            const float y = fmaf(__uint_as_float(x[j]), fmaxf(ie * r.kf, 1.17549435e-38f), r.e);
            x[j] = seen >> j & 1u ? __float_as_uint(y) : 0xFF800000u;
            mx = fmaxf(mx, __uint_as_float(x[j]));
        }
        tc_st16(t_s + c, x);
    }
    tc_wait_st();
    if (mx > R + wTau) R = mx;
    const float add = R == -INFINITY ? 0.0f : wUp - R;
#pragma unroll 1
    for (int c = c0; c < c1; c += 16) {
        uint32_t x[16];
        tc_ld16(t_s + c, x);
        tc_wait_ld();
        tc_pin(x);
#pragma unroll
        for (int j = 0; j < 16; ++j)  // weight times 2^-e, |e| <= 100
            sum = fmaf(tc_ex2(__uint_as_float(x[j]) + add), __int_as_float((127 - (int)rm[c + j].e) << 23), sum);
    }
    return sum;
}

// Scores that may be 2^24 and more: s = x f + e in place of the products x,
// rounded as R is.  (Taken in one step, x f + (e - R) is exact, and its distance
// from a rounded R of that size no exponent of a weight.)
__device__ __noinline__ void far_tile(uint32_t t_s, float f, float e, int c0, int c1)
{
#pragma unroll 1
    for (int c = c0; c < c1; c += 16) {
        uint32_t x[16];
        tc_ld16(t_s + c, x);
        tc_wait_ld();
        tc_pin(x);
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = __float_as_uint(fmaf(__uint_as_float(x[j]), f, e));
        tc_st16(t_s + c, x);
    }
    tc_wait_st();
}

}  // namespace
}  // namespace tq
