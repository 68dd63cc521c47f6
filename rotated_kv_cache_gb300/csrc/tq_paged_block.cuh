// tq_paged_block.cuh -- paged attention of trees of a few tokens on the
// fifth-generation tensor cores: blocks of up to 128 columns (a column being one
// (new token, q-head) of a kv-head) over rows that are dequantised on the chip.
//
// Between one token and a long chunk neither of the other kernels fits.  The split
// kernel (tq_attention.cuh) unpacks every row once per 16 columns, in the
// registers that feed mma.sync; the wide one (tq_paged_wide.cu) writes every row
// to memory as f16 operands, 768 bytes for 200 at head_dim 128, which pays when
// hundreds of columns read it again.  Here a tile of T rows is unpacked once for
// all columns of a block, straight into the shared-memory images that the tensor
// cores read, and is gone after one use.
//
// A CTA of 22 warps takes a run of the split kernels' line (tq_paged.cuh),
// segment after segment, and leaves partial results for the same combine:
//   warps 0-3    softmax: a thread per column (tensor-memory lane)
//   warp 21      copies packed rows to shared memory, a tile ahead (keys swizzled)
//   warps 4-19   rows, two groups in turn: packed codes into registers, from there
//                three operand tiles (keys as two f16 terms, values) of one of NS slots
//   warp 20      issues the MMAs: S(t+1) = Q K^T before O += P(t) V, so that the
//                softmax of a tile runs under the products of the next
// Q is an operand in tensor memory, as P is, so shared memory holds rows alone.
//
// Arithmetic.  Exponents of a tile, two-term keys, the lazily raised reference R
// and rows of very unlike sizes are as in the wide kernel (see there).  Keys
// k = (c + z) s come from half-precision pairs without a rounding of their own:
// the integer c + z is exact (a byte under the exponent of 1024, plus z - 1152;
// |z| <= 896 is checked, other groups go through fp32), hi = f16((c + z) s) and
// lo = fma(c + z, s, -hi), the exact rest.  Values are f16(centroid) times f16(rms),
// two roundings of 2^-12.
// The tensor cores' sums lose up to 8e-7 of the accumulator per MMA, so O is taken
// out of tensor memory every nFlush tiles and summed in fp32.
//
// Measured: 32 sequences of 28672 rows, 8 kv-heads, head_dim 128, 8-bit keys and
// 3-bit values, 8 new tokens of 64 q-heads: 624 us (2.4 TB/s of packed rows; the
// split kernel 1950), with 16 tokens 749 (2300 by expanded rows); with one group of
// four beyond |z| = 896 in every row 909 and 956 (head_dim 64 and 256: 9 to 10 %
// more).  A tile of 128 rows takes 3100 cycles, of which the tensor pipe works 1560 (three products a
// row, lanes of 64 columns idle); the rows' 16 warps and the softmax's four share
// the issue slots, and their chains of dependent instructions take the time.
// Steps: loads kept apart from arithmetic on them and rows by bulk copies instead
// of loads (1283 -> 742 us); few columns twice in the lanes, with half of the rows
// each (-> 662); low terms in one slot, so that two tiles of packed rows fit, and a
// second group of row warps (-> 637).  Not kept: one copy of the items' code (more
// instructions waited for one another: 848), packed rows on their way to L2 a tile
// ahead (717), registers moved from rows to softmax (697).
#pragma once
#include <cuda.h>
#include <type_traits>

#include "tq_common.cuh"
#include "tq_kernels.h"
#include "tq_paged.cuh"
#include "tq_paged_rows.cuh"
#include "tq_tcgen05.cuh"

namespace tq {
namespace {

constexpr int nThreads = 704, nRowThreads = 256;  // (of each of the two groups of row warps)
constexpr int nCols = 128;   // columns of a block: the MMA's M
constexpr int nFlush = 64;   // tiles whose products O sums in tensor memory

template <int D>
struct BlockGeo {
    static constexpr int T = D <= 128 ? 128 : 64;   // rows of a tile
    static constexpr int NG = D / 32;
    static constexpr int NI = T * NG / nRowThreads;  // (row, group) items of a row thread
    static constexpr int KT = T * D * 2;             // bytes of an operand tile
    static constexpr int NS = D == 64 ? 3 : 2;       // slots of keys, and of values
    // Words about a tile are in a longer ring: a row warp writes those of tile t when its
    // group's values of t - 2 are in, so P V of t - 2 - NS is done and its words have been read.
    static constexpr int NM = D == 64 ? 8 : 4;
    static_assert(NM >= NS + 2);
    static constexpr int NL = D == 64 ? NS : 1;      // slots of the keys' low terms, which are multiplied first
    static constexpr int OFF_L = NS * KT, OFF_V = OFF_L + NL * KT;
    static constexpr int S_COL = D / 2, O_COL = S_COL + 2 * T;  // tensor memory: Q, S (then P) of two tiles, O
    static_assert(O_COL + D <= 512);
    static constexpr int OPERANDS = OFF_V + NS * KT;
};

// The packed rows of a tile in shared memory (KB and VB not 0): key boxes of SW
// bytes a row as the tensor copy swizzles them, then the other planes.
template <int D, int KB, int VB>
struct BlockRaw {
    static constexpr int T = BlockGeo<D>::T, NG = D / 32;
    static constexpr bool USED = KB != 0 && VB != 0;
    static constexpr int KROW = D * KB / 8, RBV = D * VB / 8;
    static constexpr int SW = KROW == 0 ? 1 : KROW < 128 ? KROW : 128, NBOX = KROW / SW;
    static constexpr int OFF_KS = T * KROW, OFF_KZ = OFF_KS + T * NG * 2, OFF_VS = OFF_KZ + T * NG * 2, OFF_V = OFF_VS + T * NG * 2;
    static constexpr int BYTES = USED ? (OFF_V + T * RBV + 1023) / 1024 * 1024 : 0;
    static constexpr int NR = 2;  // tiles held (a tile's place is free as soon as its codes are in registers)
    static constexpr int SMEM = 1024 + BlockGeo<D>::OPERANDS + NR * BYTES;
    static_assert(SMEM + 5632 <= 227 * 1024);
    // byte of row r's 16-byte chunk `c` of the key plane
    static __device__ __forceinline__ uint32_t key_chunk(int r, int c)
    {
        constexpr int PER = SW / 16;  // chunks of a box row
        const uint32_t x = SW == 128 ? r & 7 : SW == 64 ? (r >> 1) & 3 : (r >> 2) & 1;
        return (c / PER) * (T * SW) + r * SW + (((c % PER) ^ x) << 4);
    }
};

struct BlockParams {
    PagedSplit pg;
    const uint8_t *k_codes, *v_codes;
    const uint16_t *k_scale, *k_zero, *v_scale;
    const uint16_t *q;
    float *part_o, *part_ml;  // [slot][128][D], [slot][128][2]
    uint32_t *err;
    int H, G, kb, vb;
    float scale_log2, qsign, kcmax, cmax;
    uint32_t tl0, tl1, th0, th1;  // f16 value centroids as byte-permute tables (tq_attention.cuh)
    float cen[256];
};

struct BlockMeta {  // of a slot's tile
    float kf, e, lf;
    uint32_t any;     // bit 0: value rows that are not finite; bit 1: rows have exponents of their own
    uint32_t bad[4];
};

__device__ __forceinline__ uint32_t b_prmt(uint32_t a, uint32_t b, uint32_t sel)
{
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
    return d;
}

__device__ __forceinline__ void b_tma_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }  // |e| <= 126
__device__ __forceinline__ uint32_t b_bits(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ __half2 b_half2(uint32_t w) { return *reinterpret_cast<__half2 *>(&w); }

// The packed codes and scales of a (row, group of 32 dims) item.
template <int KB, int VB>
struct BlockItem {
    uint32_t k[KB], v[VB];
    uint16_t s, z, r;  // key scale and zero, value rms
};

// Of widths that have no fast path (0): the codes are read where they are converted.
template <>
struct BlockItem<0, 0> {
    uint16_t s, z, r;
    int64_t row;  // plane row, -1: none (zeros)
};

// An item's scales from memory, of widths whose codes are read where they are converted.
template <int D>
__device__ __forceinline__ void load_item(const BlockParams &p, int64_t row, int g, BlockItem<0, 0> &x)
{
    constexpr int NG = D / 32;
    x.row = row;
    x.s = x.z = x.r = 0;
    if (row < 0) return;
    x.s = p.k_scale[row * NG + g];
    x.z = p.k_zero[row * NG + g];
    x.r = p.v_scale[row * NG + g];
}

__device__ __forceinline__ uint32_t b_lds32(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

__device__ __forceinline__ uint16_t b_lds16(uint32_t a)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}

// An item out of a tile's packed rows; scales of a row behind the last are 0, which makes zeros of whatever is there.
template <int D, int KB, int VB>
__device__ __forceinline__ void read_item(uint32_t raw, int r, int g, bool live, BlockItem<KB, VB> &x)
{
    using W = BlockRaw<D, KB, VB>;
#pragma unroll
    for (int i = 0; i < KB / 4; ++i) {  // 4 KB bytes of the group: KB / 4 chunks
        const uint4 u = lds128(raw + W::key_chunk(r, g * (KB / 4) + i));
        x.k[4 * i] = u.x;
        x.k[4 * i + 1] = u.y;
        x.k[4 * i + 2] = u.z;
        x.k[4 * i + 3] = u.w;
    }
#pragma unroll
    for (int i = 0; i < VB; ++i) x.v[i] = b_lds32(raw + W::OFF_V + r * W::RBV + g * (4 * VB) + 4 * i);
    const uint32_t m = raw + (r * W::NG + g) * 2;
    x.s = b_lds16(m + W::OFF_KS);
    x.z = b_lds16(m + W::OFF_KZ);
    x.r = b_lds16(m + W::OFF_VS);
    if (!live) x.s = x.z = x.r = 0;
}

// Eight key codes of an item, from code 8 c on, as f16 pairs 1024 + (offset) code.
template <int KB>
__device__ __forceinline__ void key_pairs16(const uint32_t (&k)[KB], int c, uint32_t (&x)[4])
{
    if constexpr (KB == 8) {
        const uint32_t a = k[2 * c] ^ 0x80808080u, b = k[2 * c + 1] ^ 0x80808080u;
        x[0] = b_prmt(a, 0x64646464u, 0x4140u);
        x[1] = b_prmt(a, 0x64646464u, 0x4342u);
        x[2] = b_prmt(b, 0x64646464u, 0x4140u);
        x[3] = b_prmt(b, 0x64646464u, 0x4342u);
    } else {
        static_assert(KB == 4);
        const uint32_t e = k[c] & 0x0F0F0F0Fu, o = (k[c] >> 4) & 0x0F0F0F0Fu;  // codes 0, 2, 4, 6 and 1, 3, 5, 7
        const uint32_t a = b_prmt(e, o, 0x5140u), b = b_prmt(e, o, 0x7362u);   // in order, a byte each
        x[0] = b_prmt(a, 0x64646464u, 0x4140u);
        x[1] = b_prmt(a, 0x64646464u, 0x4342u);
        x[2] = b_prmt(b, 0x64646464u, 0x4140u);
        x[3] = b_prmt(b, 0x64646464u, 0x4342u);
    }
}

// Eight value codes of an item, from code 8 c on, as f16 centroids.
template <int VB>
__device__ __forceinline__ void value_pairs16(const BlockParams &p, const uint32_t (&v)[VB], int c, uint32_t (&x)[4])
{
    if constexpr (VB == 3) {
        const uint32_t w = c == 0 ? v[0] : c == 1 ? __funnelshift_r(v[0], v[1], 24) : c == 2 ? __funnelshift_r(v[1], v[2], 16) : v[2] >> 8;
        // two 12-bit fields side by side, then a code per nibble (see tq_attention.cuh)
        const uint32_t f = (w & 0xFFFu) | ((w & 0xFFF000u) << 4);
        const uint32_t y = (f & 0x003F003Fu) | ((f & 0x0FC00FC0u) * 4u);
        const uint32_t e = y + (y & 0x38383838u);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            // e's bytes hold (code 0, code 1), (code 2, code 3): four selector nibbles in order
            const uint32_t sel = h ? e >> 16 : e;
            const uint32_t lo = b_prmt(p.tl0, p.tl1, sel), hi = b_prmt(p.th0, p.th1, sel);
            x[2 * h] = b_prmt(lo, hi, 0x5140u);
            x[2 * h + 1] = b_prmt(lo, hi, 0x7362u);
        }
    } else if constexpr (VB == 2) {
        const uint32_t w = v[c >> 1] >> (16 * (c & 1));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t ab = ((w >> (4 * i)) & 3u) | ((w >> (4 * i + 2)) & 3u) << 8;
            x[i] = b_prmt(p.tl0, p.tl1, ab * 0x22u + 0x1010u);
        }
    } else {
        static_assert(VB == 4);
        const uint32_t t = (~v[c] >> 3) & 0x11111111u, m = (v[c] ^ (t * 7u)) & 0x77777777u;  // sign and magnitude index
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t sel = h ? m >> 16 : m, s = h ? t >> 16 : t;
            const uint32_t lo = b_prmt(p.tl0, p.tl1, sel), hi = b_prmt(p.th0, p.th1, sel);
            x[2 * h] = b_prmt(lo, hi, 0x5140u) ^ ((s & 1u) << 15 | (s & 0x10u) << 27);
            x[2 * h + 1] = b_prmt(lo, hi, 0x7362u) ^ ((s & 0x100u) << 7 | (s & 0x1000u) << 19);
        }
    }
}

// Codes 8 c .. 8 c + 7 of a group of any width, as the 64-bit window of key_values and value_values.
__device__ __forceinline__ void code_window(const uint8_t *group, int bits, int c, uint32_t &w0, uint32_t &w1, int &sh)
{
    const int bit = 8 * c * bits, w = bit >> 5;
    const uint32_t *a = reinterpret_cast<const uint32_t *>(group);
    sh = bit & 31;
    w0 = a[w];
    w1 = w + 1 < bits ? a[w + 1] : 0u;  // (a group is `bits` words)
}

// An item's keys into its slots (first terms, and `low` bytes on the low ones), scaled by ek2.
template <int D, int KB, int VB>
__device__ __forceinline__ void convert_keys(const BlockParams &p, const BlockItem<KB, VB> &x, int r, int g, float ek2, uint32_t slot,
                                             uint32_t low)
{
    using A = BlockGeo<D>;
    const float s = f16_bits_to_f32(x.s) * ek2, z = f16_bits_to_f32(x.z);
    // (chunk c of the group is at the first one's address xor 16 c: both are xored with the row)
    const uint32_t kt = slot + (g >> 1) * (A::T * 128) + (r >> 3) * 1024 + (r & 7) * 128 + ((((g & 1) * 4) ^ (r & 7)) << 4);
    const bool fast = KB != 0 && fabsf(z) <= 896.0f && z == rintf(z) && fabsf(s) < INFINITY;
    if (fast) {
        if constexpr (KB != 0) {
            const __half2 s2 = __float2half2_rn(s), z2 = __float2half2_rn(z - (KB == 8 ? 1152.0f : 1024.0f));
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t y[4], hi[4], lo[4];
                key_pairs16<KB>(x.k, c, y);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __half2 k = __hadd2(b_half2(y[i]), z2), h = __hmul2(k, s2);
                    hi[i] = b_bits(h);
                    lo[i] = b_bits(__hfma2(k, s2, __hneg2(h)));
                }
                const uint32_t a = kt ^ (c << 4);
                sts128(a, make_uint4(hi[0], hi[1], hi[2], hi[3]));
                sts128(a + low, make_uint4(lo[0], lo[1], lo[2], lo[3]));
            }
        }
    } else {
        const float magic = p.kb == 8 ? 8388736.0f : 8388608.0f;
        [[maybe_unused]] uint32_t k[KB ? KB : 1];
        if constexpr (KB != 0)
#pragma unroll
            for (int i = 0; i < KB; ++i) k[i] = x.k[i];
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
            uint32_t hi[4] = {0u, 0u, 0u, 0u}, lo[4] = {0u, 0u, 0u, 0u};
            bool live = true;  // (scales of a row behind the last are 0: on the fast path)
            if constexpr (KB == 0) live = x.row >= 0;
            if (live) {
                float f[8];
                if constexpr (KB != 0) {
                    // codes 8 c .. 8 c + 7 stand in the first words, the others move up (indexed by c they would not stay in registers)
                    key_values<KB>(k[0], k[KB == 8 ? 1 : 0], 0, KB, s, magic - z, f);
#pragma unroll
                    for (int i = 0; i + KB / 4 < KB; ++i) k[i] = k[i + KB / 4];
                } else {
                    uint32_t w0, w1;
                    int sh;
                    code_window(p.k_codes + x.row * (D * p.kb / 8) + g * (4 * p.kb), p.kb, c, w0, w1, sh);
                    key_values<0>(w0, w1, sh, p.kb, s, magic - z, f);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    hi[i] = tc_pack_f16(f[2 * i], f[2 * i + 1]);
                    const float2 h2 = __half22float2(b_half2(hi[i]));
                    const float a = f[2 * i] - h2.x, b = f[2 * i + 1] - h2.y;  // (not finite where k is not: none)
                    lo[i] = tc_pack_f16(fabsf(a) < 1.0e30f ? a : 0.0f, fabsf(b) < 1.0e30f ? b : 0.0f);
                }
            }
            const uint32_t a = kt ^ (c << 4);
            sts128(a, make_uint4(hi[0], hi[1], hi[2], hi[3]));
            sts128(a + low, make_uint4(lo[0], lo[1], lo[2], lo[3]));
        }
    }
}

// Its values, scaled by ev2; zeros where they are not finite.
template <int D, int KB, int VB>
__device__ __forceinline__ void convert_values(const BlockParams &p, const BlockItem<KB, VB> &x, int r, int g, float ev2, bool bad,
                                               uint32_t slot, uint32_t lut)
{
    const uint32_t vt = slot + (r >> 3) * (D / 64 * 1024) + (g >> 1) * 1024 + (r & 7) * 128 + ((((g & 1) * 4) ^ (r & 7)) << 4);
    const float v = bad ? 0.0f : f16_bits_to_f32(x.r) * ev2;
    if constexpr (VB != 0) {
        const __half2 v2 = __float2half2_rn(v);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            uint32_t y[4];
            value_pairs16<VB>(p, x.v, c, y);
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = b_bits(__hmul2(b_half2(y[i]), v2));
            sts128(vt ^ (c << 4), make_uint4(y[0], y[1], y[2], y[3]));
        }
    } else {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
            float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (x.row >= 0) {
                uint32_t w0, w1;
                int sh;
                code_window(p.v_codes + x.row * (D * p.vb / 8) + g * (4 * p.vb), p.vb, c, w0, w1, sh);
                value_values<0>(w0, w1, sh, p.vb, v, lut, f);
            }
            sts128(vt ^ (c << 4),
                   make_uint4(tc_pack_f16(f[0], f[1]), tc_pack_f16(f[2], f[3]), tc_pack_f16(f[4], f[5]), tc_pack_f16(f[6], f[7])));
        }
    }
}

template <int D, int KB, int VB>
__global__ void __launch_bounds__(nThreads, 1) paged_block_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ BlockParams p)
{
    using A = BlockGeo<D>;
    using W = BlockRaw<D, KB, VB>;
    constexpr int NR = W::NR;
    constexpr int T = A::T, NI = A::NI, KT = A::KT, NS = A::NS, NL = A::NL, NM = A::NM;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t tiles = (smem_addr(smem_raw) + 1023u) & ~1023u;
    __shared__ uint64_t bars[4 * NS + NL + 9];
    __shared__ BlockMeta meta[NM];
    __shared__ RowMeta row_meta[NM][T];
    __shared__ uint4 red[2][2][8];         // of a group's tiles in turn
    __shared__ uint32_t bad_rows[2][3][4];
    __shared__ float lut[VB ? 1 : 256];
    __shared__ uint32_t tslot;
    __shared__ PagedWalk walk;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t b0 = smem_addr(bars);
    const uint32_t kfull = b0, kempty = kfull + 8 * NS, vfull = kempty + 8 * NS, vempty = vfull + 8 * NS, sfull = vempty + 8 * NS, pfull = sfull + 16, drained = pfull + 16,
                   rfull = drained + 8, rempty = rfull + 16, lempty = rempty + 16;

    pdl_wait_primary();
    pdl_allow_dependents();
    if (warp == 0) paged_walk_start(p.pg, walk, T, nCols, p.H, p.G, lane);
    if (VB == 0 && tid >= 128)
        for (int i = tid - 128; i < (1 << p.vb); i += nThreads - 128) lut[i] = p.cen[i];
    if (tid == 32) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(kfull + 8 * i, 8);   // a row warp each
            mbar_init(vfull + 8 * i, 8);
            mbar_init(kempty + 8 * i, 1);
            mbar_init(vempty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(sfull + 8 * i, 2);  // the products' end, and the issuing warp, which saw the tile's words
            mbar_init(pfull + 8 * i, 4);  // a softmax warp each
        }
        mbar_init(drained, 1);
        for (int i = 0; i < NL; ++i) mbar_init(lempty + 8 * i, 1);
        for (int i = 0; i < 2; ++i) {  // of a group's tiles: each waits for every phase of its own
            mbar_init(rfull + 8 * i, 1);
            mbar_init(rempty + 8 * i, 8);
        }
        fence_mbar_init();
    }
    if (tid < 24) bad_rows[tid / 12][tid / 4 % 3][tid % 4] = 0u;
    __syncthreads();
    if (walk.seg[0].count <= 0) return;
    if (warp == 20) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&tslot)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __reduce_max_sync(0xffffffffu, tslot);  // (uniform)
    const uint32_t t_q = tmem, t_s = tmem + A::S_COL, t_o = tmem + A::O_COL;

    // Every role goes through the same segments; between two all of them meet.
    bool ok = true;
    uint32_t it0 = 0;  // tiles of the segments before
    auto next = [&](int nseg) {  // false: no further segment, or a wait has given up
        ok = named_and(3, 704, ok);
        return ok && walk.seg[(nseg + 1) & 1].count > 0;
    };
    if (warp >= 4 && warp < 20) {
        for (int nseg = 0;; ++nseg) {
            const PagedSegment &seg = walk.seg[nseg & 1];
            const int n = seg.count;
            // ------------------------------------------------------------ rows in
            const int w = (warp - 4) & 7, group = (warp - 4) >> 3;  // a group takes every other tile
            // eight rows of a group to eight lanes: their 16-byte stores meet no bank twice
            auto item_row = [&](int j) { return D == 64 ? w * 16 + (lane >> 4) * 8 + (lane & 7) : w * 8 + (lane & 7) + (D == 128 ? 64 * j : 0); };
            auto item_group = [&](int j) { return D == 64 ? (lane >> 3) & 1 : (lane >> 3) + (D == 256 ? 4 * j : 0); };
            const int first = seg.first, len = seg.len;
            for (int t = (it0 ^ group) & 1; t < n; t += 2) {
                const uint32_t it = it0 + t, slot = it % NS, turn = it >> 1;
                BlockItem<KB, VB> cur[NI];
                if constexpr (W::USED) {
                    if (ok) ok = mbar_wait_bounded(rfull + 8 * group, turn & 1, p.err);
                    const uint32_t raw = tiles + A::OPERANDS + (it % NR) * W::BYTES;
#pragma unroll
                    for (int j = 0; j < NI; ++j)
                        read_item<D, KB, VB>(raw, item_row(j), item_group(j), (first + t) * T + item_row(j) < len, cur[j]);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(rempty + 8 * group);
                } else {
#pragma unroll
                    for (int j = 0; j < NI; ++j) {
                        const uint32_t pos = (uint32_t)((first + t) * T + item_row(j));
                        int64_t row = -1;
                        if (pos < (uint32_t)len) {
                            const uint32_t i = fast_div(pos, p.pg.v.div_page);
                            const int pg = seg.pages[i];
                            if ((uint32_t)pg < (uint32_t)p.pg.v.num_pages) row = ((int64_t)pg * p.H + seg.h) * p.pg.v.page + (pos - i * p.pg.v.page);
                            else atomicOr(p.err, kErrPage);
                        }
                        load_item<D>(p, row, item_group(j), cur[j]);
                    }
                }
                // bounds of the tile's finite groups: largest, and smallest of those that are not zero
                uint32_t bk = 0u, bv = 0u, sk0 = 0x7F800000u, sv0 = 0x7F800000u;
                bool bad[NI];
                float fk[NI], fv[NI];
#pragma unroll
                for (int j = 0; j < NI; ++j) {
                    float b = fabsf(f16_bits_to_f32(cur[j].s)) * (fabsf(f16_bits_to_f32(cur[j].z)) + p.kcmax);
                    float v = fabsf(f16_bits_to_f32(cur[j].r));
                    bad[j] = !(v < INFINITY);
                    if (bad[j]) atomicOr(&bad_rows[group][turn % 3][item_row(j) >> 5], 1u << (item_row(j) & 31));
                    fk[j] = b = b < INFINITY ? b : 0.0f;
                    fv[j] = v = v < INFINITY ? v : 0.0f;
                    bk = max(bk, __float_as_uint(b));
                    bv = max(bv, __float_as_uint(v));
                    if (b > 0.0f) sk0 = min(sk0, __float_as_uint(b));
                    if (v > 0.0f) sv0 = min(sv0, __float_as_uint(v));
                }
                bk = __reduce_max_sync(0xffffffffu, bk);
                bv = __reduce_max_sync(0xffffffffu, bv);
                sk0 = __reduce_min_sync(0xffffffffu, sk0);
                sv0 = __reduce_min_sync(0xffffffffu, sv0);
                if (lane == 0) red[group][turn & 1][w] = make_uint4(bk, bv, sk0, sv0);
                named_sync(4 + group, nRowThreads);
                const uint4 u = red[group][turn & 1][lane & 7];
                const float fbk = __uint_as_float(__reduce_max_sync(0xffffffffu, u.x)), fbv = __uint_as_float(__reduce_max_sync(0xffffffffu, u.y));
                const float fsk = __uint_as_float(__reduce_min_sync(0xffffffffu, u.z)), fsv = __uint_as_float(__reduce_min_sync(0xffffffffu, u.w));
                auto value_exponent = [&](float x) { return tile_exponent(x > 0.0f ? x * p.cmax : 1.0f); };
                const int ek = tile_exponent(fbk), ev = value_exponent(fbv);
                const bool mixed = fbk > fsk * wSpreadK || fbv > fsv * wSpreadV;  // (the same in every thread)
                // the slot's keys of before were used up
                if (it >= NS && ok) ok = mbar_wait_bounded(kempty + 8 * slot, (it / NS - 1) & 1, p.err);
                // (the wait for the tile before last comes first: the phase waited for here is then the next one, or done)
                if (NL < NS && it >= NL && ok) ok = mbar_wait_bounded(lempty + 8 * (it % NL), (it / NL - 1) & 1, p.err);
                float ek2[NI], ev2[NI];
#pragma unroll
                for (int j = 0; j < NI; ++j) {
                    ek2[j] = power_of_two(ek);
                    ev2[j] = power_of_two(ev);
                }
                if (mixed) {
                    // exponents of each row: its groups are 8 lanes apart (and, at head_dim 256, a thread's two items)
                    float rk[NI], rv[NI];
#pragma unroll
                    for (int j = 0; j < NI; ++j) {
                        rk[j] = fk[j];
                        rv[j] = fv[j];
#pragma unroll
                        for (int o = 8; o < (D == 64 ? 16 : 32); o <<= 1) {
                            rk[j] = fmaxf(rk[j], __shfl_xor_sync(0xffffffffu, rk[j], o));
                            rv[j] = fmaxf(rv[j], __shfl_xor_sync(0xffffffffu, rv[j], o));
                        }
                    }
                    if constexpr (D == 256) {
                        rk[0] = rk[1] = fmaxf(rk[0], rk[1]);
                        rv[0] = rv[1] = fmaxf(rv[0], rv[1]);
                    }
#pragma unroll
                    for (int j = 0; j < NI; ++j) {
                        const int e1 = tile_exponent(rk[j]), e2 = value_exponent(rv[j]);
                        ek2[j] = power_of_two(e1);
                        ev2[j] = power_of_two(e2);
                        if (item_group(j) == 0) row_meta[it % NM][item_row(j)] = RowMeta{power_of_two(-e1), (float)-e2};
                    }
                }
                if (w == 0 && lane == 0) {
                    BlockMeta m;
                    m.kf = power_of_two(-ek);
                    m.e = (float)-ev;
                    m.lf = power_of_two(ev);
                    m.any = mixed ? 2u : 0u;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        m.bad[i] = bad_rows[group][turn % 3][i];
                        if (m.bad[i]) m.any |= 1u;
                        bad_rows[group][(turn + 2) % 3][i] = 0u;  // (its last readers and writers were two barriers ago)
                    }
                    meta[it % NM] = m;
                }
#pragma unroll
                for (int j = 0; j < NI; ++j) convert_keys<D, KB, VB>(p, cur[j], item_row(j), item_group(j), ek2[j], tiles + slot * KT,
                                                                               A::OFF_L - slot * KT + it % NL * KT);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(kfull + 8 * slot);
                if (it >= NS && ok) ok = mbar_wait_bounded(vempty + 8 * slot, (it / NS - 1) & 1, p.err);
#pragma unroll
                for (int j = 0; j < NI; ++j)
                    convert_values<D, KB, VB>(p, cur[j], item_row(j), item_group(j), ev2[j], bad[j], tiles + A::OFF_V + slot * KT,
                                              VB ? 0u : smem_addr(lut));
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(vfull + 8 * slot);
            }
            it0 += n;
            if (!next(nseg)) break;
        }
    } else if (warp < 4) {
        for (int nseg = 0;; ++nseg) {
            const PagedSegment &seg = walk.seg[nseg & 1];
            const int n = seg.count;
            // ------------------------------------------------------------ softmax, one column a thread
            const uint32_t lane_at = (uint32_t)(32 * warp) << 16;
            // few columns stand in the lanes two or four times, each copy with its share of a tile's rows
            const int share = nCols >> p.pg.copies, c = tid & (share - 1), cols = min(seg.n * p.G - seg.hb * share, share);
            const int k0 = (tid >> (7 - p.pg.copies)) * (T / 32 >> p.pg.copies), k1 = k0 + (T / 32 >> p.pg.copies);  // 32-row pieces
            const bool real = c < cols, busy = (32 * warp & (share - 1)) < cols;  // (warps without a column only keep step)
            const int col = seg.hb * share + (real ? c : cols - 1), tok = col / p.G;
            const uint32_t *mask = p.pg.masks + (seg.s0 + tok) * p.pg.mask_words;
            int left = seg.len - seg.n - seg.first * T;  // rows before the new ones, from the tile's first on
            float ie = 0.0f;
            if (busy) {
                // q, scaled by a power of two that puts its largest |q| in [2^14, 2^15) (exact in f16), into the column's lane
                const uint16_t *qr = p.q + (seg.s0 + tok) * p.pg.q_token + ((int64_t)seg.h * p.G + (col - tok * p.G)) * p.pg.q_head;
                uint32_t m = 0u;
#pragma unroll 4
                for (int i = 0; i < D / 8; ++i) {
                    const uint4 u = reinterpret_cast<const uint4 *>(qr)[i];
                    m = bf16x2_max(m, bf16x2_max(bf16x2_max(u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu), bf16x2_max(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu)));
                }
                const float mx = fmaxf(bf16_lo(m), bf16_hi(m));
                int e = 0;
                if (mx > 0.0f && mx < INFINITY) e = 14 - (((int)(__float_as_uint(mx) >> 23) & 0xFF) - 127);
                e = e > 100 ? 100 : e;  // (-113 at least)
                const float qs = __uint_as_float((uint32_t)(127 + e) << 23) * p.qsign;
                ie = __uint_as_float((uint32_t)(127 - e) << 23) * p.scale_log2;
#pragma unroll 1
                for (int i = 0; i < D / 32; ++i) {
                    uint32_t y[16];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint4 u = reinterpret_cast<const uint4 *>(qr)[4 * i + k];
                        y[4 * k] = tc_pack_f16(bf16_lo(u.x) * qs, bf16_hi(u.x) * qs);
                        y[4 * k + 1] = tc_pack_f16(bf16_lo(u.y) * qs, bf16_hi(u.y) * qs);
                        y[4 * k + 2] = tc_pack_f16(bf16_lo(u.z) * qs, bf16_hi(u.z) * qs);
                        y[4 * k + 3] = tc_pack_f16(bf16_lo(u.w) * qs, bf16_hi(u.w) * qs);
                    }
                    tc_st16(t_q + lane_at + 16 * i, y);
                }
                tc_wait_st();
            }
            tc_fence_before();
            named_sync(2, 160);  // with the issuing warp: Q is there
            float R = -INFINITY, l = 0.0f, Rp = -INFINITY;  // Rp: the reference of what was taken out of tensor memory
            const int64_t at = seg.slot * nCols + tid;
            const bool writes = real && seg.slot < p.pg.slots;
            for (int t = 0; t < n; ++t, left -= T) {
                const uint32_t it = it0 + t, slot = it % NS, buf = it & 1;
                if (ok) ok = mbar_wait_bounded(sfull + 8 * buf, (it >> 1) & 1, p.err);
                ok = __all_sync(0xffffffffu, ok);
                tc_fence_after();
                const bool flush = (t + 1) % nFlush == 0 || t + 1 == n;
                if (busy && ok) {
                    const uint32_t ts = t_s + buf * T + lane_at;
                    const BlockMeta &mt = meta[it % NM];
                    float e = mt.e, lf = mt.lf, f = fmaxf(ie * mt.kf, 1.17549435e-38f), extra = 0.0f;
                    const uint32_t any = mt.any;
                    const TreeRows rows{mask, -left, seg.n};
                    if (!(any & 2u) && __any_sync(0xffffffffu, f > (D > 128 ? wFar / 2 : wFar))) {
                        far_tile(ts, f, e, 32 * k0, 32 * k1);
                        f = 1.0f;
                        e = 0.0f;
                    }
                    if (any & 2u) {
                        extra = mixed_tile(ts, row_meta[it % NM], ie, rows, R, 32 * k0, 32 * k1);
                        f = 1.0f;
                        e = lf = 0.0f;
                    } else if (left < T) {  // new rows in the tile: hidden scores become -inf
#pragma unroll 1
                        for (int k = 32 * k0; k < 32 * k1; k += 16) {
                            uint32_t x[16];
                            tc_ld16(ts + k, x);
                            tc_wait_ld();
                            tc_pin(x);
                            const uint32_t seen = rows.from(k);
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                if (!(seen >> j & 1u)) x[j] = 0xFF800000u;
                            tc_st16(ts + k, x);
                        }
                        tc_wait_st();
                    }
                    // largest product, 32 rows at a time (read again for the weights)
                    float mx = -INFINITY;
#pragma unroll 1
                    for (int k = k0; k < k1; ++k) {
                        uint32_t sr[32];
                        tc_ld32(ts + 32 * k, sr);
                        tc_wait_ld();
                        tc_pin(sr);
                        float m4[4] = {mx, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int j = 0; j < 32; j += 8)
#pragma unroll
                            for (int i = 0; i < 4; ++i) m4[i] = max3(m4[i], __uint_as_float(sr[j + 2 * i]), __uint_as_float(sr[j + 2 * i + 1]));
                        mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                    }
                    const float top = mx == -INFINITY ? -INFINITY : fmaf(mx, f, e);
                    if (__any_sync(0xffffffffu, top > R + wTau)) {
                        const float Rn = top > R + wTau ? top : R;
                        const float a = R == -INFINITY ? 0.0f : tc_ex2(R - Rn);  // nothing was summed before the first row seen
                        R = Rn;
                        l *= a;
                        if (t % nFlush != 0) {
                            // O holds the products up to the tile before
                            ok = __all_sync(0xffffffffu, mbar_wait_bounded(vempty + 8 * ((it - 1) % NS), ((it - 1) / NS) & 1, p.err));
                            tc_fence_after();
#pragma unroll 1
                            for (int k = 0; k < D; k += 16) {
                                uint32_t o[16];
                                tc_ld16(t_o + lane_at + k, o);
                                tc_wait_ld();
                                tc_pin(o);
#pragma unroll
                                for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * a);
                                tc_st16(t_o + lane_at + k, o);
                            }
                        }
                    }
                    const float add = R == -INFINITY ? 0.0f : e - R + wUp;
                    const float2 f2 = make_float2(f, f), a2 = make_float2(add, add);
                    float2 ls[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                    // (weights of piece k overwrite the products of piece k / 2, which have been read)
#pragma unroll 1
                    for (int k = k0; k < k1; ++k) {
                        uint32_t sr[32], pp[16];
                        tc_ld32(ts + 32 * k, sr);
                        tc_wait_ld();
                        tc_pin(sr);
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            const float2 y = __ffma2_rn(make_float2(__uint_as_float(sr[j]), __uint_as_float(sr[j + 1])), f2, a2);
                            const float p0 = tc_ex2(y.x), p1 = tc_ex2(y.y);
                            ls[(j >> 1) & 1] = __fadd2_rn(ls[(j >> 1) & 1], make_float2(p0, p1));
                            pp[j / 2] = tc_pack_f16(p0, p1);
                        }
                        tc_st16(ts + 16 * k, pp);
                    }
                    if (p.pg.copies) {  // the other copies' rows
                        const uint32_t none[16] = {};
#pragma unroll 1
                        for (int k = 0; k < T / 32; ++k)
                            if (k < k0 || k >= k1) tc_st16(ts + 16 * k, none);
                    }
                    l = fmaf((ls[0].x + ls[0].y) + (ls[1].x + ls[1].y), lf, l + extra);
                    if (any & 1u) {
#pragma unroll 1
                        for (int i = k0; i < k1; ++i)
                            if (mt.bad[i] & rows.from(32 * i)) l = NAN;
                    }
                    tc_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(pfull + 8 * buf);
                if (flush) {
                    if (ok) ok = mbar_wait_bounded(vempty + 8 * slot, (it / NS) & 1, p.err);
                    ok = __all_sync(0xffffffffu, ok);
                    tc_fence_after();
                    if (busy && ok) {
                        // the products so far on top of those taken out before (of this thread)
                        const float a = Rp == -INFINITY ? 0.0f : tc_ex2(Rp - R);
                        const bool first = t < nFlush;
#pragma unroll 1
                        for (int k = 0; k < D; k += 16) {
                            uint32_t o[16];
                            tc_ld16(t_o + lane_at + k, o);
                            tc_wait_ld();
                            tc_pin(o);
                            float4 *dst = reinterpret_cast<float4 *>(p.part_o + at * D + k);
                            if (writes)
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    float4 x = first ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : dst[j];
                                    x.x = fmaf(x.x, a, __uint_as_float(o[4 * j]));
                                    x.y = fmaf(x.y, a, __uint_as_float(o[4 * j + 1]));
                                    x.z = fmaf(x.z, a, __uint_as_float(o[4 * j + 2]));
                                    x.w = fmaf(x.w, a, __uint_as_float(o[4 * j + 3]));
                                    dst[j] = x;
                                }
                        }
                        Rp = R;
                    }
                    tc_fence_before();
                }
            }
            if (writes) {
                p.part_ml[2 * at] = ok ? R - wUp : -INFINITY;  // R = -inf (nothing seen): weight 0
                p.part_ml[2 * at + 1] = ok ? l : 0.0f;
            }
            it0 += n;
            if (tid == 0) paged_walk_next(p.pg, walk, walk.seg[(nseg + 1) & 1], T, nCols, p.H, p.G);
            if (!next(nseg)) break;
        }
    } else {
        for (int nseg = 0; warp == 20; ++nseg) {
            const PagedSegment &seg = walk.seg[nseg & 1];
            const int n = seg.count;
            // ------------------------------------------------------------ MMAs
            constexpr uint32_t idesc_qk = tc_idesc(128, T, 0), idesc_pv = tc_idesc(128, D, 1), SBO = (D / 64) * 1024;
            const uint32_t leader = tc_elect();
            const uint64_t d0 = tc_desc(tiles, 16, 1024), v0 = tc_desc(tiles + A::OFF_V, 1024, SBO);
            const uint32_t dk = (uint32_t)d0, dv = (uint32_t)v0;
            constexpr uint32_t hk = (uint32_t)(tc_desc_const(16, 1024) >> 32), hv = (uint32_t)(tc_desc_const(1024, SBO) >> 32);
            auto desc = [](uint32_t hi, uint32_t lo) { return (uint64_t)hi << 32 | lo; };
            auto wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, p.err)) != 0; };
            auto qk = [&](uint32_t it) {
                const uint32_t slot = it % NS;
                if (!wait(kfull + 8 * slot, (it / NS) & 1)) return false;
                tc_fence_after();
                if (lane == 0) mbar_arrive(sfull + 8 * (it & 1));
                auto term = [&](uint32_t at, uint32_t acc) __attribute__((always_inline)) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        tc_mma_ts_elected(leader, t_s + (it & 1) * T, t_q + kk * 8, desc(hk, dk + ((at + (kk / 4) * (T * 128) + (kk % 4) * 32) >> 4)),
                                          idesc_qk, kk > 0 ? 1u : acc);
                };
                term(A::OFF_L + it % NL * KT, 0);
                if (NL < NS) tc_commit_elected(leader, lempty + 8 * (it % NL));
                term(slot * KT, 1);
                tc_commit_elected(leader, sfull + 8 * (it & 1));
                tc_commit_elected(leader, kempty + 8 * slot);
                return true;
            };
            named_sync(2, 160);  // Q is there
            tc_fence_after();
            bool go = ok && qk(it0);
            for (int t = 0; t < n && go; ++t) {
                const uint32_t it = it0 + t, slot = it % NS;
                if (t + 1 < n) go = qk(it + 1);
                go = go && wait(pfull + 8 * (it & 1), (it >> 1) & 1) && wait(vfull + 8 * slot, (it / NS) & 1);
                if (!go) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < T / 16; ++kk)
                    tc_mma_ts_elected(leader, t_o, t_s + (it & 1) * T + kk * 8, desc(hv, dv + ((slot * KT + kk * 2 * SBO) >> 4)), idesc_pv,
                                      kk > 0 || t % nFlush != 0 ? 1u : 0u);
                tc_commit_elected(leader, vempty + 8 * slot);
            }
            if (!go && ok) {  // whatever was issued is through before tensor memory is given back (bounded)
                tc_commit_elected(leader, drained);
                mbar_wait_bounded(drained, 0, p.err);
            }
            ok = go;
            tc_fence_before();
            it0 += n;
            if (!next(nseg)) break;
        }
        // ------------------------------------------------------------ packed rows in
        for (int nseg = 0; warp == 21; ++nseg) {
            const PagedSegment &seg = walk.seg[nseg & 1];
            const int n = seg.count;
            if constexpr (W::USED) {
                const int ru = p.pg.ru, first = seg.first, len = seg.len;
                int done = 0;  // tiles under way
                int page = paged_chunk_page(p.pg, seg, first, lane);  // (a lane copies a chunk; its page a tile ahead)
                for (int t = 0; t < n; ++t) {
                    const uint32_t it = it0 + t, at = it % NR, bar = rfull + 8 * (it & 1);
                    const int this_page = page;
                    if (t + 1 < n) page = paged_chunk_page(p.pg, seg, first + t + 1, lane);
                    const int rows = min(T, len - (first + t) * T), live = (rows + ru - 1) / ru;
                    // the tile that was there is in registers
                    if (it >= NR && ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(rempty + 8 * ((it - NR) & 1), ((it - NR) >> 1) & 1, p.err));
                    if (!ok) break;
                    ++done;
                    if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(live * ru * (W::KROW + 3 * W::NG * 2 + W::RBV)));
                    __syncwarp();
                    if (lane < live) {
                        const uint32_t row = (uint32_t)paged_chunk_plane_row(p.pg, seg, p.H, this_page, first + t, lane), st = tiles + A::OPERANDS + at * W::BYTES;
                        const int r0 = lane * ru;
                        constexpr int NG = W::NG;
#pragma unroll
                        for (int j = 0; j < W::NBOX; ++j) b_tma_2d(st + j * (T * W::SW) + r0 * W::SW, &kmap, j * W::SW, (int)row, bar);
                        bulk_g2s(st + W::OFF_KS + r0 * (NG * 2), p.k_scale + (size_t)row * NG, ru * NG * 2, bar);
                        bulk_g2s(st + W::OFF_KZ + r0 * (NG * 2), p.k_zero + (size_t)row * NG, ru * NG * 2, bar);
                        bulk_g2s(st + W::OFF_VS + r0 * (NG * 2), p.v_scale + (size_t)row * NG, ru * NG * 2, bar);
                        bulk_g2s(st + W::OFF_V + r0 * W::RBV, p.v_codes + (size_t)row * W::RBV, ru * W::RBV, bar);
                    }
                }
                // the last copies land before the segment, and the CTA, ends (bounded)
                for (int i = max(done - NR, 0); i < done; ++i) mbar_wait_bounded(rfull + 8 * ((it0 + i) & 1), ((it0 + i) >> 1) & 1, p.err);
            }
            it0 += n;
            if (!next(nseg)) break;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 20) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// ---------------------------------------------------------------- host side
template <int D, typename F>
auto block_widths(const CacheView &c, F &&f)
{
    using std::integral_constant;
    auto with = [&](auto kb) {
        return c.vb == 3   ? f(kb, integral_constant<int, 3>{})
               : c.vb == 4 ? f(kb, integral_constant<int, 4>{})
                           : f(kb, integral_constant<int, 2>{});
    };
    // other widths of either by run-time shifts, of both then
    if (c.vb > 4 || (c.kb != 8 && c.kb != 4)) return f(integral_constant<int, 0>{}, integral_constant<int, 0>{});
    return c.kb == 8 ? with(integral_constant<int, 8>{}) : with(integral_constant<int, 4>{});
}

template <int D>
bool block_shape(const CacheView &c, PagedShape &sh)
{
    const int ctas = block_widths<D>(c, [](auto kb, auto vb) {
        static KernelSetup setup;
        int n;
        constexpr int smem = BlockRaw<D, kb.value, vb.value>::SMEM;
        setup.get(paged_block_kernel<D, kb.value, vb.value>, nThreads, smem, smem, n);
        return n;
    });
    sh = PagedShape{BlockGeo<D>::T, nCols, num_sms()};
    return ctas > 0;
}

template <int D>
cudaError_t block_run(const CacheView &c, const PagedSplit &pg, const PagedShape &sh, const uint16_t *q, int QH, float scale, float *part_o,
                      float *part_ml, cudaStream_t s)
{
    BlockParams p{};
    p.pg = pg;
    p.k_codes = c.k_codes;
    p.v_codes = c.v_codes;
    p.k_scale = c.k_scale;
    p.k_zero = c.k_zero;
    p.v_scale = c.v_scale;
    p.q = q;
    p.part_o = part_o;
    p.part_ml = part_ml;
    p.err = pg.v.err;
    p.H = c.H;
    p.G = QH / c.H;
    p.kb = c.kb;
    p.vb = c.vb;
    p.scale_log2 = fabsf(scale) * 1.4426950408889634f;
    p.qsign = scale < 0.0f ? -1.0f : 1.0f;
    p.kcmax = c.kb == 8 ? 127.0f : (float)((1 << c.kb) - 1);
    const Tables &tab = codebook_tables(c.vb);
    for (int i = 0; i < (1 << c.vb); ++i) {
        p.cen[i] = tab.centroids[i];
        p.cmax = p.cmax > fabsf(tab.centroids[i]) ? p.cmax : fabsf(tab.centroids[i]);
    }
    auto f16b = [](float x) { return (uint32_t)__half_as_ushort(__float2half_rn(x)); };
    if (c.vb == 2) {
        p.tl0 = f16b(tab.centroids[0]) | f16b(tab.centroids[1]) << 16;
        p.tl1 = f16b(tab.centroids[2]) | f16b(tab.centroids[3]) << 16;
    } else if (c.vb <= 4) {
        for (int i = 0; i < 8; ++i) {  // 3 bits: the eight centroids; 4 bits: the eight magnitudes
            const uint32_t h = f16b(tab.centroids[(c.vb == 3 ? 0 : 8) + i]);
            (i < 4 ? p.tl0 : p.tl1) |= (h & 0xFF) << 8 * (i & 3);
            (i < 4 ? p.th0 : p.th1) |= (h >> 8) << 8 * (i & 3);
        }
    }
    set_paged_chunks(p.pg, BlockGeo<D>::T, (int)c.cap);
    return block_widths<D>(c, [&](auto kb, auto vb) {
        using W = BlockRaw<D, kb.value, vb.value>;
        CUtensorMap map{};
        if constexpr (W::USED) {
            // the key plane's rows in boxes of SW bytes by a chunk's rows
            auto fn = tensor_map_encoder();
            if (!fn) return cudaErrorNotSupported;
            const cuuint64_t dim[2] = {(cuuint64_t)W::KROW, (cuuint64_t)c.B * c.H * c.cap}, stride[1] = {(cuuint64_t)W::KROW};
            const cuuint32_t box[2] = {(cuuint32_t)W::SW, (cuuint32_t)p.pg.ru}, one[2] = {1, 1};
            const CUtensorMapSwizzle swz = W::SW == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : W::SW == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B;
            if (fn(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, c.k_codes, dim, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swz,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
                return cudaErrorInvalidValue;
        }
        return launch_dependent(paged_block_kernel<D, kb.value, vb.value>, dim3((unsigned)sh.ctas), dim3(nThreads), (size_t)W::SMEM, s, map, p);
    });
}

}  // namespace
}  // namespace tq

// The entry points of one head_dim's translation unit.
#define TQ_PAGED_BLOCK_ENTRIES(D)                                                                                                 \
    namespace tq {                                                                                                                \
    bool paged_block_shape_d##D(const CacheView &c, PagedShape &sh) { return block_shape<D>(c, sh); }                             \
    cudaError_t launch_paged_block_d##D(const CacheView &c, const PagedSplit &pg, const PagedShape &sh, const uint16_t *q, int QH, \
                                        float scale, float *part_o, float *part_ml, cudaStream_t s)                               \
    {                                                                                                                             \
        return block_run<D>(c, pg, sh, q, QH, scale, part_o, part_ml, s);                                                         \
    }                                                                                                                             \
    }
