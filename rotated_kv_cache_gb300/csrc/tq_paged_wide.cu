// tq_paged_wide.cu -- paged attention of long chunks (prefill) on the
// fifth-generation tensor cores, head_dims 64 and 128.
//
// The split kernels dequantise every cached row once per 16 columns (a column
// being one (new token, q-head) of a kv-head), which is what a chunk of
// hundreds of columns spends its time on.  Here the rows are expanded once:
//
//  1. plan     which sequences are wide (more new tokens than `wide`), their
//              128-row tiles and 256-column blocks, as prefix sums;
//  2. expand   every (128-row tile, kv-head) becomes three f16 operand tiles
//              in the workspace (keys as two terms, values), laid out as the
//              images that the tensor cores read from shared memory (128-byte
//              swizzle; keys K-major, values MN-major), so that a tile is one
//              linear copy;
//  3. attend   persistent CTAs of two 128-column groups: one warp copies
//              tiles, one issues the MMAs, two warpgroups run the softmax (a
//              thread per column);
//  4. merge    of the few blocks that two or more CTAs shared.
//
// Range.  f16 has 11 bits and a narrow exponent, so every key tile is scaled
// by a power of two that puts its largest finite |k| in [2^13, 2^14) (undone on
// the scores) and every value tile likewise; the value exponent e of a tile is
// added to the base-2 scores, so that one accumulator holds
//   O = sum_t 2^(s_t + e - R + 6) (v_t 2^-e),   l = sum_t 2^(s_t + e - R + 6) 2^-e
// for any mixture of tiles, and O / l needs no correction.  Values and weights
// are rounded to f16 (2^-12 of them each), below the bf16 output's 2^-9.  A
// rounding of a key enters the output times the score, so keys are held as
// k = hi + lo (hi = f16(k), lo = f16(k - hi): 22 bits), and both terms' products
// go into one accumulator.  With hi alone heavy-tailed keys, whose scores
// reach 60, moved outputs of unit values by up to 0.025.
// A row may be far larger than others of its tile, and one that a column does
// not see must not take bits from those that it sees: rows of tiles where sizes
// spread too far have exponents of their own (RowMeta).
// The reference R follows the running maximum of s + e lazily: it is raised
// (and O rescaled) only when the maximum has grown by more than 2^8, so that
// the weights stay within [0, 2^14] and keep 11 bits down to 2^-20 of the
// largest.
//
// Measured: 2048 new tokens over 32768 rows, 64 q-heads, 8 kv-heads, head_dim
// 128, 4-bit keys, 3-bit values: 2020 us in all, 1.05 PFLOP/s of the attention's
// own products and 1.57 with the low terms' (of 1.88 that a large library
// product reaches); a prompt of 8191 tokens 535 us, 1.03 and 1.53.  With hi alone
// they took 1493 and 416: the tensor pipe has half as much work again, and
// bounds the kernel (77 % busy at 1024 tokens over 8192 rows; expand 18 us, attend
// 219, merge 20, cold L2).  The rest is the starts and ends of blocks.
//
// A value row with an infinity or NaN would spoil the sums of columns that do
// not see it (0 * inf), so expand writes zeros there and a bit mask; a column
// that sees a marked row gets NaN through l.
#include <type_traits>

#include "tq_common.cuh"
#include "tq_kernels.h"
#include "tq_paged.cuh"
#include "tq_tcgen05.cuh"

namespace tq {
namespace {

constexpr int wT = 128;    // rows per tile
constexpr int wC = 256;    // columns per block (two groups of the MMA's 128)
constexpr int wThreads = 384;  // two softmax warpgroups; MMA warp, tile warp (and two idle ones)
constexpr int wPlanThreads = 256;
// What a block costs besides its tiles (q in, out of tensor memory, un-rotation), in
// tiles.  A prompt of 8191 tokens, 32 q-heads, with 3 / 4 / 5 / 7 / 9: 498 / 489 /
// 493 / 502 / 510 us; of 4096 tokens 178 / 173 / 175 / 180 / 180.
constexpr int wStart = 4;
constexpr float wTau = 8.0f, wUp = 6.0f;  // lazy raise of R; weights are 2^(s - R + wUp)
// A product of the operand tiles is below 2^(15 + 14) D <= 2^36, so with a factor
// up to this the scores are below 2^24, where R's last bit is 1.
constexpr float wFar = 1.0f / 4096;

// What expand says about a tile.
struct __align__(16) TileMeta {
    float kf;       // 2^-ek: scores are (q k~) kf
    float e;        // the value tile's exponent: v = v~ 2^e
    float lf;       // 2^-e
    uint32_t any;   // bit 0: some value row is not finite; bit 1: every row has exponents of its own (RowMeta)
    uint32_t bad[4];
};

struct __align__(8) RowMeta {  // of a row of a tile whose rows are of very unlike sizes
    float kf, e;               // as the tile's
};
// A tile gets them where its largest row is larger than its smallest (not zero)
// by more than this: two f16 terms of a key 2^-16 of the tile's largest still keep
// 2^-22 of it (the low term's last bit is 2^-38 of the largest), one of a value
// 2^-24 of it 2^-12.
constexpr float wSpreadK = 65536.0f, wSpreadV = 16777216.0f;

struct WidePlan {        // device arrays, written by plan
    int32_t *tile0;      // [seqs + 1] scratch tiles before a sequence
    int32_t *entry0;     // [seqs + 1] blocks before it
    int64_t *before;     // [entries + 1] cost (tiles + wStart each) of the blocks before an entry (one kv-head's)
    int64_t *line;       // total cost of the line, cost per CTA
    struct WideShare *share;  // [CTAs] the block that a CTA began and did not finish
};

struct WideShare {
    int s, h, block;     // block of the sequence
    int last;            // the last CTA that has a share of it, or -1: nothing is shared
};

struct WideParams {
    PagedSplit pg;
    WidePlan pl;
    int64_t max_tiles, max_entries;  // room in the workspace
    int32_t *spill;      // [seqs]: a long chunk that found no room (null: the bounds leave room for all)
    const uint8_t *k_codes, *v_codes;
    const uint16_t *k_scale, *k_zero, *v_scale;
    const uint16_t *q;
    uint16_t *out;
    TileMeta *meta;      // [tile][H]
    RowMeta *row_meta;   // [tile][H][128], of tiles with rows of very unlike sizes
    uint8_t *tiles;      // [tile][H][keys hi, keys lo, values]
    float *part_o, *part_ml;  // [2 CTAs][256][D], [..][256][2]
    uint32_t *err;
    int H, QH, G, kb, vb, ctas;
    float scale_log2;    // |softmax scale| * log2(e); its sign goes into q
    float qsign, kcmax, cmax, inv_sqrt_d;
    SignBits sg;
    float cen[256];
};

template <int D>
struct WideGeo {
    static constexpr int KT = wT * D * 2;  // bytes of one operand tile
    static constexpr int NK = D == 128 ? 2 : 4, NV = NK;  // tiles in flight
    // the keys' low terms in pieces of 64 dims: a tile's at head_dim 128, where no more fits, four at 64
    static constexpr int LB = wT * 128, PL = D / 64, NL = D == 128 ? 2 : 4;
    static constexpr int OFF_K = 2 * KT, OFF_L = OFF_K + NK * KT, OFF_V = OFF_L + NL * LB, OFF_BAR = OFF_V + NV * KT;
    static constexpr int BARS = 2 * (NK + NL + NV) + 11;
    static constexpr int SMEM = 1024 + OFF_BAR + (BARS * 8 + 4 + 127) / 128 * 128;
    static_assert(SMEM + 1024 <= 227 * 1024);
    static constexpr int O_COL = 2 * wT;   // tensor memory: S (then P) of both groups, then O of both
};

// ---------------------------------------------------------------- plan
__device__ __forceinline__ int64_t block_exclusive_sum(int64_t x, int64_t &total, int64_t *sh)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const int64_t in = warp_inclusive_sum(x, lane);
    __syncthreads();  // the previous call's readers are done with sh
    if (lane == 31) sh[warp] = in;
    __syncthreads();
    int64_t base = 0;
    total = 0;
    for (int w = 0; w < nw; ++w) {
        if (w < warp) base += sh[w];
        total += sh[w];
    }
    return base + in - x;
}

// Tiles that block b of a sequence reads: up to its last column's limit (one
// at least, so that a column that sees nothing is written too).
__device__ __forceinline__ int64_t block_tiles(int64_t len, int64_t n, int G, int64_t b)
{
    const int64_t cols = n * G, last = (cols < (b + 1) * wC ? cols : (b + 1) * wC) - 1;
    const int64_t lim = len - n + 1 + last / G, t = (lim + wT - 1) / wT;
    return t < 1 ? 1 : t;
}

__global__ void __launch_bounds__(wPlanThreads) wide_plan_kernel(const __grid_constant__ WideParams p)
{
    __shared__ int64_t sh[32];
    pdl_wait_primary();
    pdl_allow_dependents();
    const int S = p.pg.v.seqs;
    int64_t want = 0, tiles = 0, entries = 0;  // tiles that all would take; tiles and blocks given
    for (int s0 = 0; s0 < S; s0 += blockDim.x) {
        const int s = s0 + threadIdx.x;
        int64_t t = 0, e = 0, all;
        if (s < S) {
            const int64_t n = paged_new(p.pg.v, s);
            if (n > p.pg.wide && n <= p.pg.max_new) {
                const int64_t len = paged_len(p.pg.v, s);
                t = len > 0 ? (len + wT - 1) / wT : 1;
                e = (n * p.G + wC - 1) / wC;
            }
        }
        // the first sequences that fit get tiles; the others are the split kernel's, or where the
        // bounds that the caller gave left no room, nobody's
        const bool fits = want + block_exclusive_sum(t, all, sh) + t <= p.max_tiles;
        want += all;
        if (s < S) {
            if (p.spill) p.spill[s] = e > 0 && !fits;
            else if (e > 0 && !fits) atomicOr(p.err, kErrLength);
        }
        if (!fits) t = e = 0;
        const int64_t at = tiles + block_exclusive_sum(t, all, sh);
        tiles += all;
        const int64_t ae = entries + block_exclusive_sum(e, all, sh);
        entries += all;
        if (s < S) {
            if (ae + e > p.max_entries) atomicOr(p.err, kErrLength);
            p.pl.tile0[s] = (int32_t)at;
            p.pl.entry0[s] = (int32_t)imin64(ae, p.max_entries);
        }
    }
    if (entries > p.max_entries) tiles = entries = 0;  // (starts out of order)
    if (threadIdx.x == 0) {
        p.pl.tile0[S] = (int32_t)tiles;
        p.pl.entry0[S] = (int32_t)entries;
    }
    __syncthreads();  // tile0, entry0 are read back below (same block)
    int64_t line = 0;
    for (int64_t e0 = 0; e0 < entries; e0 += blockDim.x) {
        const int64_t e = e0 + threadIdx.x;
        int64_t t = 0, all;
        if (e < entries) {
            int lo = 0, hi = S;  // the last sequence with entry0 <= e
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (p.pl.entry0[mid] <= e) lo = mid;
                else hi = mid - 1;
            }
            t = wStart + block_tiles(paged_len(p.pg.v, lo), paged_new(p.pg.v, lo), p.G, e - p.pl.entry0[lo]);
        }
        const int64_t at = line + block_exclusive_sum(t, all, sh);
        line += all;
        if (e < entries) p.pl.before[e] = at;
    }
    if (threadIdx.x == 0) {
        p.pl.before[entries] = line;
        const int64_t total = line * p.H;
        int64_t per = (total + p.ctas - 1) / p.ctas;
        p.pl.line[0] = total;
        p.pl.line[1] = per < wStart ? wStart : per;  // no run of less than a start
    }
}

// A place on the line (its unit is the cost of a tile): sequence after sequence, in a sequence kv-head after
// kv-head (CTAs of one head are neighbours, and share its tiles in L2), then
// block after block, in a block its start, then its tiles.  A CTA whose run
// ends within a start leaves the block to the next one.
struct WidePlace {
    int s, h, e, tile, tiles;  // entry (block) and tile in it; tiles of the block
    int e0, e1;                // entries of the sequence
    int tile0;                 // its first scratch tile
    int64_t s0, n, len;        // its first ragged row, new tokens, rows
    int64_t at;                // line position of the block's first tile

    // tiles of the block from `tile` on that a run up to x1 takes
    __device__ __forceinline__ int count(int64_t x1) const
    {
        const int64_t m = x1 - at;
        return (int)(m < tiles ? m : tiles) - tile;
    }
    __device__ __forceinline__ bool ends(int64_t x1) const { return at + tiles >= x1; }  // the run ends with this block, or in it
};

__device__ __forceinline__ void wide_sequence(const WideParams &p, WidePlace &w)
{
    w.tile0 = p.pl.tile0[w.s];
    w.s0 = paged_start(p.pg.v, w.s);
    w.n = paged_new(p.pg.v, w.s);
    w.len = paged_len(p.pg.v, w.s);
}

__device__ __forceinline__ WidePlace wide_locate(const WideParams &p, int64_t x)
{
    WidePlace w;
    int lo = 0, hi = p.pg.v.seqs - 1;  // the last sequence that starts at or before x
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.pl.before[p.pl.entry0[mid]] * p.H <= x) lo = mid;
        else hi = mid - 1;
    }
    w.s = lo;
    const int e0 = w.e0 = p.pl.entry0[lo], e1 = w.e1 = p.pl.entry0[lo + 1];
    const int64_t b0 = p.pl.before[e0], sum = p.pl.before[e1] - b0, y = x - b0 * p.H;
    w.h = (int)(y / sum);
    const int64_t z = y - w.h * sum + b0;  // within one head's blocks
    int a = e0, b = e1 - 1;
    while (a < b) {
        const int mid = (a + b + 1) >> 1;
        if (p.pl.before[mid] <= z) a = mid;
        else b = mid - 1;
    }
    w.e = a;
    const int off = (int)(z - p.pl.before[a]) - wStart;
    w.tile = off > 0 ? off : 0;
    w.tiles = (int)(p.pl.before[a + 1] - p.pl.before[a]) - wStart;
    w.at = x - off;
    wide_sequence(p, w);
    return w;
}

// From the end of a block to the next one's first tile (there is one).
__device__ __forceinline__ void wide_next(const WideParams &p, WidePlace &w)
{
    w.tile = 0;
    w.at += w.tiles + wStart;
    if (++w.e == w.e1) {
        w.e = w.e0;
        if (++w.h == p.H) {
            w.h = 0;
            w.e = w.e0 = w.e1;
            do {
                ++w.s;
                w.e1 = p.pl.entry0[w.s + 1];
            } while (w.e1 == w.e0);
            wide_sequence(p, w);
        }
    }
    w.tiles = (int)(p.pl.before[w.e + 1] - p.pl.before[w.e]) - wStart;
}

// ---------------------------------------------------------------- expand
// A block per (tile, kv-head) item: the rows' places looked up once, the tile's
// exponents from its scales alone (no pass over the codes), then eight
// elements a thread to each operand tile in 16-byte words, the loads of four of
// them together (with a load and a store at a time, 16 tokens over 4096 rows
// took 1.4 us more in all).  It writes 6 d bytes a row and kv-head: 8192 rows of
// 8 kv-heads, head_dim 128, are 50 MB, which the attend kernel finds in L2.
template <int D>
__global__ void __launch_bounds__(256, 4) wide_expand_kernel(const __grid_constant__ WideParams p)
{
    constexpr int NG = D / 32, C8 = D / 8, KT = WideGeo<D>::KT;
    static_assert(wT * C8 % 1024 == 0 && wT * NG % 256 == 0);
    __shared__ float lut[256];
    __shared__ int64_t rows[wT];   // plane row of each tile row (-1: none)
    __shared__ float row_k[wT], row_v[wT];  // bounds of each row, then its powers of two
    __shared__ float red[4][8];
    __shared__ uint32_t bad[4];
    pdl_wait_primary();
    pdl_allow_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < (1 << p.vb); i += 256) lut[i] = p.cen[i];
    const int S = p.pg.v.seqs, rbk = D * p.kb / 8, rbv = D * p.vb / 8;
    const int64_t items = (int64_t)p.pl.tile0[S] * p.H;
    const float magic = p.kb == 8 ? 8388736.0f : 8388608.0f;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int tile = (int)(item / p.H), h = (int)(item - (int64_t)tile * p.H);
        int lo = 0, hi = S - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (p.pl.tile0[mid] <= tile) lo = mid;
            else hi = mid - 1;
        }
        const int64_t t0 = (int64_t)(tile - p.pl.tile0[lo]) * wT, len = paged_len(p.pg.v, lo);
        __syncthreads();  // the previous item is done with rows, red and bad
        if (tid < 4) bad[tid] = 0;
        if (tid < wT) {
            int64_t r = -1;
            if (t0 + tid < len) {
                uint32_t slot;
                const int pg = paged_page(p.pg.v, lo, (uint32_t)(t0 + tid), slot);
                if (pg >= 0) r = ((int64_t)pg * p.H + h) * p.pg.v.page + slot;
            }
            rows[tid] = r;
        }
        __syncthreads();
        // bounds of the finite groups of all rows and of each, and the value rows that are not finite
        float bk = 0.0f, bv = 0.0f, sk0 = INFINITY, sv0 = INFINITY;  // largest, and smallest of the rows that are not zero
        constexpr int MI = wT * NG / 256;
        uint16_t ms[MI], mz[MI], mv[MI];
#pragma unroll
        for (int j = 0; j < MI; ++j) {
            const int i = tid + 256 * j;
            const int64_t r = rows[i / NG], mi = r * NG + i % NG;
            ms[j] = r < 0 ? 0 : p.k_scale[mi];
            mz[j] = r < 0 ? 0 : p.k_zero[mi];
            mv[j] = r < 0 ? 0 : p.v_scale[mi];
        }
#pragma unroll
        for (int j = 0; j < MI; ++j) {
            const int t = (tid + 256 * j) / NG;
            float b = fabsf(f16_bits_to_f32(ms[j])) * (fabsf(f16_bits_to_f32(mz[j])) + p.kcmax);
            float v = fabsf(f16_bits_to_f32(mv[j]));
            if (!(v < INFINITY)) atomicOr(&bad[t >> 5], 1u << (t & 31));
            b = b < INFINITY ? b : 0.0f;
            v = v < INFINITY ? v : 0.0f;
#pragma unroll
            for (int o = 1; o < NG; o <<= 1) {  // a row's groups are neighbouring lanes
                b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, o));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
            }
            if ((tid & (NG - 1)) == 0) {
                row_k[t] = b;
                row_v[t] = v;
            }
            bk = fmaxf(bk, b);
            bv = fmaxf(bv, v);
            if (b > 0.0f) sk0 = fminf(sk0, b);
            if (v > 0.0f) sv0 = fminf(sv0, v);
        }
#pragma unroll
        for (int o = 16; o >= NG; o >>= 1) {
            bk = fmaxf(bk, __shfl_xor_sync(0xffffffffu, bk, o));
            bv = fmaxf(bv, __shfl_xor_sync(0xffffffffu, bv, o));
            sk0 = fminf(sk0, __shfl_xor_sync(0xffffffffu, sk0, o));
            sv0 = fminf(sv0, __shfl_xor_sync(0xffffffffu, sv0, o));
        }
        if (lane == 0) {
            red[0][warp] = bk;
            red[1][warp] = bv;
            red[2][warp] = sk0;
            red[3][warp] = sv0;
        }
        __syncthreads();
        bk = bv = 0.0f;
        sk0 = sv0 = INFINITY;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            bk = fmaxf(bk, red[0][w]);
            bv = fmaxf(bv, red[1][w]);
            sk0 = fminf(sk0, red[2][w]);
            sv0 = fminf(sv0, red[3][w]);
        }
        // a tile of zeros takes the exponent of one whose largest value is 1
        auto value_exponent = [&](float x) { return tile_exponent(x > 0.0f ? x * p.cmax : 1.0f); };
        const int ek = tile_exponent(bk), ev = value_exponent(bv);
        const bool mixed = bk > sk0 * wSpreadK || bv > sv0 * wSpreadV;  // (the same in every thread)
        if (mixed) {
            if (tid < wT) {
                const int e1 = tile_exponent(row_k[tid]), e2 = value_exponent(row_v[tid]);
                row_k[tid] = ldexpf(1.0f, e1);
                row_v[tid] = ldexpf(1.0f, e2);
                p.row_meta[item * wT + tid] = RowMeta{ldexpf(1.0f, -e1), (float)-e2};
            }
            __syncthreads();
        }
        const float sk = ldexpf(1.0f, ek), sv2 = ldexpf(1.0f, ev);
        uint8_t *dst = p.tiles + item * (3 * KT);
        if (tid == 0) {
            TileMeta m;
            m.kf = ldexpf(1.0f, -ek);
            m.e = (float)-ev;
            m.lf = sv2;
            m.any = ((bad[0] | bad[1] | bad[2] | bad[3]) != 0 ? 1u : 0u) | (mixed ? 2u : 0u);
#pragma unroll
            for (int i = 0; i < 4; ++i) m.bad[i] = bad[i];
            p.meta[item] = m;
        }
        // four words of each operand at a time, their loads together
        constexpr int N = 4;
        auto pass = [&](auto kb_, auto vb_, int i0) {
            constexpr int KB = kb_.value, VB = vb_.value;  // 0: as the pool says
            uint32_t k0[N], k1[N], v0[N], v1[N];
            uint16_t ks[N], kz[N], vs[N];
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int it = i0 + 256 * j, t = it / C8, c8 = it - t * C8, g = c8 >> 2;
                const int64_t r = rows[t];
                k0[j] = k1[j] = v0[j] = v1[j] = 0u;
                ks[j] = kz[j] = vs[j] = 0;
                if (r >= 0) {
                    const int kbyte = c8 * p.kb, vbit = 8 * c8 * p.vb;
                    const uint32_t *ka = reinterpret_cast<const uint32_t *>(p.k_codes + r * rbk + (kbyte & ~3));
                    const uint32_t *va = reinterpret_cast<const uint32_t *>(p.v_codes + r * rbv) + (vbit >> 5);
                    k0[j] = ka[0];
                    if ((kbyte & 3) + p.kb > 4) k1[j] = ka[1];
                    v0[j] = va[0];
                    if ((vbit & 31) + 8 * p.vb > 32) v1[j] = va[1];
                    ks[j] = p.k_scale[r * NG + g];
                    kz[j] = p.k_zero[r * NG + g];
                    vs[j] = p.v_scale[r * NG + g];
                }
            }
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int it = i0 + 256 * j, t = it / C8, c8 = it - t * C8;
                uint4 k4 = make_uint4(0u, 0u, 0u, 0u), l4 = k4, v4 = k4;
                if (rows[t] >= 0) {
                    float x[8];
                    key_values<KB>(k0[j], k1[j], ((c8 * p.kb) & 3) * 8, p.kb, f16_bits_to_f32(ks[j]) * (mixed ? row_k[t] : sk),
                                  magic - f16_bits_to_f32(kz[j]), x);
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        hi[i] = tc_pack_f16(x[2 * i], x[2 * i + 1]);
                        const float2 h2 = __half22float2(*reinterpret_cast<const __half2 *>(&hi[i]));
                        const float a = x[2 * i] - h2.x, b = x[2 * i + 1] - h2.y;  // (not finite where k is not: none)
                        lo[i] = tc_pack_f16(fabsf(a) < 1.0e30f ? a : 0.0f, fabsf(b) < 1.0e30f ? b : 0.0f);
                    }
                    k4 = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    l4 = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    if (!((bad[t >> 5] >> (t & 31)) & 1u)) {
                        value_values<VB>(v0[j], v1[j], (8 * c8 * p.vb) & 31, p.vb, f16_bits_to_f32(vs[j]) * (mixed ? row_v[t] : sv2), smem_addr(lut), x);
                        v4 = make_uint4(tc_pack_f16(x[0], x[1]), tc_pack_f16(x[2], x[3]), tc_pack_f16(x[4], x[5]), tc_pack_f16(x[6], x[7]));
                    }
                }
                *reinterpret_cast<uint4 *>(dst + kmaj_off(wT, t, 8 * c8)) = k4;
                *reinterpret_cast<uint4 *>(dst + KT + kmaj_off(wT, t, 8 * c8)) = l4;
                *reinterpret_cast<uint4 *>(dst + 2 * KT + mnmaj_off<D>(t, 8 * c8)) = v4;
            }
        };
        // the common widths at compile time: a prompt of 4096 tokens, 4-bit keys, takes 175 us
        // so and 179 with run-time shifts, 8191 tokens with 8-bit keys 502 and 505
        using std::integral_constant;
#pragma unroll 1
        for (int i0 = tid; i0 < wT * C8; i0 += 256 * N) {
            if (p.vb == 3 && p.kb == 8) pass(integral_constant<int, 8>{}, integral_constant<int, 3>{}, i0);
            else if (p.vb == 3 && p.kb == 4) pass(integral_constant<int, 4>{}, integral_constant<int, 3>{}, i0);
            else pass(integral_constant<int, 0>{}, integral_constant<int, 0>{}, i0);
        }
    }
}

// ---------------------------------------------------------------- attend
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

// A tile whose rows have exponents of their own (their sizes are very unlike, so
// that one exponent would leave some of them too few of f16's bits): this
// column's true base-2 scores, value exponents added, in place of the products.
// The thread goes on with those as with any tile's; the weights' sum, whose terms
// need each row's value exponent, is taken here at the reference R that it will
// choose.  Out of line: rare, and its registers are not the common path's.
__device__ __noinline__ float mixed_tile(uint32_t t_s, const RowMeta *rm, float ie, int vis, float R)
{
    float mx = -INFINITY, sum = 0.0f;
#pragma unroll 1
    for (int c = 0; c < wT; c += 16) {
        uint32_t x[16];
        tc_ld16(t_s + c, x);
        tc_wait_ld();
        tc_pin(x);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const RowMeta r = rm[c + j];
            const float y = fmaf(__uint_as_float(x[j]), fmaxf(ie * r.kf, 1.17549435e-38f), r.e);
            x[j] = c + j < vis ? __float_as_uint(y) : 0xFF800000u;
            mx = fmaxf(mx, __uint_as_float(x[j]));
        }
        tc_st16(t_s + c, x);
    }
    tc_wait_st();
    if (mx > R + wTau) R = mx;
    const float add = R == -INFINITY ? 0.0f : wUp - R;
#pragma unroll 1
    for (int c = 0; c < wT; c += 16) {
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
__device__ __noinline__ void far_tile(uint32_t t_s, float f, float e)
{
#pragma unroll 1
    for (int c = 0; c < wT; c += 16) {
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

// Tensor memory holds S of both groups (128 columns each; P, f16, overwrites
// its first half) and O of both.  In one pass over a tile the issuing warp
// queues O_a += P_a V, S_a = Q_a K(next), then the same for the other group, so
// that one group's softmax runs under the other's products.  Shared memory has
// room for two tiles of hi and of values but for one of lo at head_dim 128: group
// a multiplies by lo last and group b first, so that its copy has the time of
// group b's hi and of a's next products by values and hi.  MMAs of one
// thread execute in order: S(t) complete says that P V(t - 1) is complete, so
// the softmax threads may rescale O between reading S(t) and handing over P(t)
// without a barrier of its own.
//
// The issuing warp runs as a whole with warp-uniform operands, one elected lane
// issuing (a lone thread with operands in ordinary registers took over 100
// cycles per MMA, more than the 64 that one of 128 x 128 x 16 takes to run).
// What runs once per block (q in, masks of the last tiles, un-rotation) is in
// short loops: unrolled over a row it was 10 us of instruction fetch a block.
template <int D>
__global__ void __launch_bounds__(wThreads, 1) wide_attend_kernel(const __grid_constant__ WideParams p)
{
    using A = WideGeo<D>;
    constexpr int KT = A::KT, NK = A::NK, NV = A::NV, NL = A::NL, PL = A::PL, LB = A::LB;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + A::OFF_BAR);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(bars + A::BARS);
    const uint32_t sb = smem_addr(smem), b0 = smem_addr(bars);
    const uint32_t kfull = b0, kempty = kfull + 8 * NK, vfull = kempty + 8 * NK, vempty = vfull + 8 * NV;
    const uint32_t lfull = vempty + 8 * NV, lempty = lfull + 8 * NL;
    const uint32_t qfull = lempty + 8 * NL, sfull = qfull + 16, pfull = sfull + 16, ofull = pfull + 32,
                   drained = ofull + 16;  // pfull: first halves, then second halves
    __shared__ WidePlace place[2][2];
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

    pdl_wait_primary();
    pdl_allow_dependents();
    const int64_t total = p.pl.line[0], per = p.pl.line[1];
    const int64_t x0 = blockIdx.x * per, x1 = imin64(total, x0 + per);
    if (x0 >= x1) return;
    if (tid == 0) {
        for (int i = 0; i < 2 * (NK + NL + NV); ++i) mbar_init(b0 + 8 * i, 1);
        for (int g = 0; g < 2; ++g) {
            mbar_init(qfull + 8 * g, 4);  // a warp each
            mbar_init(sfull + 8 * g, 1);
            mbar_init(pfull + 8 * g, 4);
            mbar_init(pfull + 16 + 8 * g, 4);
            mbar_init(ofull + 8 * g, 1);
        }
        mbar_init(drained, 1);
        fence_mbar_init();
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(tslot)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __reduce_max_sync(0xffffffffu, *tslot);  // (uniform)

    // registers: the softmax threads hold a row of scores each; 256 x 224 + 128 x 56 is what the launch has
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 9) {
            // ------------------------------------------------------------ tiles in
            if (lane == 0) {
                // copy i of a ring of `ring` slots, once what was there has been used
                auto copy = [&](uint32_t &i, uint32_t ring, uint32_t full, uint32_t empty, uint32_t at, const uint8_t *from,
                                uint32_t bytes) {
                    const uint32_t slot = i % ring;
                    if (i >= ring && !mbar_wait_bounded(empty + 8 * slot, (i / ring - 1) & 1, p.err)) return false;
                    mbar_arrive_expect_tx(full + 8 * slot, bytes);
                    bulk_g2s(sb + at + slot * bytes, from, bytes, full + 8 * slot);
                    ++i;
                    return true;
                };
                bool ok = true;
                uint32_t nk = 0, nl = 0, nv = 0;  // copies made
                WidePlace w = wide_locate(p, x0);
                for (int n; ok && (n = w.count(x1)) > 0; wide_next(p, w)) {
                    const uint8_t *src = p.tiles + ((int64_t)(w.tile0 + w.tile) * p.H + w.h) * (3 * KT);
                    for (int t = 0; t < n && ok; ++t, src += (int64_t)p.H * (3 * KT)) {
                        ok = copy(nk, NK, kfull, kempty, A::OFF_K, src, KT);
#pragma unroll
                        for (int i = 0; i < PL; ++i) ok = ok && copy(nl, NL, lfull, lempty, A::OFF_L, src + KT + i * LB, LB);
                        ok = ok && copy(nv, NV, vfull, vempty, A::OFF_V, src + 2 * KT, KT);
                    }
                    if (w.ends(x1)) break;
                }
                if (!ok) {  // copies still in flight land before the CTA ends (bounded)
                    auto land = [&](uint32_t n, uint32_t ring, uint32_t full) {
                        for (uint32_t i = n > ring ? n - ring : 0; i < n; ++i)
                            mbar_wait_bounded(full + 8 * (i % ring), (i / ring) & 1, p.err);
                    };
                    land(nk, NK, kfull);
                    land(nl, NL, lfull);
                    land(nv, NV, vfull);
                }
            }
            __syncwarp();
        } else if (warp == 8) {
            // ------------------------------------------------------------ MMAs
            constexpr uint32_t idesc_qk = tc_idesc(128, wT, 0), idesc_pv = tc_idesc(128, D, 1), SBO = (D / 64) * 1024;
            const uint32_t leader = tc_elect();
            // descriptors of the first q, key, low-term and value tile, low words (16-byte units are
            // added to them) and high words (the same for the key side's)
            const uint64_t d0 = tc_desc(sb, 16, 1024), v0 = tc_desc(sb + A::OFF_V, 1024, SBO);
            const uint32_t dq = (uint32_t)d0, dk = dq + (A::OFF_K >> 4), dl = dq + (A::OFF_L >> 4), dv = (uint32_t)v0;
            constexpr uint32_t hk = (uint32_t)(tc_desc_const(16, 1024) >> 32), hv = (uint32_t)(tc_desc_const(1024, SBO) >> 32);
            auto desc = [](uint32_t hi, uint32_t lo) { return (uint64_t)hi << 32 | lo; };
            auto wait = [&](uint32_t bar, uint32_t parity) {  // the same answer in every lane
                return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, p.err)) != 0;
            };
            // S_g = Q_g K(tile)^T: the first terms, and the low ones; `acc` where the others came before
            auto high = [&](int g, uint32_t tile, uint32_t acc) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t o = ((kk / 4) * (wT * 128) + (kk % 4) * 32) >> 4;
                    tc_mma_elected(leader, tmem + g * wT, desc(hk, dq + (g * KT >> 4) + o), desc(hk, dk + (tile % NK * KT >> 4) + o), idesc_qk,
                                   kk > 0 ? 1u : acc);
                }
            };
            auto low = [&](int g, uint32_t tile, int i, uint32_t acc) {  // piece i
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    tc_mma_elected(leader, tmem + g * wT, desc(hk, dq + ((g * KT + i * LB + kk * 32) >> 4)),
                                   desc(hk, dl + (((tile * PL + i) % NL * LB + kk * 32) >> 4)), idesc_qk, kk > 0 ? 1u : acc);
            };
            // group a takes the low terms last and group b first: their slots are free for the next
            // tile's a good way before that needs them
            auto qk_a = [&](uint32_t tile) {
                if (!wait(kfull + 8 * (tile % NK), (tile / NK) & 1)) return false;
                tc_fence_after();
                high(0, tile, 0);
#pragma unroll 1
                for (int i = 0; i < PL; ++i) {
                    const uint32_t j = tile * PL + i;
                    if (!wait(lfull + 8 * (j % NL), (j / NL) & 1)) return false;
                    low(0, tile, i, 1);
                }
                return true;
            };
            auto qk_b = [&](uint32_t tile, bool two) {
#pragma unroll 1
                for (int i = 0; i < PL; ++i) {
                    if (two) low(1, tile, i, i > 0);
                    tc_commit_elected(leader, lempty + 8 * ((tile * PL + i) % NL));
                }
                if (two) high(1, tile, 1);
                tc_commit_elected(leader, sfull + 8);
                tc_commit_elected(leader, kempty + 8 * (tile % NK));
            };
            auto pv = [&](int g, uint32_t vs, int half, uint32_t acc) {
#pragma unroll
                for (int kk = 0; kk < wT / 32; ++kk) {
                    const int k = half * (wT / 32) + kk;
                    tc_mma_ts_elected(leader, tmem + A::O_COL + g * D, tmem + g * wT + k * 8,
                                      desc(hv, dv + (vs * KT >> 4) + (k * 2 * SBO >> 4)), idesc_pv, kk > 0 ? 1u : acc);
                }
            };
            bool ok = true;
            uint32_t it = 0, seg = 0;
            WidePlace w = wide_locate(p, x0);
            for (;;) {
                const int left = w.count(x1);
                const int n = (int)__reduce_max_sync(0xffffffffu, left > 0 ? (unsigned)left : 0u);
                if (n == 0) break;
                const bool two = __any_sync(0xffffffffu, w.n * p.G - (int64_t)(w.e - w.e0) * wC > 128) != 0;  // both groups have columns
                // the idle group's threads keep step through the same barriers
                ok = wait(qfull, seg & 1) && qk_a(it);
                if (!ok) break;
                tc_commit_elected(leader, sfull);
                ok = wait(qfull + 8, seg & 1);
                if (!ok) break;
                tc_fence_after();
                qk_b(it, two);
                for (int t = 0; t < n; ++t, ++it) {
                    const bool more = t + 1 < n;
                    const uint32_t vs = it % NV;
                    ok = wait(vfull + 8 * vs, (it / NV) & 1) && wait(pfull, it & 1);
                    if (!ok) break;
                    tc_fence_after();
                    pv(0, vs, 0, t > 0);
                    ok = wait(pfull + 16, it & 1);
                    if (!ok) break;
                    tc_fence_after();
                    pv(0, vs, 1, 1);
                    if (more) {
                        ok = qk_a(it + 1);
                        if (!ok) break;
                    }
                    tc_commit_elected(leader, more ? sfull : ofull);
                    ok = wait(pfull + 8, it & 1);
                    if (!ok) break;
                    tc_fence_after();
                    if (two) pv(1, vs, 0, t > 0);
                    ok = wait(pfull + 24, it & 1);
                    if (!ok) break;
                    tc_fence_after();
                    if (two) pv(1, vs, 1, 1);
                    tc_commit_elected(leader, vempty + 8 * vs);
                    if (more) qk_b(it + 1, two);
                    else tc_commit_elected(leader, ofull + 8);
                }
                if (!ok || __any_sync(0xffffffffu, w.ends(x1))) break;
                wide_next(p, w);
                ++seg;
            }
            if (!ok) {  // whatever was issued is through before tensor memory is given back (bounded)
                tc_commit_elected(leader, drained);
                mbar_wait_bounded(drained, 0, p.err);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        // ------------------------------------------------------------ softmax, one column a thread
        const int g = warp >> 2, ltid = tid & 127;
        const uint32_t lane_at = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t t_s = tmem + g * wT + lane_at, t_o = tmem + A::O_COL + g * D + lane_at;
        const uint32_t bar_s = sfull + 8 * g, bar_p = pfull + 8 * g;
        bool ok = true;
        uint32_t it = 0, seg = 0;
        int shared_from = -1;  // thread 0: the block of the last segment, if it is begun here and not finished
        // the place is kept in shared memory, out of the registers that hold scores, and the next
        // one worked out by the group's first thread while the first scores are awaited
        if (ltid == 0) place[g][0] = wide_locate(p, x0);
        for (;; ++seg) {
            // the place is written, and no wait of the group has given up: all leave together
            if (!named_and(1 + g, 128, ok)) break;
            const WidePlace &w = place[g][seg & 1];
            const int n = w.count(x1);
            if (n <= 0) break;
            const int cols = (int)w.n * p.G, col = (w.e - w.e0) * wC + 128 * g + ltid;  // total * QH < 2^30
            const bool real = col < cols;
            const int tok = real ? col / p.G : (int)w.n - 1, hq = real ? col - tok * p.G : 0;
            int left = (int)(w.len - w.n) + 1 + tok - w.tile * wT;  // rows that this column sees, from the tile's first on
            // q, scaled by a power of two that puts its largest |q| in [2^14, 2^15): exact in f16.
            // D / 8 lanes read a row of the warp's 32 together, every row under way before the first is used
            float ie = 0.0f;
            {
                constexpr int LR = D / 8, RI = 32 / LR, NI = 32 / RI;  // lanes per row, rows per step, steps
                const int64_t mine = real ? (w.s0 + tok) * p.pg.q_token + ((int64_t)w.h * p.G + hq) * p.pg.q_head : -1;
                const int c8 = lane % LR, sub = lane / LR;
                uint4 u[NI];
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const int64_t at = __shfl_sync(0xffffffffu, mine, i * RI + sub);
                    u[i] = at >= 0 ? *reinterpret_cast<const uint4 *>(p.q + at + 8 * c8) : make_uint4(0u, 0u, 0u, 0u);
                }
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const uint32_t m = 0x7FFF7FFFu;
                    const uint32_t b = bf16x2_max(bf16x2_max(u[i].x & m, u[i].y & m), bf16x2_max(u[i].z & m, u[i].w & m));
                    float mx = fmaxf(bf16_lo(b), bf16_hi(b));
#pragma unroll
                    for (int o = LR / 2; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                    int e = 0;
                    if (mx > 0.0f && mx < INFINITY) e = 14 - (((int)(__float_as_uint(mx) >> 23) & 0xFF) - 127);
                    e = e > 100 ? 100 : e;  // (-113 at least)
                    const float qs = __uint_as_float((uint32_t)(127 + e) << 23) * p.qsign;
                    const int er = __shfl_sync(0xffffffffu, e, (lane % RI) * LR);  // of row i RI + lane % RI
                    if (lane / RI == i) ie = __uint_as_float((uint32_t)(127 - er) << 23) * p.scale_log2;
                    const int r = 32 * (warp & 3) + i * RI + sub;
                    sts128(sb + g * KT + (c8 / 8) * (128 * 128) + (r / 8) * 1024 + (r % 8) * 128 + (((c8 % 8) ^ (r % 8)) * 16),
                           make_uint4(tc_pack_f16(bf16_lo(u[i].x) * qs, bf16_hi(u[i].x) * qs),
                                      tc_pack_f16(bf16_lo(u[i].y) * qs, bf16_hi(u[i].y) * qs),
                                      tc_pack_f16(bf16_lo(u[i].z) * qs, bf16_hi(u[i].z) * qs),
                                      tc_pack_f16(bf16_lo(u[i].w) * qs, bf16_hi(u[i].w) * qs)));
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(qfull + 8 * g);
            if (ltid == 0 && !w.ends(x1)) {  // (the other place was last read before this segment's barrier)
                WidePlace next = w;
                wide_next(p, next);
                place[g][(seg + 1) & 1] = next;
            }
            if (col + wC < cols) {  // the next block's q on its way to L2
                const int nt = (col + wC) / p.G;
                const uint16_t *a = p.q + (w.s0 + nt) * p.pg.q_token + ((int64_t)w.h * p.G + (col + wC - nt * p.G)) * p.pg.q_head;
                asm volatile("prefetch.global.L2 [%0];" ::"l"(a));
                if constexpr (D > 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(a + 64));
            }

            const TileMeta *mt = p.meta + ((int64_t)(w.tile0 + w.tile) * p.H + w.h);
            float R = -INFINITY, l = 0.0f;
            for (int t = 0; t < n; ++t, ++it, mt += p.H, left -= wT) {
                float e = mt->e, lf = mt->lf;
                // (a scale of zero: the smallest normal, so that hidden scores stay -inf)
                float f = fmaxf(ie * mt->kf, 1.17549435e-38f);
                const uint32_t any = mt->any;
                const int vis = left < 0 ? 0 : (left > wT ? wT : left);
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar_s, it & 1, p.err));
                if (!ok) break;
                tc_fence_after();
                float extra = 0.0f;
                if (!(any & 2u) && __any_sync(0xffffffffu, f > wFar)) {
                    far_tile(t_s, f, e);
                    f = 1.0f;
                    e = 0.0f;
                }
                if (any & 2u) {
                    // rows of exponents of their own: true scores now, and the sum of the weights
                    extra = mixed_tile(t_s, p.row_meta + (mt - p.meta) * wT, ie, vis, R);
                    f = 1.0f;
                    e = lf = 0.0f;
                } else if (__any_sync(0xffffffffu, vis < wT)) {  // some column does not see the whole tile: its hidden scores become -inf
#pragma unroll 1
                    for (int c = 0; c < wT; c += 16) {
                        uint32_t x[16];
                        tc_ld16(t_s + c, x);
                        tc_wait_ld();
                        tc_pin(x);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (c + j >= vis) x[j] = 0xFF800000u;
                        tc_st16(t_s + c, x);
                    }
                    tc_wait_st();
                }
                uint32_t sr[4][32];
                float2 ls[2];
                const float2 f2 = make_float2(f, f);
                // weights of 32 rows at the reference R, into tensor memory over the scores
                auto weights = [&](int c, float add) __attribute__((always_inline)) {
                    const float2 a2 = make_float2(add, add);
                    uint32_t pp[16];
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const float2 y = __ffma2_rn(make_float2(__uint_as_float(sr[c][j]), __uint_as_float(sr[c][j + 1])), f2, a2);
                        const float p0 = tc_ex2(y.x), p1 = tc_ex2(y.y);
                        ls[(j >> 1) & 1] = __fadd2_rn(ls[(j >> 1) & 1], make_float2(p0, p1));
                        pp[j / 2] = tc_pack_f16(p0, p1);
                    }
                    tc_st16(t_s + 16 * c, pp);
                };
                auto largest = [&](int c0) __attribute__((always_inline)) {  // of 64 scores
                    float a = -INFINITY, b = -INFINITY, d = -INFINITY, h = -INFINITY;
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        a = max3(a, __uint_as_float(sr[c0][j]), __uint_as_float(sr[c0][j + 1]));
                        b = max3(b, __uint_as_float(sr[c0][j + 2]), __uint_as_float(sr[c0][j + 3]));
                        d = max3(d, __uint_as_float(sr[c0 + 1][j]), __uint_as_float(sr[c0 + 1][j + 1]));
                        h = max3(h, __uint_as_float(sr[c0 + 1][j + 2]), __uint_as_float(sr[c0 + 1][j + 3]));
                    }
                    return fmaxf(fmaxf(a, b), fmaxf(d, h));
                };
                // the first half of P is handed over while the second is still worked on
                auto hand = [&](uint32_t bar) __attribute__((always_inline)) {
                    tc_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar);
                };
                tc_ld32(t_s, sr[0]);
                tc_ld32(t_s + 32, sr[1]);
                tc_wait_ld();
                tc_pin(sr[0]);
                tc_pin(sr[1]);
                tc_ld32(t_s + 64, sr[2]);
                tc_ld32(t_s + 96, sr[3]);
                const float m0 = largest(0);
                // the weights of the first half are taken at the R there is, and again where the
                // maximum has outgrown it (on a block's first tile, and seldom after)
                float add = R == -INFINITY ? 0.0f : e - R + wUp;
                bool checked = false;
#pragma unroll 1
                for (;;) {
                    ls[0] = ls[1] = make_float2(0.0f, 0.0f);
                    weights(0, add);
                    weights(1, add);
                    if (checked) break;
                    checked = true;
                    tc_wait_ld();
                    tc_pin(sr[2]);
                    tc_pin(sr[3]);
                    const float mx = fmaxf(m0, largest(2));
                    const float top = mx == -INFINITY ? -INFINITY : fmaf(mx, f, e);
                    if (!__any_sync(0xffffffffu, top > R + wTau)) break;
                    const float Rn = top > R + wTau ? top : R;
                    const float a = R == -INFINITY ? 0.0f : tc_ex2(R - Rn);  // nothing was summed before the first row seen
                    R = Rn;
                    l *= a;
                    if (t > 0)
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            uint32_t o[16];
                            tc_ld16(t_o + c, o);
                            tc_wait_ld();
                            tc_pin(o);
#pragma unroll
                            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * a);
                            tc_st16(t_o + c, o);
                        }
                    add = R == -INFINITY ? 0.0f : e - R + wUp;
                }
                hand(bar_p);
                weights(2, add);
                weights(3, add);
                hand(bar_p + 16);
                l = fmaf((ls[0].x + ls[0].y) + (ls[1].x + ls[1].y), lf, l + extra);
                if (any & 1u) {
#pragma unroll 1
                    for (int i = 0; i < 4; ++i) {
                        const int rows = vis - 32 * i;
                        const uint32_t seen = rows >= 32 ? 0xFFFFFFFFu : (rows <= 0 ? 0u : (1u << rows) - 1u);
                        if (mt->bad[i] & seen) l = NAN;
                    }
                }
            }
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(ofull + 8 * g, seg & 1, p.err));
            tc_fence_after();
            if (ok && n == w.tiles) {
                // the whole block: un-rotate, divide, round.  The Sylvester transform of D
                // values is one of D / 16 over stride 16, then one of 16: in tensor memory
                // between the two, 16 values of the row at a time
                constexpr int NS = D / 16;
#pragma unroll 1
                for (int j = 0; j < 16; j += 4) {
                    uint32_t x[NS][4];
#pragma unroll
                    for (int k = 0; k < NS; ++k) tc_ld4(t_o + 16 * k + j, x[k]);
                    tc_wait_ld();
#pragma unroll
                    for (int k = 0; k < NS; ++k) tc_pin(x[k]);
#pragma unroll
                    for (int hs = 1; hs < NS; hs <<= 1)
#pragma unroll
                        for (int k = 0; k < NS; k += 2 * hs)
#pragma unroll
                            for (int m = k; m < k + hs; ++m)
#pragma unroll
                                for (int q = 0; q < 4; ++q) {
                                    const float u = __uint_as_float(x[m][q]), v = __uint_as_float(x[m + hs][q]);
                                    x[m][q] = __float_as_uint(u + v);
                                    x[m + hs][q] = __float_as_uint(u - v);
                                }
#pragma unroll
                    for (int k = 0; k < NS; ++k) tc_st4(t_o + 16 * k + j, x[k]);
                }
                tc_wait_st();
                const float inv = l == 0.0f ? 0.0f : p.inv_sqrt_d / l;
                const int tk = real ? col / p.G : 0;
                uint16_t *dst = p.out + ((w.s0 + tk) * p.QH + (int64_t)w.h * p.G + (real ? col - tk * p.G : 0)) * D;
#pragma unroll 2
                for (int c = 0; c < D; c += 16) {
                    uint32_t x[16];
                    tc_ld16(t_o + c, x);
                    tc_wait_ld();
                    tc_pin(x);
                    float y[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) y[j] = __uint_as_float(x[j]);
#pragma unroll
                    for (int hs = 1; hs < 16; hs <<= 1)
#pragma unroll
                        for (int k = 0; k < 16; k += 2 * hs)
#pragma unroll
                            for (int m = k; m < k + hs; ++m) {
                                const float u = y[m], v = y[m + hs];
                                y[m] = u + v;
                                y[m + hs] = u - v;
                            }
                    const uint32_t sg = p.sg.w[c >> 5] >> (c & 16);
                    uint32_t u[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        u[i] = pack_bf16x2(__uint_as_float(__float_as_uint(y[2 * i] * inv) ^ (sg << (31 - 2 * i) & 0x80000000u)),
                                           __uint_as_float(__float_as_uint(y[2 * i + 1] * inv) ^ (sg << (30 - 2 * i) & 0x80000000u)));
                    if (real) st_global_v8(dst + c, u[0], u[1], u[2], u[3], u[4], u[5], u[6], u[7]);
                }
            } else if (ok) {
                // a share of a block: slot 2 c of a CTA when the block began in an earlier one, else 2 c + 1
                const int64_t at = ((int64_t)2 * blockIdx.x + (w.tile == 0 ? 1 : 0)) * wC + 128 * g + ltid;
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                    uint32_t x[16];
                    tc_ld16(t_o + c, x);
                    tc_wait_ld();
                    tc_pin(x);
                    float *dst = p.part_o + at * D + c;
                    st_global_v8(dst, x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]);
                    st_global_v8(dst + 8, x[8], x[9], x[10], x[11], x[12], x[13], x[14], x[15]);
                }
                p.part_ml[2 * at] = R - wUp;  // R = -inf (nothing seen): weight 0
                p.part_ml[2 * at + 1] = l;
                if (tid == 0 && w.tile == 0) {
                    shared_from = w.e - w.e0;
                    p.pl.share[blockIdx.x] = WideShare{w.s, w.h, shared_from, (int)((w.at + w.tiles - 1) / per)};
                }
            }
            tc_fence_before();
            if (w.ends(x1)) break;
        }
        if (tid == 0 && shared_from < 0) p.pl.share[blockIdx.x].last = -1;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// ---------------------------------------------------------------- merge
// Blocks (c, y) merge the shares of the block that CTA c began and did not
// finish, a warp per column (256 columns over 32 y x 8 warps): its (max, sum)
// pairs one a lane, 32 at a time, the first rows under way with them.  At most
// one block per CTA is shared, 36 MB of shares at head_dim 128; bound by the
// latency of three dependent loads (share, pair and row, store).
template <int D>
__global__ void __launch_bounds__(256) wide_merge_kernel(const __grid_constant__ WideParams p)
{
    constexpr int PER = D / 32, KF = 4;
    pdl_wait_primary();
    pdl_allow_dependents();
    const int64_t total = p.pl.line[0], per = p.pl.line[1], c = blockIdx.x;
    const WideShare w = p.pl.share[c];  // (under way with the line's words; one without work left none)
    if (c * per >= total || w.last < 0) return;
    const int lane = threadIdx.x & 31, i = blockIdx.y * 8 + (threadIdx.x >> 5);
    const int cnt = w.last - (int)c + 1;
    auto slot = [&](int k) { return (k == 0 ? 2 * c + 1 : 2 * (c + k)) * wC + i; };  // share k of the block
    float v[KF][PER];
#pragma unroll
    for (int k = 0; k < KF; ++k) {
        const float *src = p.part_o + slot(k) * D + PER * lane;
#pragma unroll
        for (int j = 0; j < PER; ++j) v[k][j] = k < cnt ? src[j] : 0.0f;
    }
    const int64_t s0 = paged_start(p.pg.v, w.s), n = paged_new(p.pg.v, w.s), col = (int64_t)w.block * wC + i;
    float m = -INFINITY, l = 0.0f, x[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) x[j] = 0.0f;
    for (int k0 = 0; k0 < cnt; k0 += 32) {
        float2 ml = make_float2(-INFINITY, 0.0f);
        if (k0 + lane < cnt) ml = *reinterpret_cast<const float2 *>(p.part_ml + 2 * slot(k0 + lane));
        float mx = ml.x;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        mx = fmaxf(m, mx);
        const float mu = mx == -INFINITY ? 0.0f : mx, keep = tc_ex2(m - mu), wt = tc_ex2(ml.x - mu);
        m = mx;
        l = l * keep + ml.y * wt;
#pragma unroll
        for (int j = 0; j < PER; ++j) x[j] *= keep;
        if (k0 == 0)
#pragma unroll
            for (int k = 0; k < KF; ++k) {
                const float f = __shfl_sync(0xffffffffu, wt, k);  // (0 past the last)
#pragma unroll
                for (int j = 0; j < PER; ++j) x[j] += v[k][j] * f;
            }
        const int end = cnt - k0 < 32 ? cnt - k0 : 32;
#pragma unroll 4
        for (int k = k0 == 0 ? KF : 0; k < end; ++k) {
            const float f = __shfl_sync(0xffffffffu, wt, k);
            const float *src = p.part_o + slot(k0 + k) * D + PER * lane;
#pragma unroll
            for (int j = 0; j < PER; ++j) x[j] += src[j] * f;
        }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    fwht_warp<PER>(x, lane);
    if (col >= n * p.G) return;  // past the sequence's columns: shares that nothing wrote
    const float inv = l == 0.0f ? 0.0f : p.inv_sqrt_d / l;
    const int64_t tok = col / p.G;
    uint32_t u[PER / 2];
#pragma unroll
    for (int k = 0; k < PER; k += 2)
        u[k / 2] = pack_bf16x2(x[k] * (sign_negative(p.sg, PER * lane + k) ? -inv : inv),
                               x[k + 1] * (sign_negative(p.sg, PER * lane + k + 1) ? -inv : inv));
    store_words<PER / 2, 2 * PER>(p.out + ((s0 + tok) * p.QH + (int64_t)w.h * p.G + (col - tok * p.G)) * D + PER * lane, u);
}

// ---------------------------------------------------------------- host side
// Most bytes of expanded tiles in a workspace.  Bounds that are far above a
// batch's real lengths (256 slots of up to 131072 rows, 8 kv-heads, head_dim 128)
// would ask for 200 GB of them; chunks over 1.4 M real rows at a time go by the
// expanded tiles, and further ones of such a call by the split kernels.
constexpr int64_t kWideScratch = int64_t(8) << 30;

struct WideSizes {
    int64_t tiles, entries;
    bool spills;  // there may be chunks that find no room
    size_t off_spill, off_tile0, off_entry0, off_before, off_line, off_share, off_meta, off_rows, off_ml, off_o, off_tiles, bytes;
};

WideSizes wide_sizes(const CacheView &c, const PagedBounds &b, int QH)
{
    WideSizes z{};
    const int64_t G = QH / c.H;
    const int64_t most = imin64(b.seqs, b.total / (b.wide + 1));  // sequences that can be wide
    const int64_t bound = imin64(most * ((b.max_len + wT - 1) / wT), b.total_len / wT + most);
    const int64_t tile_bytes = c.H * (3 * wT * c.d * 2 + wT * sizeof(RowMeta) + sizeof(TileMeta));
    z.tiles = imin64(bound, kWideScratch / tile_bytes);
    z.spills = z.tiles < bound;
    z.entries = b.total * G / wC + most;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t o = at;
        at += (n + 255) / 256 * 256;
        return o;
    };
    const size_t slots = 2 * (size_t)num_sms() * wC;
    z.off_spill = take((size_t)b.seqs * 4);
    z.off_tile0 = take((size_t)(b.seqs + 1) * 4);
    z.off_entry0 = take((size_t)(b.seqs + 1) * 4);
    z.off_before = take((size_t)(z.entries + 1) * 8);
    z.off_line = take(16);
    z.off_share = take((size_t)num_sms() * sizeof(WideShare));
    z.off_meta = take((size_t)z.tiles * c.H * sizeof(TileMeta));
    z.off_rows = take((size_t)z.tiles * c.H * wT * sizeof(RowMeta));
    z.off_ml = take(slots * 8);
    z.off_o = take(slots * c.d * 4);
    z.off_tiles = take((size_t)z.tiles * c.H * 3 * wT * c.d * 2);
    z.bytes = at;
    return z;
}

// The split kernel of the other sequences stands between expand and attend, their
// combine behind merge: each waits for all of the kernel before it.  (Split
// beside expand and combine beside merge, waiting at their ends, gained 2 to 10
// us a call; but then they read pool, lengths and partials without a wait of
// their own, which the programming model does not cover.)
template <int D>
cudaError_t wide_run(WideParams &p, cudaStream_t s, const std::function<cudaError_t()> &split)
{
    using A = WideGeo<D>;
    cudaError_t e = cudaFuncSetAttribute(wide_attend_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, A::SMEM);
    if (e != cudaSuccess) return e;
    e = launch_dependent(wide_plan_kernel, dim3(1), dim3(wPlanThreads), 0, s, p);
    if (e != cudaSuccess) return e;
    const int64_t items = p.max_tiles > 0 ? p.max_tiles * p.H : 1;
    e = launch_dependent(wide_expand_kernel<D>, dim3((unsigned)imin64(items, (int64_t)num_sms() * 8)), dim3(256), 0, s, p);
    if (e != cudaSuccess) return e;
    if ((e = split()) != cudaSuccess) return e;
    e = launch_dependent(wide_attend_kernel<D>, dim3((unsigned)p.ctas), dim3(wThreads), A::SMEM, s, p);
    if (e != cudaSuccess) return e;
    return launch_dependent(wide_merge_kernel<D>, dim3((unsigned)p.ctas, wC / 8), dim3(256), 0, s, p);
}

}  // namespace

bool paged_wide_applies(const CacheView &c) { return c.d == 64 || c.d == 128; }

size_t paged_wide_workspace_bytes(const CacheView &c, const PagedBounds &b, int QH) { return wide_sizes(c, b, QH).bytes; }

bool paged_wide_spills(const CacheView &c, const PagedBounds &b, int QH) { return wide_sizes(c, b, QH).spills; }

int32_t *paged_wide_spill(const CacheView &c, const PagedBounds &b, int QH, void *ws)
{
    const WideSizes z = wide_sizes(c, b, QH);
    return z.spills ? reinterpret_cast<int32_t *>(static_cast<uint8_t *>(ws) + z.off_spill) : nullptr;
}

cudaError_t launch_paged_wide(const CacheView &c, const PagedSplit &pg, const PagedBounds &b, const uint16_t *q, int QH,
                              float scale, uint16_t *out, void *ws, cudaStream_t s,
                              const std::function<cudaError_t()> &split)
{
    const WideSizes z = wide_sizes(c, b, QH);
    uint8_t *w = static_cast<uint8_t *>(ws);
    WideParams p{};
    p.pg = pg;
    p.pl = WidePlan{reinterpret_cast<int32_t *>(w + z.off_tile0), reinterpret_cast<int32_t *>(w + z.off_entry0),
                    reinterpret_cast<int64_t *>(w + z.off_before), reinterpret_cast<int64_t *>(w + z.off_line), reinterpret_cast<WideShare *>(w + z.off_share)};
    p.max_tiles = z.tiles;
    p.max_entries = z.entries;
    p.spill = paged_wide_spill(c, b, QH, ws);
    p.k_codes = c.k_codes;
    p.v_codes = c.v_codes;
    p.k_scale = c.k_scale;
    p.k_zero = c.k_zero;
    p.v_scale = c.v_scale;
    p.q = q;
    p.out = out;
    p.meta = reinterpret_cast<TileMeta *>(w + z.off_meta);
    p.row_meta = reinterpret_cast<RowMeta *>(w + z.off_rows);
    p.tiles = w + z.off_tiles;
    p.part_o = reinterpret_cast<float *>(w + z.off_o);
    p.part_ml = reinterpret_cast<float *>(w + z.off_ml);
    p.err = pg.v.err;
    p.H = c.H;
    p.QH = QH;
    p.G = QH / c.H;
    p.kb = c.kb;
    p.vb = c.vb;
    p.ctas = num_sms();
    p.scale_log2 = fabsf(scale) * 1.4426950408889634f;
    p.qsign = scale < 0.0f ? -1.0f : 1.0f;
    p.kcmax = c.kb == 8 ? 127.0f : (float)((1 << c.kb) - 1);
    p.inv_sqrt_d = inv_sqrt_head_dim(c.d);
    p.sg = c.signs;
    const Tables &tab = codebook_tables(c.vb);
    for (int i = 0; i < (1 << c.vb); ++i) {
        p.cen[i] = tab.centroids[i];
        p.cmax = p.cmax > fabsf(tab.centroids[i]) ? p.cmax : fabsf(tab.centroids[i]);
    }
    return c.d == 64 ? wide_run<64>(p, s, split) : wide_run<128>(p, s, split);
}

}  // namespace tq
