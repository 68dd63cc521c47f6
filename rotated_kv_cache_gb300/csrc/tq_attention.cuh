// tq_attention.cuh -- the specialised split-KV attention kernel: see
// tq_attention.cu for the method and the design.  Included by the contiguous
// launches (tq_attention.cu) and the paged ones (tq_paged_split_d<head_dim>.cu).
#pragma once
#include <cuda.h>
#include "tq_common.cuh"
#include "tq_kernels.h"
#include "tq_paged.cuh"

namespace tq {
namespace {

constexpr int kG = 8;              // MMA columns: a block of 8 of a kv-head's q-heads
constexpr int kCW = 2;             // warps per CTA (all compute; the last to finish a stage refills it)
constexpr int kThreads = kCW * 32;
constexpr int kStages = 2;         // ring depth (8 CTAs of 2 x 13 KB fit on an SM)
constexpr float kOffset8 = 1152.0f;  // 8-bit keys: f16 value = 1152 + signed code

__host__ __device__ constexpr int imin_int(int a, int b) { return a < b ? a : b; }
__host__ __device__ constexpr int round_up(int x, int a) { return (x + a - 1) / a * a; }

// blocks of kG q-heads (MMA columns) per kv-head
inline int col_blocks(int group) { return (group + kG - 1) / kG; }

// NBC: column blocks per CTA (2 at head_dims up to 128 when a kv-head has
// more than kG q-heads: the key and value codes are unpacked once for both)
template <int KB, int D, int VB, int NBC = 1>
struct AGeo {
    // 16-token tiles per warp and stage, worked on together, and tokens per
    // stage: with one column block, four at head_dim 64 and three at 128 with
    // 4-bit keys (short rows: the per-stage work is spread over more of them;
    // the registers and the 2-slot ring still fit 8 CTAs on an SM)
    static constexpr int TILES = NBC != 1 ? 2 : D == 64 ? 4 : (D == 128 && KB == 4) ? 3 : 2;
    static constexpr int ST = 16 * TILES * kCW;
    static constexpr int NG = D / 32;                          // groups per row
    static constexpr int KROW = D * KB / 8;                    // key code bytes per token
    static constexpr int SW = KROW < 128 ? KROW : 128;         // key box row bytes = swizzle span
    static constexpr int NBOX = KROW / SW;                     // key boxes per row
    static constexpr int RBV = D * VB / 8;                     // value code bytes per token
    static constexpr int K_BYTES = ST * KROW;
    static constexpr int SC_BYTES = ST * NG * 2;               // one fp16 plane
    static constexpr int V_BYTES = ST * RBV;
    static constexpr int OFF_K = 0;
    static constexpr int OFF_KS = K_BYTES;
    static constexpr int OFF_KZ = OFF_KS + SC_BYTES;
    static constexpr int OFF_VS = OFF_KZ + SC_BYTES;
    static constexpr int OFF_V = OFF_VS + SC_BYTES;
    static constexpr int STAGE = round_up(OFF_V + V_BYTES + 16, 1024);  // 1024: swizzle atom alignment
    static constexpr int MERGE = kCW * NBC * kG * (D + 2) * 4;        // per-warp partials (reuse the ring)
    static constexpr int RING = kStages * STAGE > MERGE ? kStages * STAGE : MERGE;
    static constexpr int SMEM = 1024 /*align slack*/ + RING + kStages * 8 /*full barriers*/ + kStages * 4 /*counters*/;
    // resident CTAs per SM the register budget is sized for (head_dim 256, or
    // two column blocks, hold twice the q fragments and output accumulators)
    static constexpr int MIN_BLOCKS = D * NBC >= 256 ? 4 : 8;
};

struct AttnParams {
    const uint16_t *k_scale, *k_zero, *v_scale;
    const uint8_t *v_codes;
    const uint16_t *q;  // [B][QH][D] bf16
    float *part_o;      // [B][H][S][G][D]
    float *part_ml;     // [B][H][S][G][2]
    int H, QH, G, NB, splits;  // G = QH / H q-heads per kv-head; NB = ceil(G / kG) column blocks
    int64_t cap, seq_len, tokens_per_split;
    float scale_log2;  // softmax_scale * log2(e)
    uint32_t *err;
    // value centroids as byte-permute tables: 3 bits -- low bytes of the f16
    // c0..c7 (tl0, tl1), then their high bytes (th0, th1); 2 bits -- the f16
    // c0, c1 (tl0) and c2, c3 (tl1); 4 bits -- low and high bytes of the f16
    // magnitudes c8..c15 (the table is odd: c[15 - k] = -c[k])
    uint32_t tl0, tl1, th0, th1;
    uint32_t k_const, k_flip;     // key byte -> f16 (1024 + byte ^ 0x80) as one logic op (see below)
    PagedSplit pg;                // paged launches (partials [slot][NBC kG][D], [..][2])
};

// ---------------------------------------------------------------- PTX helpers
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint2 lds64(uint32_t a)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}

__device__ __forceinline__ uint32_t lds32(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

// N consecutive 32-bit words of shared memory (N = 1, 2 or 4; the address aligned to 4 N bytes)
template <int N>
__device__ __forceinline__ void lds_words(uint32_t a, uint32_t (&w)[N])
{
    if constexpr (N == 1) {
        w[0] = lds32(a);
    } else if constexpr (N == 2) {
        const uint2 v = lds64(a);
        w[0] = v.x;
        w[1] = v.y;
    } else {
        static_assert(N == 4, "one, two or four words");
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(a));
    }
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// Byte permute, default mode (used as an 8-entry table lookup: each selector
// nibble 0..7 picks one byte of the table held in a and b).
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel)
{
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
    return d;
}

// Key codes -> a pair of exact f16 integers in one 3-input logic op: where
// k_const has a bit set the result takes k_flip's bit (the f16 exponent
// pattern of 1024), elsewhere the code bit xor k_flip's bit (0x80 turns an
// int8 code into offset binary).  The f16 value is 1024 + (offset) code.
__device__ __forceinline__ uint32_t kcvt(uint32_t w, const AttnParams &p)
{
    return (p.k_const & p.k_flip) | (~p.k_const & (w ^ p.k_flip));
}

// Right shift done on the multiply-add pipe (the integer/logic pipe is the
// bottleneck of this kernel): x >> k == high word of x * 2^(32-k).
template <int K>
__device__ __forceinline__ uint32_t shr_fma(uint32_t x)
{
    return __umulhi(x, 1u << (32 - K));
}

// ---------------------------------------------------------------- the split kernel
// MODE: 0 contiguous; 1 paged, one new token a sequence at most; 2 paged, any
// (masks for the rows that some column does not see: 43 instructions per warp and
// stage, 4 % of the time of a decode step); 3 paged, the new tokens seeing one
// another by their mask rows (a column's mask words are read in the tiles that
// hold new rows alone).
// Paged: the CTA runs the segments of its share of a paged batch one after
// another (tq_paged.cuh) instead of the grid's (split, column blocks,
// sequence).  A column is then one (new token, q-head) of the kv-head, a block
// NBC * kG of them; a stage arrives chunk by chunk, each lane of the refilling
// warp copying one (a chunk lies within a page).  32 sequences of 24577 .. 32769
// rows, 64 q-heads, 8-bit keys and 3-bit values: 334 us, 4.5 TB/s (the contiguous
// call on 32769 rows each 325 us, 5.2): the look-ups and chunks of a stage are 16 %
// more instructions.  Issue is active 48 % of the time and DRAM 46 %, at 3.2 warps a
// scheduler (125 registers a thread): each warp's chains of loads and dependent
// arithmetic take the time, so instructions count although the slots are not full.
template <int KB, int D, int VB, int NBC, int MODE = 0>
__global__ void __launch_bounds__(kThreads, AGeo<KB, D, VB, NBC>::MIN_BLOCKS)
    attn_split_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ AttnParams p)
{
    using A = AGeo<KB, D, VB, NBC>;
    constexpr bool PAGED = MODE != 0, CAUSAL = MODE == 2, TREE = MODE == 3;
    constexpr int NG = A::NG;
    constexpr int NH = NBC * kG;  // MMA columns of the CTA
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *stages = smem;
    float *merge = reinterpret_cast<float *>(smem);  // after the loop, reuses the ring
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + A::RING);
    uint32_t *done = reinterpret_cast<uint32_t *>(smem + A::RING + kStages * 8);
    const uint32_t full0 = smem_addr(bars);

    pdl_wait_primary();  // whatever the previous kernel on the stream writes or reads is settled
    pdl_allow_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // blockIdx.y = (kv-head, NBC blocks of kG q-heads); the CTAs of one kv-head
    // are neighbours in the grid, so their reads of the same rows meet in L2
    const int nbp = (p.NB + NBC - 1) / NBC;  // CTAs per kv-head
    __shared__ PagedWalk walk;  // PAGED only
    if constexpr (PAGED) {
        if (warp == 0) paged_walk_start(p.pg, walk, A::ST, NH, p.H, p.G, lane);
        __syncthreads();
        if (walk.seg[0].count <= 0) return;
    }
    bool ok = true;
    uint32_t turned = 0;  // paged: bit k set when slot k's barrier has been through an odd number of phases
    int nseg = 0;         // segments done
    bool more = false;    // another one follows
    do {
    const PagedSegment &seg = walk.seg[nseg & 1];
    const int split = blockIdx.x, hv = blockIdx.y, b = blockIdx.z;
    const int h = PAGED ? seg.h : hv / nbp, hb0 = PAGED ? 0 : (hv - h * nbp) * NBC;  // the CTA's first column block
    const int64_t bh = (int64_t)b * p.H + h;
    const int64_t t_begin = PAGED ? 0 : (int64_t)split * p.tokens_per_split;
    const int64_t t_end = PAGED ? 0 : imin64(p.seq_len, t_begin + p.tokens_per_split);
    // paged: the block's columns are col0 .. col0 + cols - 1; rows that column c sees, from the
    // segment's first row on
    auto block_cols = [&] { return imin_int(seg.n * p.G - seg.hb * NH, NH); };
    auto column_rows = [&](int c) {
        return (TREE ? seg.len : seg.len - seg.n + 1 + (seg.hb * NH + c) / p.G) - seg.first * A::ST;
    };
    // tree: which of the 32 rows from row r of the segment on column c sees
    [[maybe_unused]] auto tree_rows = [&](int c, int r) {
        const int64_t tok = seg.s0 + (seg.hb * NH + imin_int(c, block_cols() - 1)) / p.G;
        return paged_tree_bits(p.pg.masks + tok * p.pg.mask_words, r - (seg.len - seg.n - seg.first * A::ST), seg.n);
    };
    // row offsets within the split fit 32 bits: a split never holds 2^31 rows
    // (136 B per row at the smallest width would take 292 GB)
    const int split_rows = PAGED ? imin_int(column_rows(block_cols() - 1), seg.count * A::ST) : (int)(t_end - t_begin);
    const int n_stages = split_rows > 0 && (!PAGED || ok) ? (split_rows + A::ST - 1) / A::ST : 0;

    // paged: every lane of the warp calls; the page look-up is in the shadow of the stage that the other slot holds
    auto issue_paged = [&](int s, int at_slot) {
        const int page = paged_chunk_page(p.pg, seg, seg.first + s, lane);
        const int ru = p.pg.ru;
        const int live = (imin_int(A::ST, split_rows - s * A::ST) + ru - 1) / ru;  // chunks with rows to read
        const uint32_t st = smem_addr(stages + at_slot * A::STAGE), bar = full0 + 8 * at_slot;
        if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(live * ru * (A::KROW + 3 * NG * 2 + A::RBV)));
        __syncwarp();
        if (lane < live) {
            const int at = lane * ru;
            const uint32_t row = (uint32_t)paged_chunk_plane_row(p.pg, seg, p.H, page, seg.first + s, lane);
#pragma unroll
            for (int j = 0; j < A::NBOX; ++j)
                tma_load_2d(st + A::OFF_K + j * (A::ST * A::SW) + at * A::SW, &kmap, j * A::SW, (int)row, bar);
            bulk_g2s(st + A::OFF_KS + at * (NG * 2), p.k_scale + (size_t)row * NG, ru * NG * 2, bar);
            bulk_g2s(st + A::OFF_KZ + at * (NG * 2), p.k_zero + (size_t)row * NG, ru * NG * 2, bar);
            bulk_g2s(st + A::OFF_VS + at * (NG * 2), p.v_scale + (size_t)row * NG, ru * NG * 2, bar);
            bulk_g2s(st + A::OFF_V + at * A::RBV, p.v_codes + (size_t)row * A::RBV, ru * A::RBV, bar);
        }
    };

    // stage s -> ring slot s % kStages: one 2-D TMA load (key codes) and four
    // 1-D bulk copies (the other planes) completing on the slot's barrier
    auto issue = [&](int s) {
        const int slot = s % kStages;
        const int64_t t = t_begin + (int64_t)s * A::ST;
        const int rows = (int)imin64(A::ST, p.cap - t);  // multiple of 16
        const int64_t row0 = bh * p.cap + t;
        const uint32_t st = smem_addr(stages + slot * A::STAGE), bar = full0 + 8 * slot;
        mbar_arrive_expect_tx(bar, (uint32_t)(A::K_BYTES + rows * (3 * NG * 2 + A::RBV)));
#pragma unroll
        for (int j = 0; j < A::NBOX; ++j)  // key rows wider than 128 bytes arrive as several boxes
            tma_load_2d(st + A::OFF_K + j * (A::ST * A::SW), &kmap, j * A::SW, (int)row0, bar);
        bulk_g2s(st + A::OFF_KS, p.k_scale + row0 * NG, rows * NG * 2, bar);
        bulk_g2s(st + A::OFF_KZ, p.k_zero + row0 * NG, rows * NG * 2, bar);
        bulk_g2s(st + A::OFF_VS, p.v_scale + row0 * NG, rows * NG * 2, bar);
        bulk_g2s(st + A::OFF_V, p.v_codes + row0 * A::RBV, rows * A::RBV, bar);
    };
    if (threadIdx.x == 0 && (!PAGED || nseg == 0)) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            done[s] = 0;
        }
        fence_mbar_init();
        if constexpr (!PAGED)
            for (int s = 0; s < kStages && s < n_stages; ++s) issue(s);
    }
    if constexpr (PAGED) {
        __syncwarp();
        if (warp == 0)
            for (int s = 0; s < kStages && s < n_stages; ++s)
                issue_paged(s, s);
    }
    if (!PAGED || nseg == 0) __syncthreads();

    // ---------------------------------------------------------------- compute warps
    const int g = lane >> 2, c = lane & 3;
    // Q fragments (B operand of QK^T): head n = g; per k-step two f16x2 registers.
    // The dim order inside a 32-group is permuted to match how key codes unpack.
    uint32_t bq[NBC][2 * NG][2];
    float qs[NBC][NG][2];  // sum over group of the f16 (scaled) q, heads 2c and 2c+1
    float qo[NBC][KB == 4 ? NG : 1][2];  // 4-bit keys: the code offsets' share of the QK^T dot
    float ie[NBC][2];      // per head: 2^-e * softmax_scale * log2(e)
#pragma unroll
    for (int nb = 0; nb < NBC; ++nb) {
        // columns past the last q-head are padding (a whole block of them past the
        // last block): they repeat head G-1 (MMA columns never mix) and their
        // partials are never written
        const int gq = kG * (hb0 + nb) + g;
        const uint16_t *qrow;
        if constexpr (PAGED) {
            const int col = seg.hb * NH + imin_int(gq, block_cols() - 1), qi = col / p.G;
            qrow = p.q + (seg.s0 + qi) * p.pg.q_token + ((int64_t)h * p.G + (col - qi * p.G)) * p.pg.q_head;
        } else {
            qrow = p.q + ((int64_t)b * p.QH + (int64_t)h * p.G + (gq < p.G ? gq : p.G - 1)) * D;
        }
        float qv[NG][8];
        float qoff[NG];
        float mx = 0.0f;
#pragma unroll
        for (int G = 0; G < NG; ++G) {
            const uint4 w = *reinterpret_cast<const uint4 *>(qrow + 32 * G + 8 * c);
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                qv[G][2 * i] = bf16_lo(ww[i]);
                qv[G][2 * i + 1] = bf16_hi(ww[i]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fabsf(qv[G][i]));
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // power-of-two scale so the largest |q| of the head lands in [2^14, 2^15)
        int e = 0;
        if (mx > 0.0f && mx < INFINITY) e = 14 - (((int)(__float_as_uint(mx) >> 23) & 0xFF) - 127);
        e = e > 100 ? 100 : e;  // (-113 at least)
        const float qscale = ldexpf(1.0f, e);
        float qsum[NG];
#pragma unroll
        for (int G = 0; G < NG; ++G) {
            float f[8];
            uint32_t hw[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                hw[i] = pack_f16x2(qv[G][2 * i] * qscale, qv[G][2 * i + 1] * qscale);
                const __half2 hv = *reinterpret_cast<const __half2 *>(&hw[i]);
                f[2 * i] = __low2float(hv);
                f[2 * i + 1] = __high2float(hv);
            }
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) s += f[i];
            qsum[G] = s;
            if constexpr (KB == 8) {
                // a word holds dims 8c+{0..3} (then {4..7}); its bytes pair as (0, 2), (1, 3)
                auto pr = [&](int i, int j) { return pack_f16x2(f[i], f[j]); };
                bq[nb][2 * G][0] = pr(0, 2);
                bq[nb][2 * G][1] = pr(1, 3);
                bq[nb][2 * G + 1][0] = pr(4, 6);
                bq[nb][2 * G + 1][1] = pr(5, 7);
            } else {
                // nibble k of the word = dim 8c+k; unpacked pairs are (k, k+4).  Odd
                // nibbles are read in place (1024 + 16 code), so their q is taken / 16
                auto pr = [&](int i, int j) { return pack_f16x2(f[i], f[j]); };
                auto pr16 = [&](int i, int j) { return pack_f16x2(f[i] * 0.0625f, f[j] * 0.0625f); };
                bq[nb][2 * G][0] = pr(0, 4);
                bq[nb][2 * G][1] = pr16(1, 5);
                bq[nb][2 * G + 1][0] = pr(2, 6);
                bq[nb][2 * G + 1][1] = pr16(3, 7);
                // the 1024 of every key element times the q it meets in the MMA
                const __half2 h1 = *reinterpret_cast<const __half2 *>(&bq[nb][2 * G][1]);
                const __half2 h3 = *reinterpret_cast<const __half2 *>(&bq[nb][2 * G + 1][1]);
                const float so = __low2float(h1) + __high2float(h1) + __low2float(h3) + __high2float(h3);
                qoff[G] = 1024.0f * (f[0] + f[2] + f[4] + f[6] + so);
            }
        }
        // group sums per head: head g lives in lanes 4g..4g+3; gather heads 2c, 2c+1
#pragma unroll
        for (int G = 0; G < NG; ++G) {
            float s = qsum[G];
            s += __shfl_xor_sync(0xffffffffu, s, 1);
            s += __shfl_xor_sync(0xffffffffu, s, 2);
            qs[nb][G][0] = __shfl_sync(0xffffffffu, s, (2 * c) * 4);
            qs[nb][G][1] = __shfl_sync(0xffffffffu, s, (2 * c + 1) * 4);
            if constexpr (KB == 4) {
                float so = qoff[G];
                so += __shfl_xor_sync(0xffffffffu, so, 1);
                so += __shfl_xor_sync(0xffffffffu, so, 2);
                qo[nb][G][0] = -__shfl_sync(0xffffffffu, so, (2 * c) * 4);
                qo[nb][G][1] = -__shfl_sync(0xffffffffu, so, (2 * c + 1) * 4);
            }
        }
        const float my_ie = ldexpf(1.0f, -e) * p.scale_log2;
        ie[nb][0] = __shfl_sync(0xffffffffu, my_ie, (2 * c) * 4);
        ie[nb][1] = __shfl_sync(0xffffffffu, my_ie, (2 * c + 1) * 4);
    }

    float o[NBC][2 * NG][4];
    float m_run[NBC][2], l_run[NBC][2];
#pragma unroll
    for (int nb = 0; nb < NBC; ++nb) {
#pragma unroll
        for (int i = 0; i < 2 * NG; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[nb][i][j] = 0.0f;
        m_run[nb][0] = m_run[nb][1] = -INFINITY;
        l_run[nb][0] = l_run[nb][1] = 0.0f;
    }

    // V field extraction: lane g owns dims 32G + 4g + {0..3}: 4 VB bits at bit
    // (32G + 4g) VB of the row (word 32G VB / 32 + v_word, shift v_shift)
    const int v_word = (4 * VB * g) >> 5, v_shift = (4 * VB * g) & 31;
    const int r0 = 16 * warp + g, r1 = r0 + 8;  // key rows of this lane in the warp's first tile
    const int vr[4] = {16 * warp + 2 * c, 16 * warp + 2 * c + 1, 16 * warp + 2 * c + 8, 16 * warp + 2 * c + 9};

    // lane-constant byte offsets in a stage: key bytes of row r0 per group (row r1 is
    // 8 rows on, the next tile 16 kCW rows on, rows SW bytes apart in a box; the
    // swizzle term is the same for all of them), value words of token vr[q] for
    // group 0 (group G is 12 G bytes on).  The swizzle of an SW-byte box row
    // xors the 16-byte chunk index with row % 8 (SW = 128), (row >> 1) % 4
    // (SW = 64) or (row >> 2) % 2 (SW = 32).
    const uint32_t xr = A::SW == 128 ? g : A::SW == 64 ? ((g >> 1) & 3) : ((g >> 2) & 1);
    uint32_t koff[NG];
#pragma unroll
    for (int G = 0; G < NG; ++G) {
        const int off = KB == 8 ? 32 * G + 8 * c : 16 * G + 4 * c;  // the lane's bytes of group G in the row
        const int box = off / A::SW, col = off % A::SW;
        koff[G] = A::OFF_K + box * (A::ST * A::SW) + r0 * A::SW + ((((uint32_t)col >> 4) ^ xr) << 4) + (col & 15);
    }
    uint32_t voff[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) voff[q] = A::OFF_V + vr[q] * A::RBV + 4 * v_word;
    const uint32_t ring0 = smem_addr(stages);
    // PAGED, several new tokens: rows from here on are hidden from some column
    const int first_hidden = TREE ? seg.len - seg.n - seg.first * A::ST : CAUSAL && seg.n > 1 ? column_rows(0) : INT32_MAX;
    if constexpr (!PAGED) ok = true;
    int slot = 0;
    uint32_t phase = 0;  // ring slot and barrier parity of stage s, from the segment's start
    int s = 0;
    for (; s < n_stages; ++s) {
        if (!mbar_wait_bounded(full0 + 8 * slot, PAGED ? phase ^ (turned >> slot & 1u) : phase, p.err)) {
            ok = false;
            break;
        }
        const uint32_t st = ring0 + slot * A::STAGE;
        // two 16-row tiles per warp and stage (rows 16 warp and 16 kCW + 16 warp): Q K^T for
        // both, one softmax step over both, P V for both; the tile loops are unrolled so
        // the compiler interleaves the tiles' independent chains
        float S[NBC][A::TILES][2][2];  // scores: [block][tile][row g, row g + 8][head 2c, 2c + 1]
#pragma unroll
        for (int t2 = 0; t2 < A::TILES; ++t2) {
            const int tile_r = s * A::ST + (16 * kCW) * t2 + 16 * warp;  // tile's first row from the split's start

            // ---------------- S = Q K^T for 16 tokens x 8 heads per block, per key group
            float acc[NBC][NG][4];
#pragma unroll
            for (int nb = 0; nb < NBC; ++nb)
#pragma unroll
                for (int G = 0; G < NG; ++G)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[nb][G][j] = 0.0f;
#pragma unroll
            for (int G = 0; G < NG; ++G) {
                uint32_t ka[2][4];  // A fragments of the group's two k-steps, shared by the blocks
                if constexpr (KB == 8) {
                    const uint2 k0 = lds64(st + koff[G] + t2 * ((16 * kCW) * A::SW));
                    const uint2 k1 = lds64(st + koff[G] + t2 * ((16 * kCW) * A::SW) + 8 * A::SW);
                    // bytes 0 and 2 (then 1 and 3) of a word -> f16 (1024 + (byte ^ 0x80)):
                    // dims (8c+0, 8c+2), (8c+1, 8c+3), then +4
                    ka[0][0] = kcvt(k0.x, p); ka[0][1] = kcvt(k1.x, p);
                    ka[0][2] = kcvt(shr_fma<8>(k0.x), p); ka[0][3] = kcvt(shr_fma<8>(k1.x), p);
                    ka[1][0] = kcvt(k0.y, p); ka[1][1] = kcvt(k1.y, p);
                    ka[1][2] = kcvt(shr_fma<8>(k0.y), p); ka[1][3] = kcvt(shr_fma<8>(k1.y), p);
                } else {
                    const uint32_t w0 = lds32(st + koff[G] + t2 * ((16 * kCW) * A::SW));
                    const uint32_t w1 = lds32(st + koff[G] + t2 * ((16 * kCW) * A::SW) + 8 * A::SW);
                    // nibbles k and k+4 -> f16: 1024 + nibble for even k, 1024 + 16 nibble
                    // (read in place) for odd k
                    const uint32_t v0 = shr_fma<8>(w0), v1 = shr_fma<8>(w1);
                    ka[0][0] = kcvt(w0, p); ka[0][1] = kcvt(w1, p);
                    ka[0][2] = (w0 & 0x00F000F0u) | 0x64006400u; ka[0][3] = (w1 & 0x00F000F0u) | 0x64006400u;
                    ka[1][0] = kcvt(v0, p); ka[1][1] = kcvt(v1, p);
                    ka[1][2] = (v0 & 0x00F000F0u) | 0x64006400u; ka[1][3] = (v1 & 0x00F000F0u) | 0x64006400u;
                }
#pragma unroll
                for (int nb = 0; nb < NBC; ++nb) {
                    mma16816(acc[nb][G], ka[0][0], ka[0][1], ka[0][2], ka[0][3], bq[nb][2 * G][0], bq[nb][2 * G][1]);
                    mma16816(acc[nb][G], ka[1][0], ka[1][1], ka[1][2], ka[1][3], bq[nb][2 * G + 1][0],
                             bq[nb][2 * G + 1][1]);
                }
            }
            // per-group affine applied to the scores: S = sum_g scale (acc + (zero - off) qsum),
            // both heads of the lane at once on packed fp32 pairs
            {
                // a row's NG fp16 scales (zero points) are NG / 2 words
                const uint32_t m0 = (r0 + (16 * kCW) * t2) * (NG * 2), m1 = (r1 + (16 * kCW) * t2) * (NG * 2);
                uint32_t sw[2][NG / 2], zw[2][NG / 2];
                lds_words(st + A::OFF_KS + m0, sw[0]);
                lds_words(st + A::OFF_KS + m1, sw[1]);
                lds_words(st + A::OFF_KZ + m0, zw[0]);
                lds_words(st + A::OFF_KZ + m1, zw[1]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float2 sacc[NBC];
#pragma unroll
                    for (int nb = 0; nb < NBC; ++nb) sacc[nb] = make_float2(0.0f, 0.0f);
#pragma unroll
                    for (int G = 0; G < NG; ++G) {
                        const uint16_t sh = (uint16_t)(sw[i][G >> 1] >> (16 * (G & 1)));
                        const uint16_t zh = (uint16_t)(zw[i][G >> 1] >> (16 * (G & 1)));
                        if constexpr (KB == 8) {
                            const float sc = f16_bits_to_f32(sh), zc = f16_bits_to_f32(zh) - kOffset8;
#pragma unroll
                            for (int nb = 0; nb < NBC; ++nb) {
                                const float2 t = __ffma2_rn(make_float2(zc, zc), make_float2(qs[nb][G][0], qs[nb][G][1]),
                                                            make_float2(acc[nb][G][2 * i], acc[nb][G][2 * i + 1]));
                                sacc[nb] = __ffma2_rn(make_float2(sc, sc), t, sacc[nb]);
                            }
                        } else {
                            const float sc = f16_bits_to_f32(sh), zc = f16_bits_to_f32(zh);
#pragma unroll
                            for (int nb = 0; nb < NBC; ++nb) {
                                const float2 t = __ffma2_rn(make_float2(zc, zc), make_float2(qs[nb][G][0], qs[nb][G][1]),
                                                            make_float2(acc[nb][G][2 * i], acc[nb][G][2 * i + 1]));
                                sacc[nb] = __ffma2_rn(make_float2(sc, sc), __fadd2_rn(t, make_float2(qo[nb][G][0], qo[nb][G][1])),
                                                      sacc[nb]);
                            }
                        }
                    }
#pragma unroll
                    for (int nb = 0; nb < NBC; ++nb) {
                        const float2 sv = __fmul2_rn(sacc[nb], make_float2(ie[nb][0], ie[nb][1]));
                        S[nb][t2][i][0] = sv.x;
                        S[nb][t2][i][1] = sv.y;
                    }
                }
                if (tile_r + 16 > split_rows) {  // ragged tail: mask rows past the range
#pragma unroll
                    for (int nb = 0; nb < NBC; ++nb) {
                        if (tile_r + g >= split_rows) S[nb][t2][0][0] = S[nb][t2][0][1] = -INFINITY;
                        if (tile_r + g + 8 >= split_rows) S[nb][t2][1][0] = S[nb][t2][1][1] = -INFINITY;
                    }
                }
                if constexpr (CAUSAL) {
                    if (tile_r + 16 > first_hidden) {
#pragma unroll
                        for (int nb = 0; nb < NBC; ++nb)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const int lim = column_rows(imin_int(kG * nb + 2 * c + j, block_cols() - 1)) - tile_r;  // rows of the tile it sees
                                if (g >= lim) S[nb][t2][0][j] = -INFINITY;
                                if (g + 8 >= lim) S[nb][t2][1][j] = -INFINITY;
                            }
                    }
                }
                if constexpr (TREE) {
                    if (tile_r + 16 > first_hidden) {
#pragma unroll
                        for (int nb = 0; nb < NBC; ++nb)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const uint32_t rows = tree_rows(kG * nb + 2 * c + j, tile_r) >> g;
                                if (!(rows & 1u)) S[nb][t2][0][j] = -INFINITY;
                                if (!(rows & 0x100u)) S[nb][t2][1][j] = -INFINITY;
                            }
                    }
                }
            }
        }
        // ---------------- online softmax (base 2) over the warp's tiles, heads 2c, 2c+1
        // The running max is reduced across the rows only when some lane sees a
        // score above it (or no max exists yet); otherwise the weights are
        // 2^(S - m) with the max unchanged, which is the same arithmetic.
        float pr[NBC][A::TILES][2][2];
#pragma unroll
        for (int nb = 0; nb < NBC; ++nb) {
            bool raise = m_run[nb][0] == -INFINITY || m_run[nb][1] == -INFINITY;
#pragma unroll
            for (int t2 = 0; t2 < A::TILES; ++t2)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    raise = raise || S[nb][t2][i][0] > m_run[nb][0] || S[nb][t2][i][1] > m_run[nb][1];
            if (__any_sync(0xffffffffu, raise)) {
                float alpha[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float mt = fmaxf(S[nb][0][0][j], S[nb][0][1][j]);
#pragma unroll
                    for (int t2 = 1; t2 < A::TILES; ++t2) mt = fmaxf(mt, fmaxf(S[nb][t2][0][j], S[nb][t2][1][j]));
                    mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 4));
                    mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 8));
                    mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 16));
                    const float mn = fmaxf(m_run[nb][j], mt);
                    const float mu = mn == -INFINITY ? 0.0f : mn;
                    alpha[j] = ex2(m_run[nb][j] - mu);
                    m_run[nb][j] = mn;
                    float ls = 0.0f;
#pragma unroll
                    for (int t2 = 0; t2 < A::TILES; ++t2) {
                        pr[nb][t2][0][j] = ex2(S[nb][t2][0][j] - mu);
                        pr[nb][t2][1][j] = ex2(S[nb][t2][1][j] - mu);
                        ls += pr[nb][t2][0][j] + pr[nb][t2][1][j];
                    }
                    l_run[nb][j] = l_run[nb][j] * alpha[j] + ls;
                }
                // o[mt][0, 1] and o[mt][2, 3] are (head 2c, head 2c+1) pairs
                const float2 a2 = make_float2(alpha[0], alpha[1]);
#pragma unroll
                for (int mt2 = 0; mt2 < 2 * NG; ++mt2) {
                    const float2 x = __fmul2_rn(make_float2(o[nb][mt2][0], o[nb][mt2][1]), a2);
                    const float2 y = __fmul2_rn(make_float2(o[nb][mt2][2], o[nb][mt2][3]), a2);
                    o[nb][mt2][0] = x.x;
                    o[nb][mt2][1] = x.y;
                    o[nb][mt2][2] = y.x;
                    o[nb][mt2][3] = y.y;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float ls = 0.0f;
#pragma unroll
                    for (int t2 = 0; t2 < A::TILES; ++t2) {
                        pr[nb][t2][0][j] = ex2(S[nb][t2][0][j] - m_run[nb][j]);
                        pr[nb][t2][1][j] = ex2(S[nb][t2][1][j] - m_run[nb][j]);
                        ls += pr[nb][t2][0][j] + pr[nb][t2][1][j];
                    }
                    l_run[nb][j] += ls;
                }
            }
        }
#pragma unroll
        for (int t2 = 0; t2 < A::TILES; ++t2) {
            const int tile_r = s * A::ST + (16 * kCW) * t2 + 16 * warp;  // tile's first row from the split's start
            // ---------------- P^T as the B operand (tokens x heads), transposed in registers
            uint32_t pt0[NBC], pt1[NBC];
#pragma unroll
            for (int nb = 0; nb < NBC; ++nb) {
                pt0[nb] = movmatrix_trans(pack_f16x2(pr[nb][t2][0][0], pr[nb][t2][0][1]));  // tokens 2c, 2c+1; head g
                pt1[nb] = movmatrix_trans(pack_f16x2(pr[nb][t2][1][0], pr[nb][t2][1][1]));  // tokens 2c+8, 2c+9
            }
            // value scales of this lane's four tokens, NG / 2 words each (zero past the range)
            uint32_t vs[4][NG / 2];
#pragma unroll
            for (int q = 0; q < 4; ++q) lds_words(st + A::OFF_VS + (vr[q] + (16 * kCW) * t2) * (NG * 2), vs[q]);
            if (tile_r + 16 > split_rows) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (tile_r + (vr[q] - 16 * warp) >= split_rows)
#pragma unroll
                        for (int k = 0; k < NG / 2; ++k) vs[q][k] = 0u;
            }
            // paged: a hidden row's rms may be anything; the weights of the lane's column (g of
            // each block) keep to the rows it sees
            uint32_t seen[NBC][2];
            const bool masked = (CAUSAL || TREE) && tile_r + 16 > first_hidden;
            if constexpr (TREE) {
                if (masked) {
#pragma unroll
                    for (int nb = 0; nb < NBC; ++nb) {
                        const uint32_t rows = tree_rows(kG * nb + g, tile_r) >> (2 * c);  // rows 2c, 2c + 1, 2c + 8, 2c + 9
                        seen[nb][0] = (rows & 1u ? 0xFFFFu : 0u) | (rows & 2u ? 0xFFFF0000u : 0u);
                        seen[nb][1] = (rows & 0x100u ? 0xFFFFu : 0u) | (rows & 0x200u ? 0xFFFF0000u : 0u);
                    }
                }
            }
            if constexpr (CAUSAL) {
                if (masked) {
#pragma unroll
                    for (int nb = 0; nb < NBC; ++nb) {
                        const int lim = column_rows(imin_int(kG * nb + g, block_cols() - 1)) - tile_r + 16 * warp;
                        seen[nb][0] = (vr[0] < lim ? 0xFFFFu : 0u) | (vr[1] < lim ? 0xFFFF0000u : 0u);
                        seen[nb][1] = (vr[2] < lim ? 0xFFFFu : 0u) | (vr[3] < lim ? 0xFFFF0000u : 0u);
                    }
                }
            }
            // ---------------- O^T += V^T P'^T, per value group.  P' = weight x rms is f16: 2^-12 of
            // it, and an absolute 2^-25 below 2^-14, which values of 2^-13 and less notice
            // (an exponent of their own would take the stage's largest rms before its products)
#pragma unroll
            for (int G = 0; G < NG; ++G) {
                const uint32_t sel = (G & 1) ? 0x7632u : 0x5410u;
                const uint32_t sp0 = __byte_perm(vs[0][G >> 1], vs[1][G >> 1], sel);
                const uint32_t sp1 = __byte_perm(vs[2][G >> 1], vs[3][G >> 1], sel);
                uint32_t b0[NBC], b1[NBC];
#pragma unroll
                for (int nb = 0; nb < NBC; ++nb) {
                    b0[nb] = hmul2(pt0[nb], sp0);
                    b1[nb] = hmul2(pt1[nb], sp1);
                    if constexpr (CAUSAL || TREE) {
                        if (masked) {
                            b0[nb] &= seen[nb][0];
                            b1[nb] &= seen[nb][1];
                        }
                    }
                }
                uint32_t av[2][2][2];  // [token pair][m-tile half][row g, row g+8]
                // the 4 VB-bit field (codes of dims 32G + 4g + 0..3 at bits 0, VB, 2 VB,
                // 3 VB) of the lane's four tokens; bits above 4 VB are don't-care
                uint32_t x[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t base = st + voff[q] + t2 * ((16 * kCW) * A::RBV) + 4 * VB * G;
                    if constexpr (VB == 3)  // 12-bit fields may straddle two words
                        x[q] = __funnelshift_r(lds32(base), lds32(base + 4), v_shift);
                    else  // 8- or 16-bit fields sit inside one word
                        x[q] = lds32(base) >> v_shift;
                }
#pragma unroll
                for (int pr2 = 0; pr2 < 2; ++pr2) {  // token pairs (2c, 2c+1) and (2c+8, 2c+9)
                    if constexpr (VB == 3) {
                        // both tokens' fields side by side (first in bits 0-15), then one
                        // code per nibble: codes r0..r3 of the first token in nibbles
                        // 0..3, of the second in nibbles 4..7
                        const uint32_t w = __byte_perm(x[2 * pr2], x[2 * pr2 + 1], 0x5410u);
                        const uint32_t y = (w & 0x003F003Fu) | ((w & 0x0FC00FC0u) * 4u);
                        // each byte of y holds two codes (bits 0-2, 3-5); adding the upper code
                        // to itself moves it to bits 4-6, and nothing carries out of a byte
                        const uint32_t e = y + (y & 0x38383838u);
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            // selector: codes (r, r+1) of the first token, then of the second
                            const uint32_t sel = __byte_perm(e, 0u, half ? 0x0031u : 0x0020u);
                            const uint32_t lo = prmt(p.tl0, p.tl1, sel);  // low f16 bytes of the 4 centroids
                            const uint32_t hi = prmt(p.th0, p.th1, sel);  // high f16 bytes
                            av[pr2][half][0] = __byte_perm(lo, hi, 0x6240u);  // dim r: (first, second)
                            av[pr2][half][1] = __byte_perm(lo, hi, 0x7351u);  // dim r + 1
                        }
                    } else if constexpr (VB == 2) {
                        // both tokens' bytes side by side; for dim r the two codes (a, b)
                        // pick the f16 pair (c[a], c[b]) out of c0..c3 in one permute:
                        // selector nibbles (2a, 2a+1, 2b, 2b+1)
                        const uint32_t u = __byte_perm(x[2 * pr2], x[2 * pr2 + 1], 0x0040u);
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const uint32_t ab = (u >> (2 * r)) & 0x0303u;
                            av[pr2][r >> 1][r & 1] = prmt(p.tl0, p.tl1, ab * 0x22u + 0x1010u);
                        }
                    } else {
                        // the two tokens' 16-bit fields side by side (a nibble per code);
                        // the table is odd, so a code is a magnitude index (code - 8 for
                        // code >= 8, 7 - code below) and a sign (negative below 8):
                        // t has bit 4i set where code i < 8, m the magnitude indices
                        const uint32_t u = __byte_perm(x[2 * pr2], x[2 * pr2 + 1], 0x5410u);
                        const uint32_t t = (~u >> 3) & 0x11111111u;
                        const uint32_t m = (u ^ (t * 7u)) & 0x77777777u;
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const uint32_t sel = __byte_perm(m, 0u, half ? 0x0031u : 0x0020u);
                            const uint32_t lo = prmt(p.tl0, p.tl1, sel), hi = prmt(p.th0, p.th1, sel);
                            // dim r = 2 half (+1): the two tokens' sign bits (bits 4r and 16 + 4r
                            // of t) moved to the f16 sign positions 15 and 31
                            const int r = 2 * half;
                            av[pr2][half][0] = __byte_perm(lo, hi, 0x6240u) ^ ((t << (15 - 4 * r)) & 0x80008000u);
                            av[pr2][half][1] = __byte_perm(lo, hi, 0x7351u) ^ ((t << (11 - 4 * r)) & 0x80008000u);
                        }
                    }
                }
#pragma unroll
                for (int half = 0; half < 2; ++half)
#pragma unroll
                    for (int nb = 0; nb < NBC; ++nb)
                        mma16816(o[nb][2 * G + half], av[0][half][0], av[0][half][1], av[1][half][0], av[1][half][1],
                                 b0[nb], b1[nb]);
            }
        }
        // the last warp to finish this stage refills its slot with stage s + kStages
        __syncwarp();
        if constexpr (PAGED) {
            uint32_t last = 0;
            if (lane == 0) {
                __threadfence_block();
                last = atomicAdd(&done[slot], 1u) == kCW - 1;
                if (last) done[slot] = 0;
            }
            if (__shfl_sync(0xffffffffu, last, 0) && s + kStages < n_stages) issue_paged(s + kStages, slot);
        } else if (lane == 0) {
            __threadfence_block();
            if (atomicAdd(&done[slot], 1u) == kCW - 1) {
                done[slot] = 0;
                if (s + kStages < n_stages) issue(s + kStages);
            }
        }
        if (++slot == kStages) {
            slot = 0;
            phase ^= 1u;
        }
    }
    if constexpr (PAGED) {
        // after a wait that gave up: the copies still in flight (bounded), and no further stage
        if (!ok)
            for (int r = s + 1; r < s + kStages && r < n_stages; ++r) {
                if (++slot == kStages) {
                    slot = 0;
                    phase ^= 1u;
                }
                mbar_wait_bounded(full0 + 8 * slot, phase ^ (turned >> slot & 1u), p.err);
            }
        ok = __syncthreads_and(ok);
#pragma unroll
        for (int k = 0; k < kStages; ++k) turned ^= ((uint32_t)(n_stages - k + kStages - 1) / kStages & 1u) << k;
    } else {
        __syncthreads();  // every warp is done with the ring before it holds the merge
    }

    // ---------------------------------------------------------------- merge the warps
    // per-lane partial row sums -> per-head sums (lanes with equal c)
#pragma unroll
    for (int nb = 0; nb < NBC; ++nb)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            l_run[nb][j] += __shfl_xor_sync(0xffffffffu, l_run[nb][j], 4);
            l_run[nb][j] += __shfl_xor_sync(0xffffffffu, l_run[nb][j], 8);
            l_run[nb][j] += __shfl_xor_sync(0xffffffffu, l_run[nb][j], 16);
        }
    float *mw = merge + warp * NH * (D + 2);  // [column][D] o, then [column] m, [column] l
#pragma unroll
    for (int nb = 0; nb < NBC; ++nb) {
#pragma unroll
        for (int mt = 0; mt < 2 * NG; ++mt) {
            const int G = mt >> 1, half = mt & 1;
            const int d0 = 32 * G + 4 * g + 2 * half;  // row g -> d0, row g+8 -> d0 + 1
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                mw[(kG * nb + 2 * c + j) * D + d0] = o[nb][mt][j];
                mw[(kG * nb + 2 * c + j) * D + d0 + 1] = o[nb][mt][2 + j];
            }
        }
        if (g == 0) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                mw[NH * D + kG * nb + 2 * c + j] = ok ? m_run[nb][j] : -INFINITY;
                mw[NH * D + NH + kG * nb + 2 * c + j] = ok ? l_run[nb][j] : 0.0f;
            }
        }
    }
    __syncthreads();
    // items (column, 8 dims), NH x D / 8 of them, over the CTA's threads
    for (int item = threadIdx.x; item < NH * (D / 8); item += kThreads) {
        const int hh = item / (D / 8), d8 = (item % (D / 8)) * 8;
        const int hb = hb0 + hh / kG;
        if (PAGED ? seg.slot >= p.pg.slots : hb >= p.NB) break;  // a padding block (columns are in block order)
        float mmax = -INFINITY;
#pragma unroll
        for (int w = 0; w < kCW; ++w) mmax = fmaxf(mmax, merge[w * NH * (D + 2) + NH * D + hh]);
        const float mu = mmax == -INFINITY ? 0.0f : mmax;
        float ov[8] = {0, 0, 0, 0, 0, 0, 0, 0}, lsum = 0.0f;
#pragma unroll
        for (int w = 0; w < kCW; ++w) {
            const float *m2 = merge + w * NH * (D + 2);
            const float wt = ex2(m2[NH * D + hh] - mu);
            lsum += m2[NH * D + NH + hh] * wt;
#pragma unroll
            for (int i = 0; i < 8; ++i) ov[i] += m2[hh * D + d8 + i] * wt;
        }
        const int64_t pidx = PAGED ? seg.slot * NH + hh
                                   : ((((int64_t)b * p.H + h) * p.NB + hb) * p.splits + split) * kG + hh % kG;
        float4 *dst = reinterpret_cast<float4 *>(p.part_o + pidx * D + d8);
        dst[0] = make_float4(ov[0], ov[1], ov[2], ov[3]);
        dst[1] = make_float4(ov[4], ov[5], ov[6], ov[7]);
        if (d8 == 0) {
            p.part_ml[2 * pidx] = mmax;
            p.part_ml[2 * pidx + 1] = lsum;
        }
    }
    if constexpr (PAGED) {
        if (threadIdx.x == 0) paged_walk_next(p.pg, walk, walk.seg[(nseg + 1) & 1], A::ST, NH, p.H, p.G);
        ++nseg;
        fence_proxy_async_smem();  // the next segment's copies land where the merge was read and written
        __syncthreads();
        more = walk.seg[nseg & 1].count > 0;
    }
    } while (PAGED && more);
}

// ---------------------------------------------------------------- host side
template <int KB, int D, int VB, int NBC, int MODE = 0>
int ctas_per_sm_for()
{
    static KernelSetup setup;
    int n;
    setup.get(attn_split_kernel<KB, D, VB, NBC, MODE>, kThreads, AGeo<KB, D, VB, NBC>::SMEM, AGeo<KB, D, VB, NBC>::SMEM, n);
    return n > 0 ? n : 1;  // (where the query failed, so will the launch)
}

// Tensor map over the key plane: rows of KROW bytes, boxes of SW bytes x rows.
template <typename A>
bool split_key_map(const CacheView &c, int rows, CUtensorMap *map)
{
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    const cuuint64_t gdim[2] = {(cuuint64_t)A::KROW, (cuuint64_t)c.B * c.H * c.cap};
    const cuuint64_t gstride[1] = {(cuuint64_t)A::KROW};
    const cuuint32_t box[2] = {(cuuint32_t)A::SW, (cuuint32_t)rows};
    const cuuint32_t estride[2] = {1, 1};
    const CUtensorMapSwizzle swz =
        A::SW == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : A::SW == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B;
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, c.k_codes, gdim, gstride, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
              swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The parameters that go by the cache alone.
template <int KB, int VB>
bool attn_params(const CacheView &c, const uint16_t *q, int QH, float scale, AttnParams &p)
{
    p.k_scale = c.k_scale;
    p.k_zero = c.k_zero;
    p.v_scale = c.v_scale;
    p.v_codes = c.v_codes;
    p.q = q;
    p.H = c.H;
    p.QH = QH;
    p.G = QH / c.H;
    p.NB = col_blocks(p.G);
    p.cap = c.cap;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.err = device_error_word();
    const Tables &tab = codebook_tables(VB);
    auto f16b = [](float x) { return (uint32_t)__half_as_ushort(__float2half_rn(x)); };
    if constexpr (VB == 2) {
        p.tl0 = f16b(tab.centroids[0]) | f16b(tab.centroids[1]) << 16;
        p.tl1 = f16b(tab.centroids[2]) | f16b(tab.centroids[3]) << 16;
    } else {
        // 3 bits: the eight centroids; 4 bits: the eight magnitudes c8..c15
        const int first = VB == 3 ? 0 : 8;
        uint32_t lo[8], hi[8];
        for (int i = 0; i < 8; ++i) {
            const uint32_t hb = f16b(tab.centroids[first + i]);
            lo[i] = hb & 0xFF;
            hi[i] = hb >> 8;
        }
        p.tl0 = lo[0] | lo[1] << 8 | lo[2] << 16 | lo[3] << 24;
        p.tl1 = lo[4] | lo[5] << 8 | lo[6] << 16 | lo[7] << 24;
        p.th0 = hi[0] | hi[1] << 8 | hi[2] << 16 | hi[3] << 24;
        p.th1 = hi[4] | hi[5] << 8 | hi[6] << 16 | hi[7] << 24;
    }
    // bits where R1 is set take R2; the others take byte ^ R2 (flip bit 7 and 23)
    p.k_const = KB == 8 ? 0xFF00FF00u : 0xFFF0FFF0u;
    p.k_flip = KB == 8 ? 0x64806480u : 0x64006400u;
    return p.err != nullptr;
}

}  // namespace
}  // namespace tq
