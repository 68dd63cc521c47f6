// tq_paged_attention.cu -- attention of ragged new tokens over a paged
// cache: the choice of kernels, the workspace, and the merge of the partials.
//
//   o_i = sum_{t seen by i} softmax_t(q_i . k_t scale) v_t
//
// for every new token i at position pos_i of its sequence, which sees the rows up
// to its own (causal), or the rows before the new ones and those that its mask
// names (trees of drafted tokens); the values stay in
// the rotated domain and the sum is un-rotated once per (token, q-head), as in
// the contiguous calls.  A token that sees no row gives zeros.
#include "tq_common.cuh"
#include "tq_kernels.h"
#include "tq_paged.cuh"

namespace tq {

#define TQ_DECLARE_PAGED_GENERIC(NAME)                                                                                 \
    bool paged_generic_shape_##NAME(const CacheView &c, int64_t cols, PagedShape &sh);                                 \
    cudaError_t launch_paged_generic_##NAME(const CacheView &c, const PagedSplit &pg, int64_t cols, const uint16_t *q, \
                                            int QH, float scale, float *part_o, float *part_ml, cudaStream_t s);
TQ_DECLARE_PAGED_GENERIC(d64)
TQ_DECLARE_PAGED_GENERIC(d128)
TQ_DECLARE_PAGED_GENERIC(d256)
TQ_DECLARE_PAGED_GENERIC(d512)
TQ_DECLARE_PAGED_GENERIC(d64_tree)
TQ_DECLARE_PAGED_GENERIC(d128_tree)
TQ_DECLARE_PAGED_GENERIC(d256_tree)
TQ_DECLARE_PAGED_GENERIC(d512_tree)
#undef TQ_DECLARE_PAGED_GENERIC
#define TQ_DECLARE_PAGED_SPLIT(NAME)                                                                                   \
    PagedShape paged_split_shape_##NAME(const CacheView &c, int64_t cols);                                             \
    cudaError_t launch_paged_split_##NAME(const CacheView &c, const PagedSplit &pg, const PagedShape &sh,              \
                                          const uint16_t *q, int QH, float scale, float *part_o, float *part_ml,       \
                                          cudaStream_t s);
TQ_DECLARE_PAGED_SPLIT(d64_one)
TQ_DECLARE_PAGED_SPLIT(d64_any)
TQ_DECLARE_PAGED_SPLIT(d128_one)
TQ_DECLARE_PAGED_SPLIT(d128_any)
TQ_DECLARE_PAGED_SPLIT(d256_one)
TQ_DECLARE_PAGED_SPLIT(d256_any)
TQ_DECLARE_PAGED_SPLIT(d64_tree)
TQ_DECLARE_PAGED_SPLIT(d128_tree)
TQ_DECLARE_PAGED_SPLIT(d256_tree)
#undef TQ_DECLARE_PAGED_SPLIT
#define TQ_DECLARE_PAGED_BLOCK(NAME)                                                                                   \
    bool paged_block_shape_##NAME(const CacheView &c, PagedShape &sh);                                                 \
    cudaError_t launch_paged_block_##NAME(const CacheView &c, const PagedSplit &pg, const PagedShape &sh,              \
                                          const uint16_t *q, int QH, float scale, float *part_o, float *part_ml,       \
                                          cudaStream_t s);
TQ_DECLARE_PAGED_BLOCK(d64)
TQ_DECLARE_PAGED_BLOCK(d128)
TQ_DECLARE_PAGED_BLOCK(d256)
#undef TQ_DECLARE_PAGED_BLOCK

namespace {

// ---------------------------------------------------------------- merge of the segments
struct PagedCombineParams {
    const float *part_o, *part_ml;
    uint16_t *out;  // bf16 [total][QH][D]
    PagedSplit pg;
    int H, QH, G, CB;
    int64_t rows;     // rows gone through: total * QH, or seqs * per_seq * QH
    int per_seq;      // > 0: that many places for tokens per sequence; 0: token by token
    float inv_sqrt_d;
    SignBits sg;
};

__device__ __forceinline__ float pc_ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// W warps per (token, q-head) row; lane holds dims PER lane .. + PER - 1.
// Warp w of a row takes its unit's segments w, w + W, ...: their (max, sum)
// pairs one a lane, 32 at a time, and their output rows with independent
// loads, the first ones under way with the pairs; the row's first warp merges the warps' results, divides, un-rotates
// (log2 d butterfly stages) and rounds once to bf16.  It moves one partial row
// per segment and does nothing else of size: bound by the latency of two
// dependent loads, so few rows take many warps (host rule below).
template <int D, int W>
__global__ void __launch_bounds__(W > 4 ? W * 32 : 128) paged_combine_kernel(const __grid_constant__ PagedCombineParams p)
{
    constexpr int PER = D / 32, CW = W > 4 ? W : 4;
    __shared__ float wo[W > 1 ? CW : 1][PER][32];
    __shared__ float wm[CW], wl[CW];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wid = warp % W, lead = warp - wid;
    const int64_t row = (int64_t)blockIdx.x * (CW / W) + warp / W;
    pdl_wait_primary();  // the partials are complete and visible
    pdl_allow_dependents();
    bool live = row < p.rows;
    int64_t t = live ? row / p.QH : 0;
    const int qh = (int)(row - t * p.QH), h = qh / p.G;
    int s = 0, col = 0;
    int64_t n = 0, len = 0, s0 = 0;
    PagedUnit unit{0, 0};  // slots of the row's unit: first .. first + count - 1
    auto load_unit = [&](int64_t i) {  // of token i of sequence s
        col = (int)i * p.G + (qh - h * p.G);
        const int hb = col / p.CB;
        if (hb < p.pg.blocks) unit = p.pg.units[((int64_t)s * p.H + h) * p.pg.blocks + hb];
        col -= hb * p.CB;
    };
    if (live && p.per_seq > 0) {
        s = (int)((uint32_t)t / (uint32_t)p.per_seq);
        t -= (int64_t)s * p.per_seq;
        load_unit(t);  // (under way with the lengths; written only where there are any)
        s0 = paged_start(p.pg.v, s);
        n = paged_new(p.pg.v, s);
        len = paged_len(p.pg.v, s);
        live = t < n && paged_split_takes(p.pg, s, n);
        t += s0;
    } else if (live) {
        int lo = 0, hi = p.pg.v.seqs + 1;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (p.pg.v.starts[mid] <= t) lo = mid + 1;
            else hi = mid;
        }
        s = lo - 1;
        live = s >= 0 && s < p.pg.v.seqs;  // else behind the last sequence: left as it was
        if (live) {
            s0 = paged_start(p.pg.v, s);
            n = paged_new(p.pg.v, s);
            len = paged_len(p.pg.v, s);
            live = t < s0 + n && paged_split_takes(p.pg, s, n);
            if (live) load_unit(t - s0);
        }
    }
    if (W == 1 && !live) return;  // no barrier below when W = 1
    // (a unit without a segment, or beyond the slots: starts out of order)
    const bool some = live && len > 0 && unit.first >= 0 && unit.count > 0 && unit.count <= p.pg.slots - unit.first;
    const int64_t first = unit.first;
    const int segs = some ? unit.count << p.pg.copies : 0, stride = p.CB >> p.pg.copies;  // partials; columns from one copy to the next
    const int mine = segs > wid ? (segs - wid + W - 1) / W : 0;
    auto part = [&](int j) {
        const int i = wid + W * j;
        return (first + (i >> p.pg.copies)) * p.CB + (i & ((1 << p.pg.copies) - 1)) * stride + col;
    };
    // the first rows are under way with their (max, sum) pairs
    constexpr int KF = PER <= 4 ? 4 : 2;
    float v[KF][PER];
#pragma unroll
    for (int j = 0; j < KF; ++j) {
        const float *src = p.part_o + part(j) * D + PER * lane;
#pragma unroll
        for (int k = 0; k < PER; ++k) v[j][k] = j < mine ? src[k] : 0.0f;
    }
    float m = -INFINITY, l = 0.0f, x[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) x[k] = 0.0f;
    for (int j0 = 0; j0 < mine; j0 += 32) {
        float2 ml = make_float2(-INFINITY, 0.0f);
        if (j0 + lane < mine) ml = *reinterpret_cast<const float2 *>(p.part_ml + 2 * part(j0 + lane));
        float mx = ml.x;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        mx = fmaxf(m, mx);
        const float mu = mx == -INFINITY ? 0.0f : mx, keep = pc_ex2(m - mu), wt = pc_ex2(ml.x - mu);
        m = mx;
        l = l * keep + ml.y * wt;
#pragma unroll
        for (int k = 0; k < PER; ++k) x[k] *= keep;
        const int cnt = mine - j0 < 32 ? mine - j0 : 32;
        if (j0 == 0)
#pragma unroll
            for (int j = 0; j < KF; ++j) {
                const float w = __shfl_sync(0xffffffffu, wt, j);  // (0 past the last)
#pragma unroll
                for (int k = 0; k < PER; ++k) x[k] += v[j][k] * w;
            }
#pragma unroll 4
        for (int j = j0 == 0 ? KF : 0; j < cnt; ++j) {
            const float w = __shfl_sync(0xffffffffu, wt, j);
            const float *src = p.part_o + part(j0 + j) * D + PER * lane;
#pragma unroll
            for (int k = 0; k < PER; ++k) x[k] += src[k] * w;
        }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if constexpr (W > 1) {
#pragma unroll
        for (int k = 0; k < PER; ++k) wo[warp][k][lane] = x[k];
        if (lane == 0) {
            wm[warp] = m;
            wl[warp] = l;
        }
        __syncthreads();
        if (wid != 0 || !live) return;
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < W; ++w) mx = fmaxf(mx, wm[lead + w]);
        const float mu = mx == -INFINITY ? 0.0f : mx;
        l = 0.0f;
#pragma unroll
        for (int k = 0; k < PER; ++k) x[k] = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float wt = pc_ex2(wm[lead + w] - mu);
            l += wl[lead + w] * wt;
#pragma unroll
            for (int k = 0; k < PER; ++k) x[k] += wo[lead + w][k][lane] * wt;
        }
    }
    const float inv = l == 0.0f ? 0.0f : p.inv_sqrt_d / l;  // nothing seen: zeros
    fwht_warp<PER>(x, lane);
    uint32_t w[PER / 2];
#pragma unroll
    for (int k = 0; k < PER; k += 2)
        w[k / 2] = pack_bf16x2(x[k] * (sign_negative(p.sg, PER * lane + k) ? -inv : inv),
                               x[k + 1] * (sign_negative(p.sg, PER * lane + k + 1) ? -inv : inv));
    store_words<PER / 2, PER * 2 < 16 ? PER * 2 : 16>(p.out + (t * p.QH + qh) * D + PER * lane, w);
}

template <int D>
cudaError_t run_combine(const PagedCombineParams &p, cudaStream_t s)
{
    // Fewer rows, more warps to each: enough warps to fill the SMs' issue slots
    // either way, and a row's partials in as few dependent loads as they allow.
    // A decode step with 64 q-heads over sequences of 4096 rows, split and merge,
    // in us with 1 / 4 / 16 warps to a row:
    //     1 sequence  (64 rows)    25.6 /  15.0 /  12.3
    //     8 sequences (512)        26.5 /  24.6 /  27.3
    //    64 sequences (4096)      106.2 / 111.7 / 139.7
    if (p.rows >= 4096)
        return launch_dependent(paged_combine_kernel<D, 1>, dim3((unsigned)((p.rows + 3) / 4)), dim3(128), 0, s, p);
    if (p.rows >= 512) return launch_dependent(paged_combine_kernel<D, 4>, dim3((unsigned)p.rows), dim3(128), 0, s, p);
    return launch_dependent(paged_combine_kernel<D, 16>, dim3((unsigned)p.rows), dim3(512), 0, s, p);
}

// ---------------------------------------------------------------- plan and workspace
bool generic_shape(const CacheView &c, int64_t cols, bool tree, PagedShape &sh)
{
    switch (c.d) {
    case 64: return tree ? paged_generic_shape_d64_tree(c, cols, sh) : paged_generic_shape_d64(c, cols, sh);
    case 128: return tree ? paged_generic_shape_d128_tree(c, cols, sh) : paged_generic_shape_d128(c, cols, sh);
    case 256: return tree ? paged_generic_shape_d256_tree(c, cols, sh) : paged_generic_shape_d256(c, cols, sh);
    case 512: return tree ? paged_generic_shape_d512_tree(c, cols, sh) : paged_generic_shape_d512(c, cols, sh);
    }
    return false;
}

struct PagedPlan {
    PagedShape split;
    bool special;   // the specialised split kernel, else the generic one
    bool block;     // the block kernel instead
    int copies;     // log2 of the times that it holds a column
    int64_t per_seq, cols;  // most new tokens of a sequence, and columns of a kv-head, that the split kernels see
    PagedBounds b;
    int64_t slots;
    int blocks;
    size_t off_ml, off_o, off_wide, bytes;  // workspace: units, partial (max, sum), partial outputs, the wide kernels'
};

// A sequence with at least this many columns (new tokens x q-heads of a
// kv-head) is wide, unless the whole batch is little work: the split kernel's
// time grows with rows x columns from nothing, the wide kernels' with rows from
// about 36 us (three launches more, a tile's first pass through the pipeline).
// Measured with 8-bit keys, 3-bit values, 8 kv-heads, head_dim 128 (64):
//   one sequence of 32768 rows   64 columns   split 81.8 us (51.3)  wide 122 (75.6)
//                               128                147.4    (87.8)       122 (75.2)
//                               256                280.4   (160.9)       124 (73.7)
//   one sequence of 2048 rows   128                 21.5    (19.3)       43.4 (36.1)
//                               512                 49.3    (33.6)       45.0 (35.8)
//   one prompt of 128 tokens   1024                 19.2    (16.7)       34.1 (27.9)
//                 256 tokens   2048                 45.7    (27.2)       36.2 (29.7)
//                 512 tokens   4096                115.7    (66.9)       41.4 (32.9)
// and at head_dim 128 with fewer kv-heads, whose blocks fill fewer CTAs:
//   2 kv-heads, 4096 rows       512 columns         29.2                 43.5
//               2048 rows      4096                 85.4                 45.2
//   1 kv-head,  2048 rows      4096                 49.7                 43.0
constexpr int64_t kWideColumns = 128;
constexpr int64_t kWideWork = int64_t(1) << 22;  // rows x kv-heads x columns, by the bounds that the host has

// The block kernel (tq_paged_block.cuh) takes the trees of a call when they have more
// columns than one pass of the split kernel, and enough rows to fill its
// pipelines; very many columns are worth the wide kernel's expanded rows.
// Measured (us), 8 kv-heads unless said, 8-bit keys, 3- or 4-bit values:
//   head_dim  sequences x rows  columns   block   split   wide
//      128       8 x 16384         16      92.6    89.2
//                                  24      92.7   158.8
//               32 x 28672         64     624    1950
//                1 x 512           64      16.8    13.7
//                1 x 2048          64      18.5    19.0
//               16 x 4352         384     218             298
//                                 512     292             302
//                                1024     558 (4-bit keys) 427
//       64       4 x 8192          24      29.4    32.2
//               16 x 4352         384     174             188
//                                 512     231             187
//      256       2 x 16384         12      41.3    49.3  (4 kv-heads, as below)
//                                 128      56.4   278.5
//                2 x 512           32      19.0    14.8
//                2 x 2048          32      22.4    22.5
// Ragged sequences, with the limit on the largest one's columns (4-bit keys; with 8-bit ones the wide kernel
// takes 5 to 25 us more):
//      128      16 x 500..8192   80..128  100             310
//                               200..320  197             233
//                               240..384  213             234
//                                 8..384  140             241
//                               320..512  320             262
//                8 x 500..32768 240..384  295             360
//               32 x 100..8192   32..384  400             449
//       64      16 x 500..8192  160..256  135             131
//                               240..384  157             166
//                               320..512  237             185
// Keys or values of other widths are cut by run-time shifts, straight from memory:
//      128       4 x 8192          32      60.1    56.7
//                                  64      61.3    95.4
//                                 384     159             164
constexpr int64_t kBlockWork = int64_t(1) << 20;  // rows x kv-heads x columns, by the bounds that the host has

bool takes_block(const CacheView &c, const PagedBounds &b, int64_t G)
{
    const int64_t most = b.max_new * G;  // columns of the largest sequence
    if (!b.tree || c.d > 256 || (int64_t)c.B * c.H * c.cap >= (int64_t(1) << 31)) return false;  // (its tensor copies count rows in 32 bits)
    const bool cut = (c.kb == 8 || c.kb == 4) && c.vb <= 4;
    if (most <= (!cut ? 32 : c.d == 256 ? 8 : 16)) return false;
    if (c.d <= 128 && most > 384) return false;
    return b.total_len >= (kBlockWork + c.H * most - 1) / (c.H * most);
}

bool block_shape(const CacheView &c, PagedShape &sh)
{
    return c.d == 64 ? paged_block_shape_d64(c, sh) : c.d == 128 ? paged_block_shape_d128(c, sh) : paged_block_shape_d256(c, sh);
}

bool paged_plan(const CacheView &c, const PagedBounds &bounds, int QH, PagedPlan &pl)
{
    const int64_t G = QH / c.H;
    pl.b = bounds;
    const int64_t most = pl.b.max_new * G;  // columns of the largest sequence
    const bool work = most >= kWideColumns && pl.b.total_len >= (kWideWork + c.H * most - 1) / (c.H * most);
    pl.block = takes_block(c, pl.b, G);
    pl.b.wide = paged_wide_applies(c) && work && !pl.block ? (kWideColumns - 1) / G : INT32_MAX;
    const bool wide = pl.b.wide != INT32_MAX;
    // new tokens of a sequence that the split kernels see, at most
    pl.per_seq = wide && !paged_wide_spills(c, pl.b, QH) ? (pl.b.wide > 0 ? pl.b.wide : 1) : pl.b.max_new;
    pl.cols = pl.per_seq * G;
    // the specialised kernel where it has the widths (its tensor copies count rows in 32 bits)
    pl.special = attention_supported(c.d, c.kb, c.vb, (int)G) && (int64_t)c.B * c.H * c.cap < (int64_t(1) << 31);
    pl.copies = 0;
    if (pl.block) {
        if (!block_shape(c, pl.split)) return false;
        pl.copies = most <= 64 ? (most <= 32 && c.d <= 128 ? 2 : 1) : 0;  // (of shares of 32 rows at least)
    } else if (pl.special)
        pl.split = pl.b.tree
                       ? (c.d == 64    ? paged_split_shape_d64_tree(c, pl.cols)
                          : c.d == 128 ? paged_split_shape_d128_tree(c, pl.cols)
                                       : paged_split_shape_d256_tree(c, pl.cols))
                   : pl.b.max_new <= 1
                       ? (c.d == 64    ? paged_split_shape_d64_one(c, pl.cols)
                          : c.d == 128 ? paged_split_shape_d128_one(c, pl.cols)
                                       : paged_split_shape_d256_one(c, pl.cols))
                       : (c.d == 64    ? paged_split_shape_d64_any(c, pl.cols)
                          : c.d == 128 ? paged_split_shape_d128_any(c, pl.cols)
                                       : paged_split_shape_d256_any(c, pl.cols));
    else if (!generic_shape(c, pl.cols, pl.b.tree, pl.split))
        return false;
    // a sequence of n new tokens has ceil(n G / block) blocks: at most this many units in all
    const int64_t units = c.H * (pl.b.total * G / pl.split.block + pl.b.seqs);
    pl.slots = pl.split.ctas + units;
    auto r256 = [](size_t x) { return (x + 255) / 256 * 256; };
    pl.blocks = (int)((pl.cols + pl.split.block - 1) / pl.split.block);
    pl.off_ml = r256((size_t)pl.b.seqs * c.H * pl.blocks * sizeof(PagedUnit));
    pl.off_o = pl.off_ml + r256((size_t)pl.slots * pl.split.block * 8);
    pl.off_wide = pl.off_o + r256((size_t)pl.slots * pl.split.block * c.d * 4);
    pl.bytes = pl.off_wide + (wide ? paged_wide_workspace_bytes(c, pl.b, QH) : 0);
    return true;
}

}  // namespace

size_t paged_attention_workspace_bytes(const CacheView &c, const PagedBounds &b, int QH)
{
    PagedPlan pl;
    return paged_plan(c, b, QH, pl) ? pl.bytes : 0;
}

cudaError_t launch_paged_attention(const CacheView &c, const PagedView &v, const PagedBounds &b, const uint16_t *q,
                                   const int64_t qs[2], int QH, float scale, const uint32_t *masks, int64_t mask_words,
                                   uint16_t *out, void *ws, size_t ws_bytes, cudaStream_t s)
{
    PagedPlan pl;
    if (!paged_plan(c, b, QH, pl)) return cudaErrorInvalidConfiguration;
    if (ws_bytes < pl.bytes) return cudaErrorInvalidValue;
    uint8_t *base = static_cast<uint8_t *>(ws);
    const bool wide = pl.b.wide != INT32_MAX;
    PagedSplit pg{v, qs[0], qs[1], reinterpret_cast<PagedUnit *>(base), pl.slots, pl.blocks, pl.b.max_new, pl.b.wide,
                  wide ? paged_wide_spill(c, pl.b, QH, base + pl.off_wide) : nullptr, 1, 1, masks, mask_words, pl.copies};
    float *part_ml = reinterpret_cast<float *>(base + pl.off_ml), *part_o = reinterpret_cast<float *>(base + pl.off_o);
    auto split = [&]() -> cudaError_t {
        const int64_t cols = pl.cols;
        if (pl.block) {
            const auto launch = c.d == 64 ? launch_paged_block_d64 : c.d == 128 ? launch_paged_block_d128 : launch_paged_block_d256;
            return launch(c, pg, pl.split, q, QH, scale, part_o, part_ml, s);
        }
        if (pl.special) {
            const auto launch = pl.b.tree
                                    ? (c.d == 64 ? launch_paged_split_d64_tree : c.d == 128 ? launch_paged_split_d128_tree : launch_paged_split_d256_tree)
                                : pl.b.max_new <= 1
                                    ? (c.d == 64 ? launch_paged_split_d64_one : c.d == 128 ? launch_paged_split_d128_one : launch_paged_split_d256_one)
                                    : (c.d == 64 ? launch_paged_split_d64_any : c.d == 128 ? launch_paged_split_d128_any : launch_paged_split_d256_any);
            return launch(c, pg, pl.split, q, QH, scale, part_o, part_ml, s);
        }
        const bool tree = pl.b.tree;
        const auto launch = c.d == 64    ? (tree ? launch_paged_generic_d64_tree : launch_paged_generic_d64)
                            : c.d == 128 ? (tree ? launch_paged_generic_d128_tree : launch_paged_generic_d128)
                            : c.d == 256 ? (tree ? launch_paged_generic_d256_tree : launch_paged_generic_d256)
                                         : (tree ? launch_paged_generic_d512_tree : launch_paged_generic_d512);
        return launch(c, pg, cols, q, QH, scale, part_o, part_ml, s);
    };
    const cudaError_t e = wide ? launch_paged_wide(c, pg, pl.b, q, QH, scale, out, base + pl.off_wide, s,
                                                   std::ref(split))  // (a reference: nothing allocated)
                               : split();
    if (e != cudaSuccess) return e;
    // by places per sequence where that goes through fewer rows (a decode step: no
    // search for a token's sequence; a long chunk: none of its tokens).  32
    // sequences of 4096 rows: 61.5 us so, 62.9 token by token
    const bool by_seq = v.seqs * pl.per_seq <= v.total;
    PagedCombineParams cp{part_o, part_ml, out, pg, c.H, QH, QH / c.H, pl.split.block,
                          (by_seq ? v.seqs * pl.per_seq : v.total) * QH, by_seq ? (int)pl.per_seq : 0, inv_sqrt_head_dim(c.d),
                          c.signs};
    switch (c.d) {
    case 64: return run_combine<64>(cp, s);
    case 128: return run_combine<128>(cp, s);
    case 256: return run_combine<256>(cp, s);
    case 512: return run_combine<512>(cp, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace tq
