// tq_attention.cu -- fused dequantise-on-fetch GQA decode attention.
//
// Method: mlx-bun "TurboQuant -- rotation-based quantization", Part A:
// "Architecture in mlx-bun" (dequantize-on-fetch: attention reads the
// dequantised window; the token being generated is appended first), the
// "Algorithm" section (key and value dequantisation), and "Deferred inverse
// FWHT" (attention is linear in V, so the weighted sum is formed in the
// rotated domain and un-rotated once per query row).  GQA replicates whole
// kv-heads: q-head h reads kv-head h / G.
//
// GB300 design (one GPU, sm_103a), for head_dims 64, 128 and 256 with 8- or
// 4-bit keys and 2-, 3- or 4-bit values:
//  * Split-KV: CTA (split, kv-head, sequence) streams its token range through
//    a 2-stage shared-memory ring; each of its 2 warps takes two 16-token tiles
//    of a 64-token stage (four of a 128-token stage at head_dim 64, whose rows
//    are short; three of a 96-token stage at head_dim 128 with 4-bit keys) and
//    works on them at once (independent dependency chains to interleave).  A
//    stage is 2-D TMA loads of the key codes (boxes of at most 128 bytes per
//    row -- two at head_dim 256 with 8-bit keys -- with the swizzle of the box
//    width, so the per-row fragment reads of the MMA are bank-conflict-free)
//    and four 1-D bulk copies of the other planes, completing on the slot's
//    mbarrier; the last warp to finish a stage issues the copies that refill
//    its slot, so no warp is set aside as a producer (8 CTAs fit on an SM at
//    head_dims 64 and 128, 4 at 256).
//  * QK^T on tensor cores (mma.sync m16n8k16, f16 in, f32 accumulate): M = 16
//    tokens, N = 8 columns: 8 of the G q-heads sharing the kv-head, K =
//    head_dim.  A group above 8 has ceil(G/8) column blocks: at head_dims 64
//    and 128 a CTA takes two of them, so the key and value codes it unpacks
//    serve 16 columns (4 CTAs per SM at 128, for the doubled registers); at
//    256 each block is its own CTA, neighbours in the grid so their reads of
//    the same rows meet in L2.  Columns past G repeat the last head and are
//    dropped.  Key codes become exact f16 integers with one logic op each:
//    offset + code (a shift first for the upper bytes; 4-bit codes in odd
//    nibbles are read in place as 1024 + 16 code, their q taken / 16), so
//    S = sum_g scale_g * (acc_g + zero_g * sum_{j in g} q_j - offsets' share)
//    -- the per-group affine is applied to the 8-head scores, not to each
//    element.
//  * PV in the rotated domain (mma.sync, M = 16 dims, N = 8 heads, K = 16
//    tokens): value codes are mapped to f16 centroids by byte-permute table
//    lookups in registers (3 bits: four codes spread to nibbles per lookup;
//    2 bits: one f16 pair of the four centroids per lookup; 4 bits: the
//    magnitude index and sign of each code, the table being odd); the
//    per-group RMS scale is folded into P.
//  * Online softmax (base 2) per warp; warps merge in shared memory; each CTA
//    writes (max, sum, unnormalised o) per head.  A second kernel merges the
//    splits (log-sum-exp) and applies the inverse transform and signs once per
//    (sequence, q-head): the one below at head_dim 128, the generic kernel's
//    (same partial layout) at 64 and 256.
#include <mutex>

#include "tq_attention.cuh"

namespace tq {
namespace {

// ---------------------------------------------------------------- combine + deferred un-rotation
struct CombineParams {
    const float *part_o, *part_ml;
    float *out;  // [B][QH][D]
    int H, QH, G, NB, splits, rows;  // rows = B * QH
    float inv_sqrt_d;
    SignBits sg;  // value signs
};

// Each (sequence, q-head) row takes W warps (32 above 128 splits, 16 from 64,
// 4 from 16, else 1, so small merges are not spread thin); a CTA holds
// max(8, W) warps.  Lane holds dims
// 4 lane .. 4 lane + 3.  Warp w of a row merges the splits w, w + W, ...:
// up to kFew of them with every load issued before any is used (one memory
// round trip), more in chunks of 32 whose (max, sum) pairs are read one per
// lane, the weights 2^(m_s - m) computed one per lane and broadcast, and the
// chunk's output rows read with independent loads.  The row's first warp
// then merges its warps' results.
constexpr int kCombineWarps = 8;
constexpr int kFew = 8;
constexpr int kCombD = 128;  // head_dim of this merge (other head_dims take the generic kernel's)

__host__ __device__ constexpr int combine_cta_warps(int W) { return W > kCombineWarps ? W : kCombineWarps; }

template <int W>
__global__ void __launch_bounds__(combine_cta_warps(W) * 32) attn_combine_kernel(const __grid_constant__ CombineParams p)
{
    constexpr int CW = combine_cta_warps(W);
    __shared__ float4 wo[W > 1 ? CW : 1][32];
    __shared__ float wm[CW], wl[CW];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = blockIdx.x * (CW / W) + warp / W, wid = warp % W, lead = warp - wid;
    const bool live = row < p.rows;
    pdl_wait_primary();  // the split kernel's partials are complete and visible
    pdl_allow_dependents();
    if (W == 1 && !live) return;  // no barrier below when W = 1
    const int b = row / p.QH, qh = row % p.QH;
    const int h = qh / p.G, hq = qh % p.G;
    const int hh = hq % kG;  // column of block hq / kG
    const int64_t base = ((int64_t)b * p.H * p.NB + (int64_t)h * p.NB + hq / kG) * p.splits;
    // this warp's splits: wid + W i, i = 0 .. n_mine - 1
    const int n_mine = live && p.splits > wid ? (p.splits - wid + W - 1) / W : 0;
    auto split_index = [&](int i) { return (base + wid + (int64_t)W * i) * kG + hh; };
    float mw = -INFINITY;
    float4 xw = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float lw = 0.0f;
    if (n_mine <= kFew) {
        float2 ml = make_float2(-INFINITY, 0.0f);
        if (lane < n_mine) ml = *reinterpret_cast<const float2 *>(p.part_ml + 2 * split_index(lane));
        float4 v[kFew];
#pragma unroll
        for (int j = 0; j < kFew; ++j)
            v[j] = j < n_mine ? *reinterpret_cast<const float4 *>(p.part_o + split_index(j) * kCombD + 4 * lane)
                              : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        mw = ml.x;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) mw = fmaxf(mw, __shfl_xor_sync(0xffffffffu, mw, o));
        const float muw = mw == -INFINITY ? 0.0f : mw;
        const float wt = lane < n_mine ? ex2(ml.x - muw) : 0.0f;
        if (lane < n_mine) lw = ml.y * wt;
#pragma unroll
        for (int j = 0; j < kFew; ++j) {
            const float w = __shfl_sync(0xffffffffu, wt, j);
            xw.x += v[j].x * w; xw.y += v[j].y * w; xw.z += v[j].z * w; xw.w += v[j].w * w;
        }
    } else {
        for (int i = lane; i < n_mine; i += 32) mw = fmaxf(mw, p.part_ml[2 * split_index(i)]);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) mw = fmaxf(mw, __shfl_xor_sync(0xffffffffu, mw, o));
        const float muw = mw == -INFINITY ? 0.0f : mw;
        for (int i0 = 0; i0 < n_mine; i0 += 32) {
            // lane j: weight and sum of split i0 + j
            float wt = 0.0f;
            if (i0 + lane < n_mine) {
                const float2 ml = *reinterpret_cast<const float2 *>(p.part_ml + 2 * split_index(i0 + lane));
                wt = ex2(ml.x - muw);
                lw += ml.y * wt;
            }
            const int cnt = n_mine - i0 < 32 ? n_mine - i0 : 32;
#pragma unroll 8
            for (int j = 0; j < cnt; ++j) {
                const float w = __shfl_sync(0xffffffffu, wt, j);
                const float4 v = *reinterpret_cast<const float4 *>(p.part_o + split_index(i0 + j) * kCombD + 4 * lane);
                xw.x += v.x * w; xw.y += v.y * w; xw.z += v.z * w; xw.w += v.w * w;
            }
        }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, o);
    float x[4] = {xw.x, xw.y, xw.z, xw.w}, l = lw;
    if constexpr (W > 1) {
        wo[warp][lane] = xw;
        if (lane == 0) {
            wm[warp] = mw;
            wl[warp] = lw;
        }
        __syncthreads();
        if (wid != 0 || !live) return;
        float mmax = -INFINITY;
#pragma unroll
        for (int w = 0; w < W; ++w) mmax = fmaxf(mmax, wm[lead + w]);
        const float mu = mmax == -INFINITY ? 0.0f : mmax;
        l = 0.0f;
        x[0] = x[1] = x[2] = x[3] = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            // a warp without live splits carries zeros; the others rescale to the common max
            const float wt = wm[lead + w] == -INFINITY ? 0.0f : ex2(wm[lead + w] - mu);
            l += wl[lead + w] * wt;
            const float4 v = wo[lead + w][lane];
            x[0] += v.x * wt; x[1] += v.y * wt; x[2] += v.z * wt; x[3] += v.w * wt;
        }
    }
    const float inv_l = 1.0f / l;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] *= inv_l;
    // inverse transform: 2 stages in-lane, 5 across lanes (Sylvester order)
#pragma unroll
    for (int hs = 1; hs < 4; hs <<= 1)
#pragma unroll
        for (int i = 0; i < 4; i += 2 * hs)
#pragma unroll
            for (int j = i; j < i + hs; ++j) {
                const float a = x[j], bb = x[j + hs];
                x[j] = a + bb;
                x[j + hs] = a - bb;
            }
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const bool upper = (lane & m) != 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float other = __shfl_xor_sync(0xffffffffu, x[i], m);
            x[i] = upper ? other - x[i] : x[i] + other;
        }
    }
    float4 r;
    float *rr = &r.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int dim = 4 * lane + i;
        const bool neg = sign_negative(p.sg, dim);
        rr[i] = x[i] * (neg ? -p.inv_sqrt_d : p.inv_sqrt_d);
    }
    *reinterpret_cast<float4 *>(p.out + ((int64_t)b * p.QH + qh) * kCombD + 4 * lane) = r;
}

// ---------------------------------------------------------------- host side
struct SplitPlan {
    int splits;
    int64_t tokens_per_split;
};

SplitPlan plan_splits(int B, int H, int64_t seq_len, int ctas_per_sm, int stage_t)
{
    const int64_t units = (int64_t)B * H;
    const int64_t stages = (seq_len + stage_t - 1) / stage_t;
    const int64_t slots = (int64_t)num_sms() * ctas_per_sm;
    SplitPlan best{1, stages * stage_t};
    double best_cost = 1e300;
    for (int waves = 1; waves <= 16; ++waves) {
        int64_t s = (waves * slots + units - 1) / units;
        if (s < 1) s = 1;
        if (s > stages) s = stages;
        const int64_t per = (stages + s - 1) / s;  // stages per split
        const int64_t sp = (stages + per - 1) / per;
        const int64_t ctas = units * sp;
        const double cost = (double)((ctas + slots - 1) / slots) * (double)(per + 2);  // +2: fixed cost per CTA
        if (cost < best_cost - 1e-9) {
            best_cost = cost;
            best = SplitPlan{(int)sp, per * stage_t};
        }
    }
    return best;
}

// Launch the split kernel and the combine with a given split plan, the
// partials in `buf` (at least the plan's bytes; see plan_bytes).
template <int KB, int D, int VB, int NBC>
cudaError_t run_attention_plan(const CacheView &c, const uint16_t *q, int QH, int64_t seq_len, float scale, float *out,
                               void *buf, const SplitPlan &plan, cudaStream_t s)
{
    using A = AGeo<KB, D, VB, NBC>;
    if (plan.tokens_per_split % A::ST != 0) return cudaErrorInvalidValue;  // splits start on stage boundaries
    cudaError_t e =
        cudaFuncSetAttribute(attn_split_kernel<KB, D, VB, NBC>, cudaFuncAttributeMaxDynamicSharedMemorySize, A::SMEM);
    if (e != cudaSuccess) return e;
    const size_t need_o = (size_t)c.B * c.H * col_blocks(QH / c.H) * plan.splits * kG * D * 4;

    CUtensorMap map;
    if (!split_key_map<A>(c, A::ST, &map)) return cudaErrorInvalidValue;

    AttnParams p{};
    if (!attn_params<KB, VB>(c, q, QH, scale, p)) return cudaErrorInvalidDevice;
    p.part_o = static_cast<float *>(buf);
    p.part_ml = reinterpret_cast<float *>(static_cast<uint8_t *>(buf) + need_o);
    p.splits = plan.splits;
    p.seq_len = seq_len;
    p.tokens_per_split = plan.tokens_per_split;

    dim3 grid(plan.splits, c.H * ((p.NB + NBC - 1) / NBC), c.B);
    e = launch_dependent(attn_split_kernel<KB, D, VB, NBC>, grid, dim3(kThreads), A::SMEM, s, map, p);
    if (e != cudaSuccess) return e;
    if constexpr (D != kCombD)  // the generic kernel's merge: the same partial layout (one query row)
        return launch_attention_combine_parts(D, p.part_o, p.part_ml, out, c.B, c.H, QH, 1, p.NB, kG, plan.splits,
                                              c.signs, s);

    CombineParams cp{};
    cp.part_o = p.part_o;
    cp.part_ml = p.part_ml;
    cp.out = out;
    cp.H = c.H;
    cp.QH = QH;
    cp.G = QH / c.H;
    cp.NB = col_blocks(cp.G);
    cp.rows = c.B * QH;
    cp.splits = plan.splits;
    cp.inv_sqrt_d = inv_sqrt_head_dim(kCombD);
    cp.sg = c.signs;
    // the merge is a programmatic dependent of the split kernel: its CTAs take
    // SMs as split CTAs retire and wait for the whole split grid before reading
    const dim3 cb(kCombineWarps * 32);
    if (plan.splits > 128) return launch_dependent(attn_combine_kernel<32>, dim3(cp.rows), dim3(32 * 32), 0, s, cp);
    if (plan.splits >= 64) return launch_dependent(attn_combine_kernel<16>, dim3(cp.rows), dim3(16 * 32), 0, s, cp);
    if (plan.splits >= 16) return launch_dependent(attn_combine_kernel<4>, dim3((cp.rows + 1) / 2), cb, 0, s, cp);
    return launch_dependent(attn_combine_kernel<1>, dim3((cp.rows + 7) / 8), cb, 0, s, cp);
}

// Bytes of the split partials of a plan: (d output sums + max + sum) per
// column of each (sequence, kv-head, column block, split).
size_t plan_bytes(const CacheView &c, int QH, const SplitPlan &plan)
{
    return (size_t)c.B * c.H * col_blocks(QH / c.H) * plan.splits * kG * (c.d + 2) * 4;
}

// Column blocks per CTA: two where a kv-head has more than one block and the
// head_dim is at most 128 (at 256 the doubled registers would not fit), else one.
int blocks_per_cta(const CacheView &c, int QH) { return c.d <= 128 && col_blocks(QH / c.H) >= 2 ? 2 : 1; }

template <int D, int VB, int NBC>
int ctas_per_sm_dvn(const CacheView &c)
{
    return c.kb == 8 ? ctas_per_sm_for<8, D, VB, NBC>() : ctas_per_sm_for<4, D, VB, NBC>();
}

template <int D, int VB>
int ctas_per_sm_dv(const CacheView &c, int nbc)
{
    if constexpr (D <= 128)
        if (nbc == 2) return ctas_per_sm_dvn<D, VB, 2>(c);
    return ctas_per_sm_dvn<D, VB, 1>(c);
}

template <int D>
int ctas_per_sm_d(const CacheView &c, int nbc)
{
    return c.vb == 2 ? ctas_per_sm_dv<D, 2>(c, nbc) : c.vb == 4 ? ctas_per_sm_dv<D, 4>(c, nbc) : ctas_per_sm_dv<D, 3>(c, nbc);
}

int ctas_per_sm(const CacheView &c, int nbc)
{
    return c.d == 64 ? ctas_per_sm_d<64>(c, nbc) : c.d == 256 ? ctas_per_sm_d<256>(c, nbc) : ctas_per_sm_d<128>(c, nbc);
}

// Tokens per stage of the split kernel that serves this cache and group.
// (the stage size depends on the key width, head_dim and column blocks, not
// on the value width)
int stage_rows(const CacheView &c, int QH)
{
    const bool two = blocks_per_cta(c, QH) == 2;
    switch (c.d) {
    case 64:
        if (two) return c.kb == 8 ? AGeo<8, 64, 3, 2>::ST : AGeo<4, 64, 3, 2>::ST;
        return c.kb == 8 ? AGeo<8, 64, 3, 1>::ST : AGeo<4, 64, 3, 1>::ST;
    case 256: return c.kb == 8 ? AGeo<8, 256, 3, 1>::ST : AGeo<4, 256, 3, 1>::ST;
    default:
        if (two) return c.kb == 8 ? AGeo<8, 128, 3, 2>::ST : AGeo<4, 128, 3, 2>::ST;
        return c.kb == 8 ? AGeo<8, 128, 3, 1>::ST : AGeo<4, 128, 3, 1>::ST;
    }
}

SplitPlan usual_plan(const CacheView &c, int QH, int64_t seq_len)
{
    const int nbc = blocks_per_cta(c, QH);
    return plan_splits(c.B, c.H * ((col_blocks(QH / c.H) + nbc - 1) / nbc), seq_len, ctas_per_sm(c, nbc),
                       stage_rows(c, QH));
}

template <int D, int VB>
cudaError_t run_attention_dv(const CacheView &c, const uint16_t *q, int QH, int64_t seq_len, float scale, float *out,
                             void *buf, const SplitPlan &plan, cudaStream_t s)
{
    if constexpr (D <= 128) {
        if (blocks_per_cta(c, QH) == 2) {
            if (c.kb == 8) return run_attention_plan<8, D, VB, 2>(c, q, QH, seq_len, scale, out, buf, plan, s);
            return run_attention_plan<4, D, VB, 2>(c, q, QH, seq_len, scale, out, buf, plan, s);
        }
    }
    if (c.kb == 8) return run_attention_plan<8, D, VB, 1>(c, q, QH, seq_len, scale, out, buf, plan, s);
    return run_attention_plan<4, D, VB, 1>(c, q, QH, seq_len, scale, out, buf, plan, s);
}

template <int D>
cudaError_t run_attention_d(const CacheView &c, const uint16_t *q, int QH, int64_t seq_len, float scale, float *out,
                            void *buf, const SplitPlan &plan, cudaStream_t s)
{
    if (c.vb == 2) return run_attention_dv<D, 2>(c, q, QH, seq_len, scale, out, buf, plan, s);
    if (c.vb == 4) return run_attention_dv<D, 4>(c, q, QH, seq_len, scale, out, buf, plan, s);
    return run_attention_dv<D, 3>(c, q, QH, seq_len, scale, out, buf, plan, s);
}

cudaError_t run_attention(const CacheView &c, const uint16_t *q, int QH, int64_t seq_len, float scale, float *out,
                          void *buf, const SplitPlan &plan, cudaStream_t s)
{
    switch (c.d) {
    case 64: return run_attention_d<64>(c, q, QH, seq_len, scale, out, buf, plan, s);
    case 256: return run_attention_d<256>(c, q, QH, seq_len, scale, out, buf, plan, s);
    default: return run_attention_d<128>(c, q, QH, seq_len, scale, out, buf, plan, s);
    }
}

// The 4-bit lookup reads magnitudes and a sign: the table must be odd
// (c[15 - k] = -c[k], as the optimum for a symmetric density is).
bool four_bit_table_odd()
{
    const Tables &t = codebook_tables(4);
    for (int k = 0; k < 8; ++k)
        if (t.centroids[15 - k] != -t.centroids[k]) return false;
    return true;
}

}  // namespace

bool attention_supported(int d, int kb, int vb, int group)
{
    static const bool odd4 = four_bit_table_odd();
    return (d == 64 || d == 128 || d == 256) && (vb == 3 || vb == 2 || (vb == 4 && odd4)) && group >= 1 &&
           (kb == 8 || kb == 4);
}

size_t attention_workspace_bytes(const CacheView &c, int q_heads, int64_t seq_len)
{
    if (!attention_supported(c.d, c.kb, c.vb, q_heads / c.H)) return 0;
    return plan_bytes(c, q_heads, usual_plan(c, q_heads, seq_len));
}

cudaError_t launch_attention(const CacheView &c, const uint16_t *q, int q_heads, int64_t seq_len, float scale,
                             float *out, void *ws, size_t ws_bytes, cudaStream_t s)
{
    const SplitPlan plan = usual_plan(c, q_heads, seq_len);
    if (ws_bytes < plan_bytes(c, q_heads, plan)) return cudaErrorInvalidValue;
    return run_attention(c, q, q_heads, seq_len, scale, out, ws, plan, s);
}

}  // namespace tq

// ---------------------------------------------------------------- allocation-free variant
// Same kernels as launch_attention, but the split partials live in a fixed
// array that belongs to the library instead of a caller-provided workspace.
namespace tq {
namespace {

constexpr size_t kNoAllocScratchBytes = size_t(16) << 20;  // 16 MiB on every device that loads the library

// Holds the (max, sum, unnormalised output) partials of the splits.  Every
// call overwrites the part it uses before reading it, so nothing here has to
// start at zero; calls that overlap on the GPU share it and would race.
static __device__ __align__(256) uint8_t g_noalloc_scratch[kNoAllocScratchBytes];

constexpr int kMaxDevicesNoAlloc = 64;
std::mutex g_noalloc_mu;
void *g_noalloc_ptr[kMaxDevicesNoAlloc];

// Device address of the scratch array on the current device.  In host code
// the array's name is only a stand-in, so the address is looked up once per
// device (with that device current) and cached.
void *noalloc_scratch_address()
{
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevicesNoAlloc) return nullptr;
    std::lock_guard<std::mutex> lk(g_noalloc_mu);
    if (!g_noalloc_ptr[dev]) {
        void *ptr = nullptr;
        if (cudaGetSymbolAddress(&ptr, g_noalloc_scratch) != cudaSuccess || !ptr) return nullptr;
        g_noalloc_ptr[dev] = ptr;
    }
    return g_noalloc_ptr[dev];
}

}  // namespace

size_t noalloc_scratch_bytes() { return kNoAllocScratchBytes; }

bool noalloc_fits(const CacheView &c, int q_heads) { return plan_bytes(c, q_heads, SplitPlan{1, 0}) <= kNoAllocScratchBytes; }

cudaError_t launch_attention_noalloc(const CacheView &c, const uint16_t *q, int q_heads, int64_t seq_len, float scale,
                                     float *out, cudaStream_t s)
{
    void *scratch = noalloc_scratch_address();
    if (!scratch) return cudaErrorInvalidSymbol;
    // the usual split plan, with fewer splits if its partials would not fit
    SplitPlan plan = usual_plan(c, q_heads, seq_len);
    const size_t per_split = plan_bytes(c, q_heads, SplitPlan{1, 0});
    const int64_t max_splits = (int64_t)(kNoAllocScratchBytes / per_split);
    if (max_splits < 1) return cudaErrorInvalidValue;
    if (plan.splits > max_splits) {
        const int st = stage_rows(c, q_heads);
        const int64_t stages = (seq_len + st - 1) / st;
        const int64_t per = (stages + max_splits - 1) / max_splits;
        plan = SplitPlan{(int)((stages + per - 1) / per), per * st};
    }
    return run_attention(c, q, q_heads, seq_len, scale, out, scratch, plan, s);
}

}  // namespace tq
