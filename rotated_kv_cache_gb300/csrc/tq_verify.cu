// tq_verify.cu -- drafted tokens against the target's probabilities.
//
// A sequence's new tokens form a tree: node 0 is the token that is certain, the
// children of a node were drawn for the place behind it.  At an accepted node
// with target row p and draft row r, its children are tried in index order; one
// of token x with the random number u is accepted where
//   u r(x) M < max(p(x) - C r(x), 0),   C = 0, M = 1 at first,
// and a rejected one leaves the rest of the target's probabilities to the others:
// max(R - M r, 0) in place of R, where R sums to M.  Since
// max(max(p - a r, 0) - b r, 0) = max(p - (a + b) r, 0) for b r >= 0, what is
// left after any number of rejections is max(p - C r, 0) with one number C:
//   C += M,  M = sum_v max(p(v) - C r(v), 0)
// -- no division, and no row to keep.  Without draft probabilities (drafts that
// were not drawn at random: r is 1 at x) a rejected token is crossed out: M -= p(x),
// p(x) = 0.  When the children are through, the next token is drawn from what is
// left: the first v whose running sum passes last * sum (where nothing is left, the vocabulary's size).
//
// The sums decide which token comes out, so they are kept to 2^-45 or so: every
// addition is one of pairs of floats (sum and what its roundings left out, the
// product C r(v) in two parts).  64-bit additions would take this chip 64 times as
// long as 32-bit ones; they are left for the few numbers of a sequence.
//
// A cluster of CTAs goes through a row, a run of elements per warp, a run in up to
// four pieces with a sum each, so that the one that holds the drawn token is short.
// The first warp of the first CTA alone reads the tree and decides; all the others are told what
// to sum, so that no two of them can disagree on how often they meet.  A pass moves
// the row once: bound by memory for many sequences, by the latency of four
// dependent loads (tree, its tokens' entries, row, drawn piece) and of the
// cluster's barriers for few.
//
// 16 chains of 5 nodes, 32000 tokens, with draft probabilities: 12.7 us; 64 trees of 8
// to 32 nodes, 131072 tokens, without: 20.7 us (1.6 TB/s; 24.4 with a node's children
// looked up one after another).  With 64-bit sums by every
// thread of the deciding CTA and 32 KB runs searched element by element they took 32
// and 76; without the template for drafts, whose registers halve what is under way,
// 12.7 and 31.  Clusters of 4: 15 and 34; 512 threads: 23 and 85 (fewer CTAs fit).
// 64 chains with draft probabilities, 131072 tokens: 37.5 us (39.9 with eight pieces; a run's lines
// called to L2 ahead of its loads 43: the arithmetic of pairs bounds it).
#include "tq_common.cuh"
#include "tq_kernels.h"
#include "tq_paged.cuh"

namespace tq {
namespace {

constexpr int vfThreads = 256, vfWarps = vfThreads / 32;
constexpr int vfCluster = 8, vfRuns = vfWarps * vfCluster;  // warps to a sequence
constexpr int vfPieces = 4;                                 // of a run, at most

struct VerifyParams {
    VerifyCall c;
};

// What the CTAs of a cluster are to sum, as the first one says.
struct VerifyOrder {
    int64_t row;    // of target and draft; -1: nothing more
    double C;
    int gone;       // tokens crossed out (a list of the first CTA)
};

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// The address of `p` (shared memory) in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(const void *p, uint32_t rank)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    return a;
}

__device__ __forceinline__ int cluster_load(uint32_t a)
{
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ int64_t cluster_load64(uint32_t a)
{
    int64_t v;
    asm volatile("ld.shared::cluster.s64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ void cluster_store(uint32_t a, float2 v)
{
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(v.x), "f"(v.y) : "memory");
}

// A probability as it counts: neither negative, NaN nor infinite.
__device__ __forceinline__ float vf_clean(float x) { return x > 0.0f && x < INFINITY ? x : 0.0f; }

__device__ __forceinline__ float vf_at(const float *row, int64_t v) { return vf_clean(row[v]); }
__device__ __forceinline__ float vf_at(const uint16_t *row, int64_t v) { return vf_clean(__uint_as_float((uint32_t)row[v] << 16)); }

// A sum in two floats, s + e.
struct TwoSum {
    float s = 0.0f, e = 0.0f;
    __device__ __forceinline__ void add(float x)
    {
        const float t = __fadd_rn(s, x), z = __fsub_rn(t, s);
        e = __fadd_rn(e, __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(x, z)));
        s = t;
    }
    __device__ __forceinline__ void add(float x, float rest)
    {
        add(x);
        e = __fadd_rn(e, rest);
    }
    __device__ __forceinline__ double value() const { return (double)s + (double)e; }
};

__device__ __forceinline__ TwoSum warp_total(TwoSum x)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) x.add(__shfl_xor_sync(0xffffffffu, x.s, o), __shfl_xor_sync(0xffffffffu, x.e, o));
    return x;
}

__device__ __forceinline__ TwoSum warp_running(TwoSum x, int lane)  // the sum up to each lane
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float s = __shfl_up_sync(0xffffffffu, x.s, o), e = __shfl_up_sync(0xffffffffu, x.e, o);
        if (lane >= o) x.add(s, e);
    }
    return x;
}

// max(p - C r, 0) in two floats, C = c1 + c2
struct TwoFloat {
    float hi, lo;
};

__device__ __forceinline__ TwoFloat vf_left(float p, float r, float c1, float c2)
{
    const float m = __fmul_rn(c1, r), ml = __fmaf_rn(c2, r, __fmaf_rn(c1, r, -m));  // C r
    const float d = __fsub_rn(p, m), z = __fsub_rn(d, p);
    const float l = __fsub_rn(__fsub_rn(__fsub_rn(p, __fsub_rn(d, z)), __fadd_rn(m, z)), ml);
    const float hi = __fadd_rn(d, l), lo = __fadd_rn(__fsub_rn(d, hi), l);
    return hi > 0.0f ? TwoFloat{hi, lo} : TwoFloat{0.0f, 0.0f};
}

// A warp's run of a row: tiles of 32 E elements, counted from the 16-byte
// boundary at or before the row's start, so that a lane's E elements are one
// access wherever the row starts.
template <typename T, bool DRAFT>
struct VerifyRow {
    static constexpr int E = 16 / sizeof(T), U = (DRAFT ? 8 : 16) / E;  // elements of an access; accesses of a row under way
    const T *p, *r;  // (r without DRAFT: none)
    int64_t vocab;
    int off;         // elements from the boundary to the row's start
    bool same;       // r starts as far from a boundary as p

    __device__ __forceinline__ VerifyRow(const VerifyCall &c, int64_t row)
    {
        p = static_cast<const T *>(c.target) + row * c.target_stride;
        r = DRAFT ? static_cast<const T *>(c.draft) + row * c.draft_stride : nullptr;
        vocab = c.vocab;
        off = (int)((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
        same = DRAFT && off == (int)((reinterpret_cast<uintptr_t>(r) & 15u) / sizeof(T));
    }
    // tiles of a piece: a multiple of U of them, vfPieces pieces a warp and vfRuns warps at most
    __device__ __forceinline__ int piece() const
    {
        const uint32_t tiles = (uint32_t)(vocab + off + 32 * E - 1) / (32 * E), run = (tiles + vfRuns - 1) / vfRuns;
        return (int)((run + vfPieces * U - 1) / (vfPieces * U)) * U;
    }
    // the element of a tile that the lane's first one is (may lie before or behind the row)
    __device__ __forceinline__ int64_t first(int64_t tile, int lane) const { return (tile * 32 + lane) * E - off; }

    static __device__ __forceinline__ void load(const T *row, int64_t v, int64_t vocab, bool whole, float (&x)[E])
    {
        if (whole && v >= 0 && v + E <= vocab) {
            const uint4 u = *reinterpret_cast<const uint4 *>(row + v);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < E; ++i) {
                if constexpr (E == 4) x[i] = __uint_as_float(w[i]);
                else x[i] = i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const bool in = v + i >= 0 && v + i < vocab;
                if constexpr (E == 4) x[i] = in ? row[v + i] : 0.0f;
                else x[i] = in ? __uint_as_float((uint32_t)row[v + i] << 16) : 0.0f;
            }
        }
    }
    // what is left of the lane's elements from v on
    __device__ __forceinline__ void left(const float (&x)[E], const float (&y)[E], float c1, float c2, TwoFloat (&z)[E]) const
    {
#pragma unroll
        for (int i = 0; i < E; ++i)
            z[i] = DRAFT ? vf_left(vf_clean(x[i]), vf_clean(y[i]), c1, c2) : TwoFloat{vf_clean(x[i]), 0.0f};
    }
};

// Pieces of a row, in order: tiles of a piece, pieces in all and of a warp.
struct VerifyPieces {
    int tiles, all, each;
    template <typename T, bool DRAFT>
    __device__ __forceinline__ explicit VerifyPieces(const VerifyRow<T, DRAFT> &a)
    {
        constexpr int E = VerifyRow<T, DRAFT>::E;
        const uint32_t n = (uint32_t)(a.vocab + a.off + 32 * E - 1) / (32 * E);
        tiles = a.piece();
        all = (int)((n + tiles - 1) / tiles);
        each = (all + vfRuns - 1) / vfRuns;
    }
};

// Elements of crossed-out tokens (a list of `gone` at address `list` of the first CTA; its first 32 in `mine`) become
// 0 where they are among the lane's, from v[u] on.
template <int U, int E>
__device__ __forceinline__ void cross_out(float (&x)[U][E], const int64_t (&v)[U], int64_t lo, int64_t hi, int mine, uint32_t list, int gone,
                                          int lane)
{
    for (int i0 = 0; i0 < gone; i0 += 32) {
        const int g = i0 == 0 ? mine : i0 + lane < gone ? cluster_load(list + 4 * (i0 + lane)) : -1;
        for (uint32_t hit = __ballot_sync(0xffffffffu, g >= lo && g < hi); hit; hit &= hit - 1) {
            const int t = __shfl_sync(0xffffffffu, g, __ffs(hit) - 1);
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < E; ++i)
                    if (v[u] + i == t) x[u][i] = 0.0f;
        }
    }
}

// What is left in the pieces of warp `w`, a sum each, to the first CTA's `part`.
template <typename T, bool DRAFT>
__device__ __forceinline__ void verify_sums(const VerifyRow<T, DRAFT> &a, int w, double C, uint32_t list, int gone, uint32_t part, int lane)
{
    constexpr int E = VerifyRow<T, DRAFT>::E, U = VerifyRow<T, DRAFT>::U;
    const VerifyPieces pc(a);
    const float c1 = (float)C, c2 = (float)(C - (double)c1);
    const int mine = lane < gone ? cluster_load(list + 4 * lane) : -1;
    for (int q = w * pc.each; q < (w + 1) * pc.each && q < pc.all; ++q) {
        TwoSum sum;
#pragma unroll 1
        for (int t = 0; t < pc.tiles; t += U) {
            const int64_t t0 = (int64_t)q * pc.tiles + t;
            float x[U][E], y[U][E];
            int64_t v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                v[u] = a.first(t0 + u, lane);
                VerifyRow<T, DRAFT>::load(a.p, v[u], a.vocab, true, x[u]);
                if constexpr (DRAFT) VerifyRow<T, DRAFT>::load(a.r, v[u], a.vocab, a.same, y[u]);
            }
            if (!DRAFT && gone) cross_out(x, v, a.first(t0, 0), a.first(t0 + U, 0), mine, list, gone, lane);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                TwoFloat z[E];
                a.left(x[u], y[u], c1, c2, z);
#pragma unroll
                for (int i = 0; i < E; ++i) sum.add(z[i].hi, z[i].lo);
            }
        }
        sum = warp_total(sum);
        if (lane == 0) cluster_store(part + 8 * q, make_float2(sum.s, sum.e));
    }
}

// The first element of piece q whose running sum, from `before` on, passes `goal`; the
// piece's last one that is left where roundings leave none (-1: none is left).
template <typename T, bool DRAFT>
__device__ __forceinline__ int64_t verify_find(const VerifyRow<T, DRAFT> &a, int q, double C, uint32_t list, int gone, double before, double goal,
                                               int lane)
{
    constexpr int E = VerifyRow<T, DRAFT>::E, U = VerifyRow<T, DRAFT>::U;
    const VerifyPieces pc(a);
    const float c1 = (float)C, c2 = (float)(C - (double)c1);
    const int mine = lane < gone ? cluster_load(list + 4 * lane) : -1;
    int64_t found = -1;
#pragma unroll 1
    for (int t = 0; t < pc.tiles; t += U) {
        const int64_t t0 = (int64_t)q * pc.tiles + t;
        float x[U][E], y[U][E];
        int64_t v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            v[u] = a.first(t0 + u, lane);
            VerifyRow<T, DRAFT>::load(a.p, v[u], a.vocab, true, x[u]);
            if constexpr (DRAFT) VerifyRow<T, DRAFT>::load(a.r, v[u], a.vocab, a.same, y[u]);
        }
        if (!DRAFT && gone) cross_out(x, v, a.first(t0, 0), a.first(t0 + U, 0), mine, list, gone, lane);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            TwoFloat z[E];
            a.left(x[u], y[u], c1, c2, z);
            TwoSum own;
            int last = -1;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                own.add(z[i].hi, z[i].lo);
                if (z[i].hi > 0.0f) last = i;
            }
            const TwoSum upto = warp_running(own, lane);
            const uint32_t over = __ballot_sync(0xffffffffu, last >= 0 && before + upto.value() > goal);
            if (over) {
                // in the first such lane, element after element
                double at = before + (upto.value() - own.value());
                int pick = -1;
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    at += (double)z[i].hi + (double)z[i].lo;
                    if (pick < 0 && z[i].hi > 0.0f && (at > goal || i == last)) pick = i;
                }
                return __shfl_sync(0xffffffffu, v[u] + pick, __ffs(over) - 1);
            }
            const uint32_t some = __ballot_sync(0xffffffffu, last >= 0);
            if (some) found = __shfl_sync(0xffffffffu, v[u] + last, 31 - __clz(some));
            before += __shfl_sync(0xffffffffu, upto.value(), 31);
        }
    }
    return found;
}

template <typename T, bool DRAFT>
__global__ void __launch_bounds__(vfThreads, 4) verify_kernel(const __grid_constant__ VerifyParams p)
{
    extern __shared__ int tree[];  // first CTA: parents, tokens, crossed-out tokens, numbers, p and r of each node's token
    __shared__ VerifyOrder order;
    __shared__ float2 part[vfRuns * vfPieces];  // first CTA: sums of the sequence's pieces
    pdl_wait_primary();
    pdl_allow_dependents();
    const VerifyCall &c = p.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank();
    const int s = blockIdx.x / vfCluster, M = (int)c.max_new;
    const uint32_t order_at = cluster_addr(&order, 0), part_at = cluster_addr(part, 0), gone_at = cluster_addr(tree + 2 * M, 0);
    auto pass = [&](int64_t row, double C, int gone) {
        verify_sums<T, DRAFT>(VerifyRow<T, DRAFT>(c, row), rank * vfWarps + warp, C, gone_at, gone, part_at, lane);
    };
    int *parent = tree, *token = tree + M, *gone = tree + 2 * M;
    float *num = reinterpret_cast<float *>(tree + 3 * M), *pp = num + M, *rr = pp + M;
    int64_t s0 = 0;
    int n = 0;
    if (rank == 0) {
        s0 = c.starts[s];
        const int64_t s1 = c.starts[s + 1];
        n = (int)(s1 - s0);
        if (s0 < 0 || s1 < s0 || s1 > c.total || s1 - s0 > c.max_new) {
            if (tid == 0) atomicOr(c.err, kErrLength);
            n = 0;
        }
        for (int j = tid; j < n; j += vfThreads) {
            int up = c.parents[s0 + j];
            const int x = c.tokens[s0 + j];
            const float u = c.uniforms[s0 + j];
            if (up < -1 || up >= j || (j > 0 && (x < 0 || x >= c.vocab))) {
                atomicOr(c.err, kErrTree);
                up = -1;  // of no node: never reached
            }
            parent[j] = j > 0 ? up : -1;
            token[j] = x;
            num[j] = u;
            if (j > 0 && up >= 0) {
                pp[j] = vf_at(static_cast<const T *>(c.target) + (s0 + up) * c.target_stride, x);
                rr[j] = DRAFT ? vf_at(static_cast<const T *>(c.draft) + (s0 + up) * c.draft_stride, x) : 1.0f;
            }
        }
        for (int k = tid; k < M; k += vfThreads) c.path[s * c.path_stride + k] = -1;
        __syncthreads();
    }
    if (rank != 0 || warp != 0) {
        // told what to sum, until there is nothing more
        for (;;) {
            cluster_sync();  // the order is there
            const int64_t row = cluster_load64(order_at);
            if (row < 0) break;
            pass(row, __longlong_as_double(cluster_load64(order_at + 8)), cluster_load(order_at + 16));
            cluster_sync();  // the sums are there
        }
        cluster_sync();  // (the first CTA's memory is read no more)
        return;
    }

    // The deciding warp; every lane walks the tree, to the same end.
    int32_t *path = c.path + s * c.path_stride;
    int cur = 0, kept = n > 0 ? 1 : 0, crossed = 0;
    double C = 0.0, mass = 1.0;
    bool summed = false;  // the parts are those of cur and C
    double mine = 0.0, upto = 0.0;  // sums of the lane's parts, and of those up to it
    int parts = 0, each = 0;        // pieces, and of a lane
    auto total = [&](int64_t row) {
        if (lane == 0) order = VerifyOrder{row, C, crossed};
        cluster_sync();
        pass(row, C, crossed);
        cluster_sync();
        parts = VerifyPieces(VerifyRow<T, DRAFT>(c, row)).all;
        each = (parts + 31) / 32;
        TwoSum x;
        for (int i = lane * each; i < (lane + 1) * each && i < parts; ++i) x.add(part[i].x, part[i].y);
        mine = x.value();
        upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        return __shfl_sync(0xffffffffu, upto, 31);
    };
    double sum = 0.0;
    if (n > 0 && lane == 0) path[0] = 0;
    auto accept = [&](int j) {
        if (lane == 0) path[kept] = j;
        ++kept;
        cur = j;
        C = 0.0;
        mass = 1.0;
        crossed = 0;
        summed = false;
    };
    for (int j0 = 0; j0 < n; j0 += 32) {
        const int at = j0 + lane, up = at < n ? parent[at] : -1;  // (no node's children: -1)
        uint32_t later = 0xffffffffu;                             // nodes behind the last one tried
        if constexpr (DRAFT) {
            for (;;) {
                const uint32_t kids = __ballot_sync(0xffffffffu, up == cur) & later;
                if (kids == 0) break;
                const int j = j0 + __ffs(kids) - 1;
                later = 0xfffffffeu << (j - j0);
                const double u = num[j], rj = rr[j], here = (double)pp[j] - C * rj;
                if (u * rj * mass < (here > 0.0 ? here : 0.0)) {
                    accept(j);
                } else {
                    C += mass;
                    sum = mass = total(s0 + cur);
                    summed = true;
                }
            }
        } else {
            // Only tokens with a probability that no earlier child had can be accepted or crossed out: each lane
            // finds out for its own node, and what is left of the walk is a product and a difference a child.
            const int x = up >= 0 ? token[at] : -1;
            const double u = up >= 0 ? num[at] : 0.0f, here = up >= 0 ? pp[at] : 0.0f;
            bool again = (__match_any_sync(0xffffffffu, up) & __match_any_sync(0xffffffffu, x) & ((1u << lane) - 1)) != 0;
            for (int i = 0; i < crossed; ++i) again |= up == cur && gone[i] == x;
            __syncwarp();  // (from here on gone is written)
            for (;;) {
                uint32_t kids = __ballot_sync(0xffffffffu, up == cur && here > 0.0 && !again) & later;
                int j = -1;
                for (; kids; kids &= kids - 1) {
                    const int l = __ffs(kids) - 1;
                    const double p = __shfl_sync(0xffffffffu, here, l);
                    if (__shfl_sync(0xffffffffu, u, l) * mass < p) {
                        j = l;
                        break;
                    }
                    mass -= p;
                    if (lane == l) gone[crossed] = x;
                    ++crossed;
                }
                if (j < 0) break;
                accept(j0 + j);
                later = 0xfffffffeu << j;
                __syncwarp();  // (what was crossed out before is written over by other lanes)
            }
            __syncwarp();  // (the next nodes' lanes read what is crossed out)
        }
    }
    int64_t next = -1;
    if (n > 0) {
        if (!summed) sum = total(s0 + cur);
        next = c.vocab;
        if (sum > 0.0) {
            const double goal = (double)c.last[s] * sum;
            // the first lane whose running sum passes the goal, else the last one that has something; then its part
            const uint32_t over = __ballot_sync(0xffffffffu, mine > 0.0 && upto > goal), some = __ballot_sync(0xffffffffu, mine > 0.0);
            const int l = over ? __ffs(over) - 1 : 31 - __clz(some);
            double before = __shfl_sync(0xffffffffu, upto - mine, l), at = before;
            int q = -1;
            for (int i = l * each; i < (l + 1) * each && i < parts; ++i) {
                const double x = (double)part[i].x + (double)part[i].y;
                if (x > 0.0) {
                    q = i;
                    before = at;
                    if (at + x > goal) break;
                }
                at += x;
            }
            if (q >= 0) {
                const int64_t v = verify_find<T, DRAFT>(VerifyRow<T, DRAFT>(c, s0 + cur), q, C, gone_at, crossed, before, goal, lane);
                next = v >= 0 ? v : next;
            }
        }
    }
    if (lane == 0) {
        c.kept[s] = kept;
        c.next[s] = (int)next;
        order.row = -1;
    }
    cluster_sync();
    cluster_sync();
}

}  // namespace

cudaError_t launch_verify(const VerifyCall &v, cudaStream_t s)
{
    VerifyParams p{v};
    const size_t smem = (size_t)v.max_new * 6 * 4;
    const dim3 grid((unsigned)v.seqs * vfCluster);
    const auto kern = v.draft ? (v.f32 ? verify_kernel<float, true> : verify_kernel<uint16_t, true>)
                              : (v.f32 ? verify_kernel<float, false> : verify_kernel<uint16_t, false>);
    return launch_dependent_clusters(kern, grid, vfCluster, dim3(vfThreads), smem, s, p);
}

}  // namespace tq
