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
// The sums decide which token comes out, so they are kept to 2^-45 or so: a
// thread adds in pairs of floats (sum and what its roundings left out, the
// product C r(v) in two parts), whole threads' sums are added in 64 bits.  (64-bit
// additions for every element would take this chip 64 times as long as 32-bit ones.)
//
// A cluster of CTAs goes through a row, a run of elements per warp.  The first CTA
// alone reads the tree and decides; the others are told what to sum, so that
// no two of them can disagree on how often they meet.  A pass moves the row once:
// bound by memory for many sequences, by the latency of loads and cluster
// barriers for few.
#include "tq_common.cuh"
#include "tq_kernels.h"
#include "tq_paged.cuh"

namespace tq {
namespace {

constexpr int vfThreads = 256, vfWarps = vfThreads / 32;
constexpr int vfCluster = 8, vfParts = vfWarps * vfCluster;  // warps to a sequence

struct VerifyParams {
    VerifyCall c;
    int parts;      // warps to a sequence: vfWarps * CTAs of a cluster
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

__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
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

__device__ __forceinline__ void cluster_store64(uint32_t a, double v)
{
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(a), "d"(v) : "memory");
}

// A probability as it counts: neither negative, NaN nor infinite.
__device__ __forceinline__ float vf_clean(float x) { return x > 0.0f && x < INFINITY ? x : 0.0f; }

__device__ __forceinline__ float vf_at(const float *row, int64_t v) { return vf_clean(row[v]); }
__device__ __forceinline__ float vf_at(const uint16_t *row, int64_t v) { return vf_clean(__uint_as_float((uint32_t)row[v] << 16)); }

// A running sum in two floats: s + e.
struct TwoSum {
    float s = 0.0f, e = 0.0f;
    __device__ __forceinline__ void add(float x)
    {
        const float t = __fadd_rn(s, x), z = __fsub_rn(t, s);
        e = __fadd_rn(e, __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(x, z)));
        s = t;
    }
};

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
template <typename T>
struct VerifyRow {
    static constexpr int E = 16 / sizeof(T);
    const T *p, *r;  // r null: none
    int64_t vocab;
    int off;         // elements from the boundary to the row's start
    bool same;       // r starts as far from a boundary as p

    __device__ __forceinline__ VerifyRow(const VerifyCall &c, int64_t row)
    {
        p = static_cast<const T *>(c.target) + row * c.target_stride;
        r = c.draft ? static_cast<const T *>(c.draft) + row * c.draft_stride : nullptr;
        vocab = c.vocab;
        off = (int)((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
        same = r && off == (int)((reinterpret_cast<uintptr_t>(r) & 15u) / sizeof(T));
    }
    // tiles of a warp's run, and the run of warp w
    __device__ __forceinline__ int64_t run(int parts) const
    {
        const int64_t tiles = (vocab + off + 32 * E - 1) / (32 * E);
        return (tiles + parts - 1) / parts;
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
            z[i] = r ? vf_left(vf_clean(x[i]), vf_clean(y[i]), c1, c2) : TwoFloat{vf_clean(x[i]), 0.0f};
    }
};

// Sum of what is left over the run of warp `w`.  `gone`: addresses of the first CTA's list of crossed-out tokens.
template <typename T>
__device__ __forceinline__ double verify_sum(const VerifyRow<T> &a, int64_t run, int w, double C, uint32_t list, int gone, int lane)
{
    constexpr int E = VerifyRow<T>::E, U = 4;
    const int64_t t0 = w * run, v_lo = a.first(t0, 0), v_hi = a.first(t0 + run, 0);
    const float c1 = (float)C, c2 = (float)(C - (double)c1);
    TwoSum sum;
    if (v_lo < a.vocab) {
        for (int64_t t = t0; t < t0 + run; t += U) {
            float x[U][E], y[U][E];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t v = t + u < t0 + run ? a.first(t + u, lane) : a.vocab;
                VerifyRow<T>::load(a.p, v, a.vocab, true, x[u]);
                if (a.r) VerifyRow<T>::load(a.r, v, a.vocab, a.same, y[u]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                TwoFloat z[E];
                a.left(x[u], y[u], c1, c2, z);
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    sum.add(z[i].hi);
                    sum.e += z[i].lo;
                }
            }
        }
        // (crossed-out tokens of the run: taken out of the sum of the lane that the list's place falls to)
        for (int i = lane; i < gone; i += 32) {
            const int x = cluster_load(list + 4 * i);
            if (x >= v_lo && x < v_hi) sum.add(-vf_at(a.p, x));
        }
    }
    double d = (double)sum.s + (double)sum.e;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    return d > 0.0 ? d : 0.0;
}

// The first element of warp w's run whose running sum, from `before` on, passes
// `goal`; the run's last one that is left where roundings leave none.  Whole warps call.
template <typename T>
__device__ __forceinline__ int64_t verify_find(const VerifyRow<T> &a, int64_t run, int w, double C, const int *list, int gone,
                                               double before, double goal, int lane)
{
    constexpr int E = VerifyRow<T>::E;
    const float c1 = (float)C, c2 = (float)(C - (double)c1);
    int64_t found = -1;
    for (int64_t t = w * run; t < (w + 1) * run; ++t) {
        const int64_t v = a.first(t, lane);
        float x[E], y[E];
        VerifyRow<T>::load(a.p, v, a.vocab, true, x);
        if (a.r) VerifyRow<T>::load(a.r, v, a.vocab, a.same, y);
        TwoFloat z[E];
        a.left(x, y, c1, c2, z);
        for (int i = 0; i < gone; ++i) {
            const int64_t k = list[i] - v;
#pragma unroll
            for (int j = 0; j < E; ++j)
                if (k == j) z[j] = TwoFloat{0.0f, 0.0f};
        }
        double own = 0.0;
        int last = -1;
#pragma unroll
        for (int j = 0; j < E; ++j) {
            own += (double)z[j].hi + (double)z[j].lo;
            if (z[j].hi > 0.0f) last = j;
        }
        double in = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double y2 = __shfl_up_sync(0xffffffffu, in, o);
            if (lane >= o) in += y2;
        }
        const uint32_t over = __ballot_sync(0xffffffffu, last >= 0 && before + in > goal);
        if (over) {
            const int l = __ffs(over) - 1;
            double acc = before + (in - own);
            int pick = last;
#pragma unroll
            for (int j = E - 1; j >= 0; --j) {  // the first that passes: from behind
                double upto = acc;
#pragma unroll
                for (int k = 0; k <= j; ++k) upto += (double)z[k].hi + (double)z[k].lo;
                if (z[j].hi > 0.0f && upto > goal) pick = j;
            }
            return __shfl_sync(0xffffffffu, v + pick, l);
        }
        const uint32_t some = __ballot_sync(0xffffffffu, last >= 0);
        if (some) found = __shfl_sync(0xffffffffu, v + last, 31 - __clz(some));
        before += __shfl_sync(0xffffffffu, in, 31);
    }
    return found;
}

template <typename T>
__global__ void __launch_bounds__(vfThreads) verify_kernel(const __grid_constant__ VerifyParams p)
{
    extern __shared__ int tree[];  // first CTA: parents, tokens, crossed-out tokens, numbers, p and r of each node's token
    __shared__ VerifyOrder order;
    __shared__ double part[vfParts];  // first CTA: sums of the sequence's warps
    pdl_wait_primary();
    pdl_allow_dependents();
    const VerifyCall &c = p.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank(), ctas = cluster_size();
    const int s = blockIdx.x / ctas, M = (int)c.max_new;
    const uint32_t order_at = cluster_addr(&order, 0), part_at = cluster_addr(part, 0), gone_at = cluster_addr(tree + 2 * M, 0);

    // one sum over the cluster, of every CTA: order, run, sums to the first CTA
    auto pass = [&](int64_t row, double C, int gone) {
        const VerifyRow<T> a(c, row);
        const int w = rank * vfWarps + warp;
        const double d = verify_sum<T>(a, a.run(p.parts), w, C, gone_at, gone, lane);
        if (lane == 0) cluster_store64(part_at + 8 * w, d);
    };
    if (rank != 0) {
        for (;;) {
            cluster_sync();  // the order is there
            const int64_t row = cluster_load64(order_at);
            if (row < 0) break;
            const double C = __longlong_as_double(cluster_load64(order_at + 8));
            const int gone = cluster_load(order_at + 16);
            pass(row, C, gone);
            cluster_sync();  // the sums are there
        }
        cluster_sync();  // (the first CTA's memory is read no more)
        return;
    }

    const int64_t s0 = c.starts[s], s1 = c.starts[s + 1];
    int n = (int)(s1 - s0);
    if (s0 < 0 || s1 < s0 || s1 > c.total || s1 - s0 > c.max_new) {
        if (tid == 0) atomicOr(c.err, kErrLength);
        n = 0;
    }
    int *parent = tree, *token = tree + M, *gone = tree + 2 * M;
    float *num = reinterpret_cast<float *>(tree + 3 * M), *pp = num + M, *rr = pp + M;
    for (int j = tid; j < n; j += vfThreads) {
        int up = c.parents[s0 + j];
        const int x = c.tokens[s0 + j];
        if (up < -1 || up >= j || (j > 0 && (x < 0 || x >= c.vocab))) {
            atomicOr(c.err, kErrTree);
            up = -1;  // of no node: never reached
        }
        parent[j] = j > 0 ? up : -1;
        token[j] = x;
        num[j] = c.uniforms[s0 + j];
        if (j > 0 && up >= 0) {
            pp[j] = vf_at(static_cast<const T *>(c.target) + (s0 + up) * c.target_stride, x);
            rr[j] = c.draft ? vf_at(static_cast<const T *>(c.draft) + (s0 + up) * c.draft_stride, x) : 1.0f;
        }
    }
    int32_t *path = c.path + s * c.path_stride;
    for (int k = tid; k < M; k += vfThreads) path[k] = -1;
    __syncthreads();

    // every thread of the CTA walks the tree, to the same end
    auto total = [&](int64_t row, double C, int crossed) {
        if (tid == 0) order = VerifyOrder{row, C, crossed};
        cluster_sync();
        pass(row, C, crossed);
        cluster_sync();
        double sum = 0.0;
        for (int i = 0; i < p.parts; ++i) sum += part[i];
        return sum;
    };
    int cur = 0, kept = n > 0 ? 1 : 0, crossed = 0;
    double C = 0.0, mass = 1.0;
    bool summed = false;  // the sums are those of cur and C
    if (n > 0 && tid == 0) path[0] = 0;
    for (int j = 1; j < n; ++j) {
        if (parent[j] != cur) continue;
        const double u = num[j], pj = pp[j], rj = rr[j];
        double here = pj - C * rj;
        if (!c.draft) {
            here = pj;
            for (int i = 0; i < crossed; ++i)
                if (gone[i] == token[j]) here = 0.0;
        }
        here = here > 0.0 ? here : 0.0;
        if (u * rj * mass < here) {
            if (tid == 0) path[kept] = j;
            ++kept;
            cur = j;
            C = 0.0;
            mass = 1.0;
            crossed = 0;
            summed = false;
        } else if (c.draft) {
            C += mass;
            mass = total(s0 + cur, C, 0);
            summed = true;
        } else if (here > 0.0) {
            mass -= here;
            __syncthreads();  // (the list's readers are done)
            if (tid == 0) gone[crossed] = token[j];
            ++crossed;
            __syncthreads();
        }
    }
    int64_t next = -1;
    if (n > 0) {
        double sum = 0.0;
        if (!summed) sum = total(s0 + cur, C, crossed);
        else
            for (int i = 0; i < p.parts; ++i) sum += part[i];
        next = c.vocab;
        if (warp == 0 && sum > 0.0) {
            const double goal = (double)c.last[s] * sum;
            // the first warp whose running sum passes the goal, else the last one that has something
            double before = 0.0, upto = 0.0, from = 0.0;
            int w = -1;
            for (int i = 0; i < p.parts; ++i) {
                before = upto;
                upto += part[i];
                if (part[i] > 0.0) {
                    w = i;
                    from = before;
                    if (upto > goal) break;
                }
            }
            const VerifyRow<T> a(c, s0 + cur);
            const int64_t v = verify_find<T>(a, a.run(p.parts), w, C, gone, crossed, from, goal, lane);
            next = v >= 0 ? v : next;
        }
    }
    if (tid == 0) {
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
    VerifyParams p{v, vfParts};
    const size_t smem = (size_t)v.max_new * 6 * 4;
    const dim3 grid((unsigned)v.seqs * vfCluster);
    return launch_dependent_clusters(v.f32 ? verify_kernel<float> : verify_kernel<uint16_t>, grid, vfCluster, dim3(vfThreads), smem, s, p);
}

}  // namespace tq
