// tq_page_table.cu -- page tables kept on the device: the pages of sequences
// whose lengths change, out of and back to a stack of free ones, and the places
// (position, slot, mask of ancestors) of a step's new tokens.
//
// update   with c(n) = ceil(n / P) pages for n rows, a sequence of old length a
//   and wanted length b gives back table entries c(b) .. c(a) - 1, or lacks
//   entries c(a) .. c(b) - 1.  Two exclusive sums over the sequences say where on
//   the stack each of them pushes and pops, a third where its new tokens start;
//   all pushes come before the first pop, so a page may go from one sequence to
//   another in one call.  A few words a sequence: bound by the latency of its
//   loads and barriers, one CTA, so that nothing but barriers orders the two.
// layout   a thread per token: its sequence by bisection of the starts, its row
//   from the lengths; of a tree's node the way to the root by its parents, whose
//   indices fall, so that a mask is written word by word from its last one and
//   never held whole.
#include "tq_common.cuh"
#include "tq_kernels.h"
#include "tq_paged.cuh"

namespace tq {
namespace {

constexpr int ptThreads = 1024;

// pages of n rows (n below 2^31, as the division wants its dividend)
__device__ __forceinline__ int pt_pages(int n, FastDiv div) { return n > 0 ? (int)fast_div((uint32_t)n - 1u, div) + 1 : 0; }

// Sums of three numbers over the block; x becomes the exclusive sums, t the totals.
__device__ __forceinline__ void pt_block_sums(int64_t (&x)[3], int64_t (&t)[3], int64_t (*sh)[32])
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t in[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) in[k] = warp_inclusive_sum(x[k], lane);
    __syncthreads();  // the previous call's readers are done with sh
    if (lane == 31)
#pragma unroll
        for (int k = 0; k < 3; ++k) sh[k][warp] = in[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        const int64_t w = sh[k][lane], ws = warp_inclusive_sum(w, lane);
        t[k] = __shfl_sync(0xffffffffu, ws, 31);
        x[k] = __shfl_sync(0xffffffffu, ws - w, warp) + in[k] - x[k];
    }
}

__global__ void __launch_bounds__(ptThreads) page_table_update_kernel(const __grid_constant__ PagedUpdate u)
{
    __shared__ int64_t sh[3][32];
    pdl_wait_primary();
    pdl_allow_dependents();
    const int tid = threadIdx.x, lane = tid & 31, S = u.seqs;
    const int64_t count = *u.free_count;
    // a sequence's old and wanted length and new tokens; 0 for what is out of range
    auto read = [&](int s, int &a, int &b, int &m) {
        a = s < S ? u.lens[s] : 0;
        b = s < S ? u.want[s] : 0;
        m = s < S && u.fresh ? u.fresh[s] : 0;
        return a >= 0 && a <= u.max_len && b >= 0 && b <= u.max_len && m >= 0 && m <= b;
    };
    int64_t all[3] = {0, 0, 0};  // pushes, pops, new tokens
    bool good = true;
    for (int s0 = 0; s0 < S; s0 += ptThreads) {
        int a, b, m;
        int64_t x[3] = {0, 0, 0}, t[3];
        if (read(s0 + tid, a, b, m)) {
            const int ca = pt_pages(a, u.div_page), cb = pt_pages(b, u.div_page);
            x[0] = ca > cb ? ca - cb : 0;
            x[1] = cb > ca ? cb - ca : 0;
            x[2] = m;
        } else {
            good = false;
        }
        pt_block_sums(x, t, sh);
#pragma unroll
        for (int k = 0; k < 3; ++k) all[k] += t[k];
    }
    good = __syncthreads_and(good) && all[2] <= INT32_MAX;
    const bool room = count >= 0 && count + all[0] <= u.free_cap && all[1] <= count + all[0];
    if (!good || !room) {  // nothing changes, and no token is new
        for (int s = tid; s < S; s += ptThreads) u.lens_out[s] = u.lens[s];
        if (u.starts)
            for (int s = tid; s <= S; s += ptThreads) u.starts[s] = 0;
        if (tid == 0) {
            *u.count_out = (int)count;
            atomicOr(u.err, (good ? 0u : kErrLength) | (room ? 0u : kErrFull));
        }
        return;
    }
    // twice over the sequences: pushes, starts and lengths, then pops
    const int top = (int)(count + all[0]);  // of the stack between the two
    for (int pass = 0; pass < 2; ++pass) {
        if (pass == 1 && all[1] == 0) break;
        int64_t at[3] = {0, 0, 0};
        for (int s0 = 0; s0 < S; s0 += ptThreads) {
            const int s = s0 + tid;
            int a, b, m;
            read(s, a, b, m);
            const int ca = pt_pages(a, u.div_page), cb = pt_pages(b, u.div_page);
            int64_t x[3] = {ca > cb ? ca - cb : 0, cb > ca ? cb - ca : 0, m}, t[3];
            const int64_t mine = x[pass];
            pt_block_sums(x, t, sh);
            if (pass == 0 && s < S && u.starts) u.starts[s] = (int)(at[2] + x[2]);
            // entries from `from` on, stack places from `place` on (pops: downwards)
            const int from = ca < cb ? ca : cb, place = (int)(pass == 0 ? count + at[0] + x[0] : top - 1 - (at[1] + x[1]));
            auto move = [&](int s1, int entry, int slot) {
                int32_t *e = u.pages + s1 * u.stride + entry;
                if (pass == 0) {
                    const int page = *e;
                    if ((uint32_t)page >= (uint32_t)u.num_pages) atomicOr(u.err, kErrPage);
                    u.free_pages[slot] = page;
                } else {
                    *e = u.free_pages[slot];
                }
            };
            // the first entry by the sequence's own thread, the others of a sequence by its warp
            if (mine > 0) move(s, from, place);
            for (uint32_t more = __ballot_sync(0xffffffffu, mine > 1); more; more &= more - 1) {
                const int l = __ffs(more) - 1;
                const int n = (int)__shfl_sync(0xffffffffu, mine, l), f = __shfl_sync(0xffffffffu, from, l),
                          q = __shfl_sync(0xffffffffu, place, l);
                for (int i = 1 + lane; i < n; i += 32) move(s - lane + l, f + i, pass == 0 ? q + i : q - i);
            }
#pragma unroll
            for (int k = 0; k < 3; ++k) at[k] += t[k];
        }
        __syncthreads();  // every push is done before the first pop
    }
    __syncthreads();  // every reader of the lengths and the count is done: either may be written in place
    for (int s = tid; s < S; s += ptThreads) u.lens_out[s] = u.want[s];
    if (tid == 0) {
        if (u.starts) u.starts[S] = (int)all[2];
        *u.count_out = top - (int)all[1];
    }
}

// ---------------------------------------------------------------- places of the new tokens
struct LayoutParams {
    PagedView v;
    const int32_t *parents;  // null: the tokens of a sequence follow one another
    int64_t max_new;
    int32_t *positions;
    int64_t *slots;
    uint32_t *masks;
    int64_t mask_words;
};

__global__ void __launch_bounds__(128) paged_layout_kernel(const __grid_constant__ LayoutParams p)
{
    pdl_wait_primary();
    pdl_allow_dependents();
    const int64_t t = (int64_t)blockIdx.x * 128 + threadIdx.x;
    if (t >= p.v.total) return;
    int lo = 0, hi = p.v.seqs + 1;  // the last sequence that starts at or before t
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (p.v.starts[mid] <= t) lo = mid + 1;
        else hi = mid;
    }
    const int s = lo - 1;
    bool live = s >= 0 && s < p.v.seqs;
    int64_t row = -1;
    int n = 0, node = 0, len = 0;
    if (live) {
        const int64_t s0 = p.v.starts[s], s1 = p.v.starts[s + 1];
        len = p.v.lens[s];
        live = s0 >= 0 && s1 <= p.v.total && s1 >= s0 && len >= 0 && len <= p.v.max_len && (!p.parents || s1 - s0 <= p.max_new);
        if (!live) atomicOr(p.v.err, kErrLength);
        live = live && t < s1;
        n = (int)(s1 - s0);
        node = (int)(t - s0);
        row = (int64_t)len - n + node;
    }
    int64_t slot = -1;
    if (live && row >= 0) {
        uint32_t in;
        const int page = paged_page(p.v, s, (uint32_t)row, in);
        if (page >= 0) slot = (int64_t)page * p.v.page + in;
    }
    if (p.slots) p.slots[t] = slot;
    int64_t pos = row;
    if (p.parents) {
        uint32_t *mask = p.masks ? p.masks + t * p.mask_words : nullptr;
        int64_t w = p.mask_words - 1;  // words above are written
        uint32_t bits = 0;
        int depth = -1;
        for (int j = live ? node : -1; j >= 0;) {
            ++depth;
            if (mask) {
                for (; w > j >> 5; --w) {
                    mask[w] = bits;
                    bits = 0;
                }
                bits |= 1u << (j & 31);
            }
            const int up = p.parents[t - node + j];
            if (up < -1 || up >= j) {
                atomicOr(p.v.err, kErrTree);
                break;
            }
            j = up;
        }
        if (mask)
            for (; w >= 0; --w) {
                mask[w] = bits;
                bits = 0;
            }
        pos = (int64_t)len - n + depth;
    }
    if (p.positions) p.positions[t] = live && pos >= 0 ? (int)pos : -1;
}

}  // namespace

cudaError_t launch_page_table_update(const PagedUpdate &u, cudaStream_t s)
{
    return launch_dependent(page_table_update_kernel, dim3(1), dim3(ptThreads), 0, s, u);
}

cudaError_t launch_paged_layout(const PagedView &v, const int32_t *parents, int64_t max_new, int32_t *positions, int64_t *slots,
                                uint32_t *masks, int64_t mask_words, cudaStream_t s)
{
    return launch_dependent(paged_layout_kernel, dim3((unsigned)((v.total + 127) / 128)), dim3(128), 0, s,
                            LayoutParams{v, parents, max_new, positions, slots, masks, mask_words});
}

}  // namespace tq
