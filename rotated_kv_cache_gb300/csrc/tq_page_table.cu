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
//
// 256 sequences with trees of 20 to 64 nodes, 16 of which begin or end with up to 512
// pages: update 5.7 us (12.9 with one sequence's pages after another's by its own
// warp), layout of 10263 tokens 4.2 us (its chains of reads from memory: 5.4).  64
// sequences one token on: 5.1 and 2.1 us, of which a launch is 2.
#include "tq_common.cuh"
#include "tq_kernels.h"
#include "tq_paged.cuh"

namespace tq {
namespace {

constexpr int ptThreads = 1024;
constexpr int ptBatch = 8;  // page numbers of a lane under way

struct PtMove {
    int s, from, place, n;  // n entries of sequence s from `from` on, stack places from `place` on (pops: downwards)
};

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
    __shared__ PtMove list[ptThreads];
    __shared__ int listed;
    pdl_wait_primary();
    pdl_allow_dependents();
    if (threadIdx.x == 0) listed = 0;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, S = u.seqs;
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
    const bool once = S <= ptThreads;  // a thread's sequence stays in its registers
    int a, b, m;
    int64_t x[3], t[3];
    for (int s0 = 0; s0 < S; s0 += ptThreads) {
        x[0] = x[1] = x[2] = 0;
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
            if (!once) read(s, a, b, m);
            const int ca = pt_pages(a, u.div_page), cb = pt_pages(b, u.div_page);
            const int64_t mine = pass == 0 ? (ca > cb ? ca - cb : 0) : (cb > ca ? cb - ca : 0);
            if (!once) {
                x[0] = ca > cb ? ca - cb : 0;
                x[1] = cb > ca ? cb - ca : 0;
                x[2] = m;
                pt_block_sums(x, t, sh);
            }
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
            // the first entry by the sequence's own thread; sequences of more are listed, and go to a warp each
            if (mine > 0) move(s, from, place);
            if (mine > 1) list[atomicAdd(&listed, 1)] = PtMove{s, from, place, (int)mine};
            __syncthreads();
            for (int e = warp; e < listed; e += ptThreads / 32) {
                const PtMove v = list[e];
                int32_t *entry = u.pages + v.s * u.stride + v.from;
                for (int i0 = 1 + lane; i0 < v.n; i0 += 32 * ptBatch) {  // (loads of a batch together)
                    int page[ptBatch];
#pragma unroll
                    for (int k = 0; k < ptBatch; ++k) {
                        const int i = i0 + 32 * k;
                        if (i < v.n) page[k] = pass == 0 ? entry[i] : u.free_pages[v.place - i];
                    }
#pragma unroll
                    for (int k = 0; k < ptBatch; ++k) {
                        const int i = i0 + 32 * k;
                        if (i >= v.n) break;
                        if (pass == 0) {
                            if ((uint32_t)page[k] >= (uint32_t)u.num_pages) atomicOr(u.err, kErrPage);
                            u.free_pages[v.place + i] = page[k];
                        } else {
                            entry[i] = page[k];
                        }
                    }
                }
            }
            __syncthreads();
            if (tid == 0) listed = 0;
#pragma unroll
            for (int k = 0; k < 3; ++k) at[k] += t[k];  // (read where there is another chunk alone)
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

constexpr int plThreads = 128, plStarts = 1024, plParents = 1024;

__global__ void __launch_bounds__(plThreads) paged_layout_kernel(const __grid_constant__ LayoutParams p)
{
    // The starts, and the parents of the block's sequences, where they are few: bisection and the way to a root
    // are chains of dependent reads, of 30 cycles each from here.
    __shared__ int32_t sh_starts[plStarts], sh_parents[plParents];
    pdl_wait_primary();
    pdl_allow_dependents();
    const int64_t t = (int64_t)blockIdx.x * plThreads + threadIdx.x, t_last = imin64(p.v.total, ((int64_t)blockIdx.x + 1) * plThreads) - 1;
    const int32_t *starts = p.v.starts;
    if (p.v.seqs < plStarts) {
        for (int i = threadIdx.x; i <= p.v.seqs; i += plThreads) sh_starts[i] = p.v.starts[i];
        __syncthreads();
        starts = sh_starts;
    }
    if (blockIdx.x == 0)  // (a token alone does not see that starts elsewhere fall)
        for (int i = threadIdx.x; i < p.v.seqs; i += plThreads)
            if (starts[i] > starts[i + 1]) atomicOr(p.v.err, kErrLength);
    auto sequence = [&](int64_t x) {  // the last sequence that starts at or before x, plus one
        int lo = 0, hi = p.v.seqs + 1;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (starts[mid] <= x) lo = mid + 1;
            else hi = mid;
        }
        return lo;
    };
    int64_t held = INT64_MAX;  // tokens from this one on have their parents in shared memory
    if (p.parents) {
        const int s0 = sequence((int64_t)blockIdx.x * plThreads) - 1;
        const int64_t from = s0 >= 0 && starts[s0] >= 0 ? starts[s0] : 0;
        if (t_last - from < plParents) {
            for (int i = threadIdx.x; i <= t_last - from; i += plThreads) sh_parents[i] = p.parents[from + i];
            __syncthreads();
            held = from;
        }
    }
    if (t >= p.v.total) return;
    const int lo = sequence(t);
    const int s = lo - 1;
    bool live = s >= 0 && s < p.v.seqs;
    int64_t row = -1;
    int n = 0, node = 0, len = 0;
    if (live) {
        const int64_t s0 = starts[s], s1 = starts[s + 1];
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
            // (a sequence of starts out of order may lie before those that the block holds)
            const int64_t at = t - node + j;
            const int up = at >= held ? sh_parents[at - held] : p.parents[at];
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
    return launch_dependent(paged_layout_kernel, dim3((unsigned)((v.total + plThreads - 1) / plThreads)), dim3(plThreads), 0, s,
                            LayoutParams{v, parents, max_new, positions, slots, masks, mask_words});
}

}  // namespace tq
