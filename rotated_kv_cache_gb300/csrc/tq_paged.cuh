// tq_paged.cuh -- where the rows of a paged cache are: device-side reading of
// a page table and of the ragged tokens' starts, with every index checked.
//
// The pool is a cache whose batch is the number of pages and whose capacity is
// the page size, so row r of page p of kv-head h is plane row (p H + h) P + r.
// Token t of the ragged tensors belongs to the sequence s with
// starts[s] <= t < starts[s + 1] and stands at position
//   len(s) - (starts[s + 1] - starts[s]) + (t - starts[s])
// of it (new tokens are the last ones).  Lengths, starts and page numbers are
// device data that the host cannot check: a value out of range is recorded in
// the device error word and never used as an address.
#pragma once
#include "tq_common.cuh"
#include "tq_kernels.h"

namespace tq {

constexpr uint32_t kErrPage = 2u;    // a page number outside the pool
constexpr uint32_t kErrLength = 4u;  // a length above max_len, or starts out of order

// Rows of sequence s, in [0, max_len].
__device__ __forceinline__ int64_t paged_len(const PagedView &v, int s)
{
    const int n = v.lens[s];
    if (n < 0 || n > v.max_len) {
        atomicOr(v.err, kErrLength);
        return n < 0 ? 0 : v.max_len;
    }
    return n;
}

// First ragged row of sequence s, in [0, total].
__device__ __forceinline__ int64_t paged_start(const PagedView &v, int s)
{
    const int x = v.starts[s];
    return x < 0 ? 0 : (x > v.total ? v.total : x);
}

// New tokens of sequence s (never negative).
__device__ __forceinline__ int64_t paged_new(const PagedView &v, int s)
{
    const int64_t n = paged_start(v, s + 1) - paged_start(v, s);
    if (n < 0) atomicOr(v.err, kErrLength);
    return n < 0 ? 0 : n;
}

// The page of chunk position pos (0 <= pos < max_len), or -1 when its number is bad.
__device__ __forceinline__ int paged_page(const PagedView &v, int s, uint32_t pos, uint32_t &slot)
{
    const uint32_t i = fast_div(pos, v.div_page);
    slot = pos - i * v.page;
    const int p = v.pages[s * v.stride + i];
    if ((uint32_t)p < (uint32_t)v.num_pages) return p;
    atomicOr(v.err, kErrPage);
    return -1;
}

// Plane row of ragged token t for kv-head 0 (add h * page for kv-head h), or
// -1: t lies behind the last sequence, before its sequence's first row (more
// new tokens than rows), or in a bad page.  The sequence is the last one
// that starts at or before t (empty sequences share a start).
__device__ __forceinline__ int64_t paged_row(const PagedView &v, int64_t t, int H)
{
    if (t >= v.total) return -1;
    int lo = 0, hi = v.seqs + 1;  // starts[lo - 1] <= t < starts[hi]
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (v.starts[mid] <= t) lo = mid + 1;
        else hi = mid;
    }
    const int s = lo - 1;
    if (s < 0 || s >= v.seqs) return -1;
    const int64_t s0 = paged_start(v, s), n = paged_new(v, s), pos = paged_len(v, s) - n + (t - s0);
    if (t >= s0 + n || pos < 0) return -1;
    uint32_t slot;
    const int p = paged_page(v, s, (uint32_t)pos, slot);
    return p < 0 ? -1 : (int64_t)p * H * v.page + slot;
}

// ------------------------------------------------------------------ split attention over a paged batch
// The work of a batch is one line of stages (ST rows each): sequence after
// sequence, in a sequence its units (kv-head, block of CB columns) one after
// another, in a unit its stages in row order.  CTA c takes the c-th run of
// `per` stages, whatever lengths the sequences have, so all CTAs finish
// together; a run's part of one unit is a segment, and a unit's segments are
// merged by the combine.  Segment (c, unit u) writes partial slot c + u:
// along the line c or u grows by one at every new segment, so slots are
// distinct, and at most CTAs + units of them are used.
//
// Every warp works the line out for itself from the lengths (two passes of 32
// sequences at a time); the first CTA leaves the prefix sums for the combine.
// Stages and units of sequence s (none where it has no rows, no new tokens, or too many).
__device__ __forceinline__ void paged_shape(const PagedSplit &ps, int s, int ST, int CB, int H, int G, int64_t &stages,
                                            int64_t &blocks)
{
    stages = blocks = 0;
    if (s >= ps.v.seqs) return;
    const int64_t n = paged_new(ps.v, s), len = paged_len(ps.v, s);
    if (n == 0 || n > ps.wide || len == 0) return;
    stages = (len + ST - 1) / ST;
    blocks = (n * G + CB - 1) / CB;
}

__device__ __forceinline__ int64_t warp_inclusive_sum(int64_t x, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

struct PagedWalk {
    int64_t x, end;        // stages of the line still to do
    int s;                 // sequence of x
    int64_t sp, up;        // stages, units before it
    int64_t stages, blocks;
    // the segment at x
    int64_t s0, n, len;    // first ragged row, new tokens, rows
    int h, hb, first, count;
    int64_t slot;

    // Call from whole warps.  False: nothing for this CTA.
    __device__ __forceinline__ bool start(const PagedSplit &ps, int ST, int CB, int H, int G, int lane)
    {
        int64_t total = 0;
        for (int b = 0; b < ps.v.seqs; b += 32) {
            int64_t st, bl;
            paged_shape(ps, b + lane, ST, CB, H, G, st, bl);
            total += st * bl * H;
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        int64_t per = (total + gridDim.x - 1) / gridDim.x;
        if (per < 1) per = 1;
        x = blockIdx.x * per;
        end = imin64(total, x + per);
        const bool writer = blockIdx.x == 0 && threadIdx.x < 32;
        if (x >= end && !writer) return false;
        int64_t sbase = 0, ubase = 0;
        bool found = false;
        for (int b = 0; b < ps.v.seqs && (writer || !found); b += 32) {
            int64_t st, bl;
            paged_shape(ps, b + lane, ST, CB, H, G, st, bl);
            const int64_t w = st * bl * H, u = bl * H;
            const int64_t ws = warp_inclusive_sum(w, lane), us = warp_inclusive_sum(u, lane);
            const int64_t s_at = sbase + ws - w, u_at = ubase + us - u;
            if (writer && b + lane <= ps.v.seqs) {
                ps.plan[b + lane] = s_at;
                ps.plan[ps.v.seqs + 1 + b + lane] = u_at;
            }
            const uint32_t hit = __ballot_sync(0xffffffffu, w > 0 && s_at <= x && x < s_at + w);
            if (hit) {
                const int l = __ffs(hit) - 1;
                s = b + l;
                sp = __shfl_sync(0xffffffffu, s_at, l);
                up = __shfl_sync(0xffffffffu, u_at, l);
                stages = __shfl_sync(0xffffffffu, st, l);
                blocks = __shfl_sync(0xffffffffu, bl, l);
                found = true;
            }
            sbase += __shfl_sync(0xffffffffu, ws, 31);
            ubase += __shfl_sync(0xffffffffu, us, 31);
        }
        if (writer && lane == 0) {
            ps.plan[ps.v.seqs] = sbase;
            ps.plan[2 * ps.v.seqs + 1] = ubase;
            ps.plan[2 * ps.v.seqs + 2] = per;
        }
        return x < end;
    }

    // The segment at x.
    __device__ __forceinline__ void segment(const PagedSplit &ps)
    {
        const int64_t y = x - sp, u = y / stages;
        first = (int)(y - u * stages);
        count = (int)imin64(stages - first, end - x);
        h = (int)(u / blocks);
        hb = (int)(u - h * blocks);
        slot = blockIdx.x + up + u;
        s0 = paged_start(ps.v, s);
        n = paged_new(ps.v, s);
        len = paged_len(ps.v, s);
    }

    // To the segment after this one.  False: the CTA's run is done.
    __device__ __forceinline__ bool next(const PagedSplit &ps, int ST, int CB, int H, int G)
    {
        x += count;
        if (x >= end) return false;
        while (x >= sp + stages * blocks * H) {  // to the next sequence with work: x < end says that there is one
            sp += stages * blocks * H;
            up += blocks * H;
            ++s;
            paged_shape(ps, s, ST, CB, H, G, stages, blocks);
        }
        return true;
    }
};

// The pages of a segment's chunks (RU = gcd(stage rows, page rows) rows each,
// so that no chunk crosses a page), 32 / NCH stages ahead at a time, one
// chunk a lane: a refill finds its pages in registers.
template <int ST>
struct PagedPages {
    int nch = 1, spl = 32;     // chunks per stage, stages per warp load
    int base = 0;              // first stage of `cur`
    int64_t cur = 0, nxt = 0;  // plane row of the lane's chunk for kv-head 0 (+ h page)

    __device__ __forceinline__ int64_t load(const PagedSplit &ps, const PagedWalk &w, int H, int stage0, int lane) const
    {
        const int st = stage0 + lane / nch, ch = lane - (lane / nch) * nch;
        const int64_t row = (int64_t)st * ST + ch * (ST / nch);
        if (lane >= spl * nch || row >= w.len) return 0;
        uint32_t slot;
        const int pg = paged_page(ps.v, w.s, (uint32_t)row, slot);
        return ((int64_t)(pg < 0 ? 0 : pg) * H + w.h) * ps.v.page + slot;
    }

    __device__ __forceinline__ void start(const PagedSplit &ps, const PagedWalk &w, int H, int stage, int lane)
    {
        nch = ST / gcd_int(ST, (int)ps.v.page);
        spl = 32 / nch;
        base = stage;
        cur = load(ps, w, H, base, lane);
        nxt = load(ps, w, H, base + spl, lane);
    }

    // Plane row of chunk (lane) of `stage`, which is base or later and at most a load ahead.
    __device__ __forceinline__ int64_t rows(const PagedSplit &ps, const PagedWalk &w, int H, int stage, int lane)
    {
        while (stage >= base + spl) {
            base += spl;
            cur = nxt;
            nxt = load(ps, w, H, base + spl, lane);
        }
        return __shfl_sync(0xffffffffu, cur, (stage - base) * nch + (lane < nch ? lane : 0));
    }
};

}  // namespace tq
