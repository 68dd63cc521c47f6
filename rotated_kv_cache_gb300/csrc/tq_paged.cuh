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

// The starts and lengths of the first 31 sequences, one a lane (starts[lane],
// lens[lane]): with no more sequences than that, a token's sequence is found
// without a load.
struct PagedLanes {
    int start, len;
};

__device__ __forceinline__ PagedLanes paged_lanes(const PagedView &v, int lane)
{
    PagedLanes l;
    l.start = v.starts[lane < v.seqs ? lane : v.seqs];
    l.len = v.lens[lane < v.seqs ? lane : v.seqs - 1];
    return l;
}

// A token's place: its page number as the table gives it (a load that may still
// be under way) and its row in the page, kNoRow where it has none.
constexpr uint32_t kNoRow = 0xFFFFFFFFu;

struct PagedPlace {
    int page;
    uint32_t slot;
};

// Plane row of a place for kv-head 0 (add h * page for kv-head h), or -1.
__device__ __forceinline__ int64_t paged_place_row(const PagedView &v, const PagedPlace &a, int H)
{
    if (a.slot == kNoRow) return -1;
    if ((uint32_t)a.page >= (uint32_t)v.num_pages) {
        atomicOr(v.err, kErrPage);
        return -1;
    }
    return (int64_t)a.page * H * v.page + a.slot;
}

// Place of ragged token t; none: t lies behind the last sequence, before its sequence's first row (more
// new tokens than rows), or in a bad page.  The sequence is the last one
// that starts at or before t (empty sequences share a start).  Whole warps
// call it, each lane with a token of its own.
__device__ __forceinline__ PagedPlace paged_seek(const PagedView &v, const PagedLanes &l, int64_t t)
{
    const PagedPlace none{0, kNoRow};
    int s, len;
    int64_t s0, s1;
    if (v.seqs < 32) {
        int lo = 0;  // sequences that start at or before t, found bit by bit
#pragma unroll
        for (int step = 16; step >= 1; step >>= 1) {
            const int x = __shfl_sync(0xffffffffu, l.start, lo + step - 1);
            if (lo + step - 1 <= v.seqs && x <= t) lo += step;
        }
        s = lo - 1;
        s0 = __shfl_sync(0xffffffffu, l.start, s < 0 ? 0 : s);
        s1 = __shfl_sync(0xffffffffu, l.start, s < 0 ? 0 : s + 1 > 31 ? 31 : s + 1);
        len = __shfl_sync(0xffffffffu, l.len, s < 0 ? 0 : s);
        if (s < 0 || s >= v.seqs) return none;
    } else {
        int lo = 0, hi = v.seqs + 1;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (v.starts[mid] <= t) lo = mid + 1;
            else hi = mid;
        }
        s = lo - 1;
        if (s < 0 || s >= v.seqs) return none;
        s0 = v.starts[s];
        s1 = v.starts[s + 1];
        len = v.lens[s];
    }
    if (t >= v.total) return none;
    if (len < 0 || len > v.max_len || s0 < 0 || s1 > v.total || s1 < s0) {
        atomicOr(v.err, kErrLength);
        return none;
    }
    const int64_t pos = len - (s1 - s0) + (t - s0);
    if (t >= s1 || pos < 0) return none;
    const uint32_t i = fast_div((uint32_t)pos, v.div_page);
    return PagedPlace{v.pages[s * v.stride + i], (uint32_t)pos - i * v.page};
}

__device__ __forceinline__ int64_t paged_row(const PagedView &v, const PagedLanes &l, int64_t t, int H)
{
    return paged_place_row(v, paged_seek(v, l, t), H);
}

// ------------------------------------------------------------------ split attention over a paged batch
// The work of a batch is one line: sequence after sequence, in a sequence its
// units (kv-head, block of CB columns) one after another, in a unit its start
// (what a segment costs besides its stages, in stages: kSegStart, or nothing
// where the CTAs are enough for a stage each) and its stages of ST rows in row
// order.  CTA c takes the c-th run of `per` places,
// whatever lengths the sequences have, so all CTAs finish together; a run's
// stages of one unit are a segment (a run that ends within a start leaves the
// unit to the next CTA), and a unit's segments are merged by the combine.
// Segment (c, unit u) writes partial slot c + u: along the line c or u grows by
// one at every new segment, so slots are distinct, and at most CTAs + units of
// them are used.
//
// A CTA's first warp works the line out from the lengths (32 sequences at a
// time); the CTA of a unit's first segment leaves word of its slots for the
// combine.
//
// 16 sequences of 4096 rows with 4 new tokens and 64 q-heads: 82.0 us with a
// start of 2 stages, 83.9 with none, 84.2 with 4; with 1 token and head_dim 64
// (64 sequences of 2048 rows) 40.8, 40.3 and 43.3.
constexpr int kSegStart = 2;

// Whether sequence s, of n new tokens, is the split kernels'.
__device__ __forceinline__ bool paged_split_takes(const PagedSplit &ps, int s, int64_t n)
{
    return n <= ps.max_new && (n <= ps.wide || (ps.spill && ps.spill[s]));
}

// Stages and units of sequence s (none where it has no rows, no new tokens, or too many: those of long chunks are
// another kernel's, more than the call's bound nobody's).
__device__ __forceinline__ void paged_shape(const PagedSplit &ps, int s, int ST, int CB, int H, int G, int &stages, int &units)
{
    stages = units = 0;
    if (s >= ps.v.seqs) return;
    const int64_t n = paged_new(ps.v, s), len = paged_len(ps.v, s);
    if (n > ps.max_new) atomicOr(ps.v.err, kErrLength);
    if (n == 0 || len == 0 || !paged_split_takes(ps, s, n)) return;
    stages = (int)((uint32_t)(len + ST - 1) / (uint32_t)ST);
    units = (int)((uint32_t)(n * G + CB - 1) / (uint32_t)CB) * H;
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

// a / b for a, b >= 0: in 32 bits where they fit
__device__ __forceinline__ int64_t div_small(int64_t a, int64_t b)
{
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// A segment, as the CTA's threads read it from shared memory.
struct PagedSegment {
    int64_t s0, slot;              // first ragged row of the sequence; partial slot
    const int32_t *pages;          // the sequence's row of the page table
    int n, len;                    // new tokens, rows
    int h, hb, first, count;       // kv-head, column block, first stage, stages (none: the run is done)
};

// The CTA's place on the line and its current segment (two, so that the next
// one can be written while the current one is still read).
struct PagedWalk {
    int64_t end, per;     // of the CTA's run; places per CTA
    int64_t at;           // line position of the current unit's first stage
    int64_t up;           // units before sequence s
    int s, u, stages, units;  // sequence, unit in it; its stages per unit and its units
    int start;            // places of a unit's start
    PagedSegment seg[2];
};

// The segment of the current unit from `first` on, by one thread.
__device__ __forceinline__ void paged_segment(const PagedSplit &ps, const PagedWalk &w, PagedSegment &g, int first, int H)
{
    g.first = first;
    g.count = (int)imin64(w.stages, w.end - w.at) - first;
    const int blocks = w.units / H;
    g.h = w.u / blocks;
    g.hb = w.u - g.h * blocks;
    g.slot = blockIdx.x + w.up + w.u;
    g.pages = ps.v.pages + w.s * ps.v.stride;
    if (first == 0 && g.count > 0 && g.hb < ps.blocks)
        ps.units[((int64_t)w.s * H + g.h) * ps.blocks + g.hb] =
            PagedUnit{(int)g.slot, (int)(div_small(w.at + w.stages - 1, w.per) - blockIdx.x) + 1};
    g.s0 = paged_start(ps.v, w.s);
    g.n = (int)paged_new(ps.v, w.s);
    g.len = (int)paged_len(ps.v, w.s);
}

// The CTA's first segment into w.seg[0], by the first warp (whole).  The caller
// synchronises the CTA before w is read.
__device__ __forceinline__ void paged_walk_start(const PagedSplit &ps, PagedWalk &w, int ST, int CB, int H, int G, int lane)
{
    const int S = ps.v.seqs;
    int st, un;
    paged_shape(ps, lane, ST, CB, H, G, st, un);
    int64_t total = (int64_t)st * un, units = un;
    for (int b = 32; b < S; b += 32) {
        int st1, un1;
        paged_shape(ps, b + lane, ST, CB, H, G, st1, un1);
        total += (int64_t)st1 * un1;
        units += un1;
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        total += __shfl_xor_sync(0xffffffffu, total, o);
        units += __shfl_xor_sync(0xffffffffu, units, o);
    }
    const int start = total <= gridDim.x ? 0 : kSegStart;
    total += start * units;
    int64_t per = div_small(total + gridDim.x - 1, gridDim.x);
    if (per < start + 1) per = start + 1;
    const int64_t x = blockIdx.x * per, end = imin64(total, x + per);
    if (lane == 0) {
        w.end = end;
        w.per = per;
        w.start = start;
        w.seg[0].count = 0;
    }
    __syncwarp();
    int64_t sbase = 0, ubase = 0;
    bool found = x >= end;
    for (int b = 0; b < S && !found; b += 32) {
        if (b > 0) paged_shape(ps, b + lane, ST, CB, H, G, st, un);
        const int64_t c = (int64_t)(st + start) * un;
        const int64_t ws = warp_inclusive_sum(c, lane), us = warp_inclusive_sum(un, lane);
        const int64_t s_at = sbase + ws - c, u_at = ubase + us - un;
        const bool mine = c > 0 && s_at <= x && x < s_at + c;
        if (mine) {
            const int64_t u = div_small(x - s_at, st + start);
            w.s = b + lane;
            w.up = u_at;
            w.stages = st;
            w.units = un;
            w.u = (int)u;
            w.at = s_at + u * (st + start) + start;
            paged_segment(ps, w, w.seg[0], x > w.at ? (int)(x - w.at) : 0, H);
        }
        found |= __any_sync(0xffffffffu, mine);
        sbase += __shfl_sync(0xffffffffu, ws, 31);
        ubase += __shfl_sync(0xffffffffu, us, 31);
    }
}

// On to the next unit's segment, by one thread, into `nxt` (count <= 0: the run is done).
__device__ __forceinline__ void paged_walk_next(const PagedSplit &ps, PagedWalk &w, PagedSegment &nxt, int ST, int CB, int H, int G)
{
    nxt.count = 0;
    w.at += w.stages + w.start;  // of the next unit
    if (w.at >= w.end) return;
    if (++w.u == w.units) {  // the next sequence with work (w.at < w.end says that there is one)
        w.up += w.units;
        w.u = 0;
        do {
            ++w.s;
            paged_shape(ps, w.s, ST, CB, H, G, w.stages, w.units);
        } while (w.units == 0);
    }
    paged_segment(ps, w, nxt, 0, H);
}

// A stage is copied in chunks of ps.ru = gcd(stage rows, page rows) rows, so that
// no chunk crosses a page; lane c of the refilling warp copies chunk c.

// Row of the sequence where chunk `chunk` of `stage` starts.
__device__ __forceinline__ uint32_t paged_chunk_row(const PagedSplit &ps, int stage, int chunk)
{
    return (uint32_t)((stage * ps.nch + chunk) * ps.ru);
}

// Page number (unchecked) of the lane's chunk of `stage`, 0 where it has no rows.
__device__ __forceinline__ int paged_chunk_page(const PagedSplit &ps, const PagedSegment &g, int stage, int lane)
{
    const uint32_t row = paged_chunk_row(ps, stage, lane);
    if (lane >= ps.nch || row >= (uint32_t)g.len) return 0;
    return g.pages[fast_div(row, ps.v.div_page)];
}

// Plane row of that chunk for the segment's kv-head; a bad page number is
// recorded, and page 0 read in its place.
__device__ __forceinline__ int64_t paged_chunk_plane_row(const PagedSplit &ps, const PagedSegment &g, int H, int page,
                                                         int stage, int chunk)
{
    if ((uint32_t)page >= (uint32_t)ps.v.num_pages) {
        atomicOr(ps.v.err, kErrPage);
        page = 0;
    }
    const uint32_t row = paged_chunk_row(ps, stage, chunk);
    return ((int64_t)page * H + g.h) * ps.v.page + (row - fast_div(row, ps.v.div_page) * ps.v.page);
}

}  // namespace tq
