"""The paged calls on the host: argument refusals (nothing here launches a
kernel; the pointers are never read) and a model of the split kernels' schedule."""
import ctypes

import numpy as np
import pytest

from test_abi_host import _struct

NULL, SHAPE, CAPACITY, ALIGN, WORKSPACE = 1, 4, 5, 6, 7


def _table(tqlib, **kw):
    f = dict(pages=0x100000, seq_lens=0x200000, stride=4, max_len=128, total_len=0, num_seqs=3, reserved=0)
    f.update(kw)
    return tqlib._PageTableStruct(*[f[n] for n, _ in tqlib._PageTableStruct._fields_])


def _two(*x):
    return (ctypes.c_int64 * 2)(*x)


def test_shared_refusals(tqlib):
    """Pool, table, starts and total are checked alike by all three calls."""
    L = tqlib.lib()
    ref = ctypes.byref

    def calls(pool, table, starts=0x300000, total=4):
        p, t = (ref(pool) if pool is not None else None), (ref(table) if table is not None else None)
        st = _two(256, 128)
        return {L.tq_paged_append(p, t, starts, total, 0x10000, st, 0x20000, st, None),
                L.tq_paged_decode(p, t, starts, total, 0, 0x10000, 0x20000, None),
                L.tq_paged_attention(p, t, starts, total, 1, 0x10000, st, 4, 1.0, 0x20000, None, 0, None)}

    pool, table = _struct(tqlib, batch=12), _table(tqlib)  # 12 pages of 32 rows, 2 kv-heads
    assert calls(None, table) == {NULL}
    assert calls(pool, None) == {NULL}
    assert calls(pool, table, starts=None) == {NULL}
    assert calls(_struct(tqlib, capacity=40), table) == {SHAPE}
    assert calls(pool, _table(tqlib, pages=0)) == {NULL}
    assert calls(pool, _table(tqlib, seq_lens=0)) == {NULL}
    assert calls(pool, _table(tqlib, num_seqs=0)) == {SHAPE}
    assert calls(pool, _table(tqlib, reserved=1)) == {SHAPE}
    assert calls(pool, _table(tqlib, max_len=0)) == {SHAPE}
    assert calls(pool, _table(tqlib, total_len=-1)) == {SHAPE}
    assert calls(pool, _table(tqlib, max_len=1 << 31, stride=1 << 30)) == {SHAPE}
    assert calls(pool, _table(tqlib, max_len=129)) == {CAPACITY}  # 4 pages of 32 rows hold 128
    assert calls(pool, table, total=-1) == {SHAPE}
    assert calls(pool, table, total=1 << 31) == {SHAPE}
    assert calls(pool, table, total=0) == {0}  # nothing to do


def test_append_and_decode_refusals(tqlib):
    L, ref = tqlib.lib(), ctypes.byref
    pool, table = _struct(tqlib, batch=12), _table(tqlib)

    def append(k=0x10000, ks=(256, 128), v=0x20000, vs=(256, 128)):
        return L.tq_paged_append(ref(pool), ref(table), 0x300000, 4, k, _two(*ks), v, _two(*vs), None)

    assert append(k=None) == NULL and append(v=None) == NULL
    assert append(k=0x10008) == ALIGN and append(vs=(256, 100)) == ALIGN
    assert append(ks=(-256, 128)) == SHAPE
    decode = lambda k, v, dt=0: L.tq_paged_decode(ref(pool), ref(table), 0x300000, 4, dt, k, v, None)  # noqa: E731
    assert decode(0x10010, None) == ALIGN and decode(None, 0x10010) == ALIGN
    assert decode(0x10000, 0x20000, 7) == SHAPE
    assert decode(None, None) == 0


def test_attention_refusals(tqlib):
    L, ref = tqlib.lib(), ctypes.byref
    pool, table = _struct(tqlib, batch=12), _table(tqlib)

    def attend(q=0x10000, qs=(512, 128), heads=4, total=4, max_new=1, out=0x20000, ws=None, nbytes=0):
        return L.tq_paged_attention(ref(pool), ref(table), 0x300000, total, max_new, q, _two(*qs), heads, 1.0, out, ws,
                                    nbytes, None)

    assert attend(heads=3) == SHAPE and attend(heads=0) == SHAPE
    assert attend(max_new=0) == SHAPE
    assert attend(total=1 << 29, heads=4) == SHAPE  # 2^31 output rows
    assert attend(q=None) == NULL and attend(out=None) == NULL
    assert attend(q=0x10004) == ALIGN and attend(qs=(512, 4)) == ALIGN and attend(out=0x20008) == ALIGN
    assert attend(qs=(512, -128)) == SHAPE
    size = L.tq_paged_attention_workspace_bytes
    assert size(ref(pool), ref(table), 3, 4, 1) == 0
    assert size(ref(pool), ref(table), 4, 4, 0) == 0
    assert size(ref(pool), ref(_table(tqlib, max_len=129)), 4, 4, 1) == 0


def test_device_error_codes_match_the_header(tqlib):
    from conftest import ROOT

    text = open(f"{ROOT}/include/tq.h").read()
    assert f"#define TQ_DEVICE_ERR_PAGE {tqlib.TQ_DEVICE_ERR_PAGE}u" in text
    assert f"#define TQ_DEVICE_ERR_LENGTH {tqlib.TQ_DEVICE_ERR_LENGTH}u" in text


def test_binding_refusals_on_the_host(tqlib):
    """Shapes and types that the binding refuses before the library is reached."""
    import torch

    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        tqlib.PageTable(torch.zeros(2, 3, dtype=torch.int64), i32(2), 16)
    with pytest.raises(ValueError):
        tqlib.PageTable(i32(2, 3), i32(3), 16)
    with pytest.raises(ValueError):
        tqlib.PageTable(i32(3, 2).t(), i32(2), 16)  # a sequence's pages not contiguous
    with pytest.raises(ValueError):
        tqlib.PageTable(i32(2, 3), i32(2))  # no bound
    with pytest.raises(ValueError):
        tqlib.PageTable(i32(2, 3), i32(2), 16)  # not on a CUDA device
    with pytest.raises(ValueError):
        tqlib.Cache.from_planes(*[torch.zeros(2, 1, 16, 5, dtype=torch.uint8)] * 5, head_dim=64)


def _schedule(lens, new, H, G, ST, CB, ctas, seg_start=2):
    """The split kernels' line: per CTA its segments (sequence, kv-head, block, first stage, count, slot), and per
    unit the word that its first segment leaves (first slot, segments)."""
    units = []  # (sequence, kv-head, block, stages)
    for s, (n, m) in enumerate(zip(lens, new)):
        if n and m:
            units += [(s, h, b, -(-n // ST)) for h in range(H) for b in range(-(-(m * G) // CB))]
    stages = sum(u[3] for u in units)
    start = 0 if stages <= ctas else seg_start
    per = max(start + 1, -(-(stages + start * len(units)) // ctas))
    out, words, at = {}, [], 0
    for i, (s, h, b, n) in enumerate(units):
        at += start  # its first stage
        x = at
        words.append((at // per + i, (at + n - 1) // per - at // per + 1))
        while x < at + n:
            c = x // per
            count = min(at + n, (c + 1) * per) - x
            out.setdefault(c, []).append((s, h, b, x - at, count, c + i))
            x += count
        at += n
    return out, words


@pytest.mark.parametrize("seed", range(8))
def test_schedule_slots_are_distinct_and_bounded(seed):
    rng = np.random.default_rng(seed)
    S, H, G = int(rng.integers(1, 40)), int(rng.integers(1, 9)), int(rng.integers(1, 17))
    lens = rng.integers(0, 5000 if seed < 6 else 70, S) * (rng.random(S) > 0.2)
    new = np.minimum(lens, rng.integers(0, 6, S))
    ST, CB, ctas = 64, 8, int(rng.integers(1, 1300))
    segs, words = _schedule(lens, new, H, G, ST, CB, ctas)
    units = len(words)
    assert all(c < ctas for c in segs)
    flat = [x for c in sorted(segs) for x in segs[c]]
    slots = [x[5] for x in flat]
    assert slots == sorted(set(slots))                     # distinct, growing along the line
    assert not slots or slots[-1] < ctas + units           # what the workspace has room for
    assert units <= H * (int(new.sum()) * G // CB + S)     # the host's bound of the units
    # every unit's segments are consecutive slots, and the word of its first one names them
    seen = {}
    for s, h, b, first, count, slot in flat:
        seen.setdefault((s, h, b), []).append((first, count, slot))
    for ((s, h, b), parts), word in zip(seen.items(), words):
        assert parts[0][0] == 0 and sum(p[1] for p in parts) == -(-int(lens[s]) // ST)
        assert [p[2] for p in parts] == list(range(word[0], word[0] + word[1]))


@pytest.mark.parametrize("seed", range(6))
def test_wide_line_covers_every_block_once(seed):
    """The wide kernel's line: each run's tiles of a block from its first tile on, shares in two slots a CTA, and the
    CTA that begins a block knowing the last one that has a share."""
    rng = np.random.default_rng(100 + seed)
    tiles = [int(x) for x in rng.integers(1, 60, int(rng.integers(1, 200)))]
    start, ctas = 7, int(rng.integers(1, 160))
    total = sum(tiles) + start * len(tiles)
    per = max(start, -(-total // ctas))
    firsts, at = [], 0
    for n in tiles:
        firsts.append(at + start)
        at += start + n
    done = [0] * len(tiles)
    used, shares = set(), {}
    for c in range(ctas):
        x0, x1 = c * per, min(total, (c + 1) * per)
        for b, n in enumerate(tiles):
            if firsts[b] + n <= x0 or firsts[b] - start >= x1:
                continue
            lo, hi = max(0, x0 - firsts[b]), min(n, x1 - firsts[b])
            if hi <= lo:
                continue
            assert done[b] == lo
            done[b] = hi
            if hi - lo < n:  # a share: slot 2 c of a CTA that goes on with the block, 2 c + 1 of the one that begins it
                slot = 2 * c + (lo == 0)
                assert slot not in used
                used.add(slot)
                shares.setdefault(b, []).append(slot)
    assert done == tiles
    for b, slots in shares.items():
        c = slots[0] // 2
        last = (firsts[b] + tiles[b] - 1) // per
        assert slots == [2 * c + 1] + [2 * k for k in range(c + 1, last + 1)]


@pytest.mark.parametrize("stage", [64, 96, 128])
@pytest.mark.parametrize("page", [16, 32, 48, 64, 80, 96, 128, 160, 256])
def test_stage_chunks_never_cross_a_page(stage, page):
    ru = int(np.gcd(stage, page))
    assert ru >= 16 and stage % ru == 0 and stage // ru <= 8
    for st in range(2 * page):
        for c in range(stage // ru):
            row = st * stage + c * ru
            assert row // page == (row + ru - 1) // page


def test_bounds_above_any_memory(tqlib):
    """Workspace sizes grow with the bounds and pass no integer's range: above 2^37 rows x kv-heads no expanded tiles
    (512 bytes a row and kv-head at head_dim 128) are asked for, whose counts are 32-bit."""
    L, ref = tqlib.lib(), ctypes.byref
    pool = _struct(tqlib, batch=12)
    H = pool.num_kv_heads

    def size(seqs, max_len, total):
        table = _table(tqlib, num_seqs=seqs, max_len=max_len, stride=1 << 32)
        return L.tq_paged_attention_workspace_bytes(ref(pool), ref(table), 2 * H, total, total)

    rows = 1 << 20
    assert size(1, rows, 4096) > rows * H * 512
    last = 0
    for seqs, max_len in ((64, 1 << 20), (1 << 10, 1 << 24), (1 << 22, 1 << 30), (1 << 26, (1 << 31) - 1)):
        new = size(seqs, max_len, 1 << 28)
        assert last < new < 1 << 60
        if seqs * max_len * H >= 1 << 37:
            assert new < seqs * max_len * H
        last = new


def test_workspace_of_ordinary_serving_bounds(tqlib):
    """Slots and lengths as a server states them once and for all, far above what a batch holds: a bounded workspace,
    and a smaller one where the sum of the lengths is known."""
    L, ref = tqlib.lib(), ctypes.byref
    pool = _struct(tqlib, head_dim=128, num_kv_heads=8, batch=20000, capacity=64, v_bits=3)

    def size(seqs, max_len, total, new, total_len=0):
        table = _table(tqlib, num_seqs=seqs, max_len=max_len, stride=max_len // 64, total_len=total_len)
        return L.tq_paged_attention_workspace_bytes(ref(pool), ref(table), 64, total, new)

    gib = 1 << 30
    for seqs, max_len, total, new in ((256, 131072, 8192, 8192), (64, 131072, 2048, 2048), (1024, 1 << 20, 4096, 512)):
        assert 0 < size(seqs, max_len, total, new) < 9 * gib
    assert size(64, 131072, 2048, 2048, total_len=262144) < 2 * gib  # 262144 rows x 8 kv-heads x 768 bytes and the rest
    one = size(1, 131072, 2048, 2048)  # within the limit: room for every row
    assert one > 131072 * 8 * 6 * 128


@pytest.mark.parametrize("capacity", [1 << 31, (1 << 32) - 16, 1 << 32, (1 << 32) + 32, 1 << 40])
def test_pages_of_2_31_rows_are_refused(tqlib, capacity):
    """Positions and page sizes are 32-bit in the kernels: a larger page is refused before its size is cut off."""
    L, ref = tqlib.lib(), ctypes.byref
    pool, table = _struct(tqlib, batch=12, capacity=capacity), _table(tqlib)
    st = _two(256, 128)
    assert L.tq_paged_append(ref(pool), ref(table), 0x300000, 4, 0x10000, st, 0x20000, st, None) == SHAPE
    assert L.tq_paged_decode(ref(pool), ref(table), 0x300000, 4, 0, 0x10000, 0x20000, None) == SHAPE
    assert L.tq_paged_attention(ref(pool), ref(table), 0x300000, 4, 1, 0x10000, st, 4, 1.0, 0x20000, None, 0, None) == SHAPE
    assert L.tq_paged_attention_workspace_bytes(ref(pool), ref(table), 4, 4, 1) == 0
    most = _struct(tqlib, batch=12, capacity=(1 << 31) - 16)
    assert L.tq_paged_append(ref(most), ref(table), 0x300000, 0, 0x10000, st, 0x20000, st, None) == 0
