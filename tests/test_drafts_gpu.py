"""A step of drafted tokens on the GPU: page tables, layouts, rotary positions, attention of trees, verification and kept
rows, each against a plain implementation in 64 bits (or whole numbers), and all of them together."""
import numpy as np
import pytest
import torch

from pagedtest import ATOL, RTOL, Batch, dequantised, rows_of

pytestmark = pytest.mark.gpu


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x)).to(dtype).cuda()


def random_parents(rng, n, wide=4):
    return [-1 if i == 0 else int(max(0, rng.integers(max(0, (i - 1) // wide - 1), i))) for i in range(n)]


def ancestors(parents):
    up = []
    for i, p in enumerate(parents):
        up.append([i] + (up[p] if p >= 0 else []))
    return up


def pack(seen, words):
    """Truth values [rows][n] -> int32 [rows][words]."""
    out = np.zeros((len(seen), words), np.uint32)
    for i, row in enumerate(seen):
        for j in np.flatnonzero(row):
            out[i, j // 32] |= np.uint32(1) << np.uint32(j % 32)
    return out.view(np.int32)


# ------------------------------------------------------------------ attention of trees
def tree_masks(b, kind, seed=3):
    """What every new token sees of its sequence's new ones: truth values [n][n] per sequence."""
    rng = np.random.default_rng(seed)
    out = []
    for n in b.new:
        if kind == "tree":
            m = np.zeros((n, n), bool)
            for i, up in enumerate(ancestors(random_parents(rng, n))):
                m[i, up] = True
        elif kind == "chain":
            m = np.tril(np.ones((n, n), bool))
        else:  # anything, later tokens and empty rows among it
            m = rng.random((n, n)) < 0.4
            if n > 1:
                m[rng.integers(0, n)] = False
        out.append(m)
    return out


def attend64(q, k, v, before, seen):
    """q [n][QH][d] over k, v [H][len][d]: rows below `before` and those of `seen` [n][len - before]."""
    n, QH, d = q.shape
    H, L = k.shape[:2]
    k, v = torch.from_numpy(k).double(), torch.from_numpy(v).double()
    vis = torch.ones(n, L, dtype=torch.bool)
    vis[:, before:] = torch.from_numpy(seen[:, :L - before])
    s = torch.einsum("mhgd,hnd->hmgn", q.double().view(n, H, QH // H, d), k) * d ** -0.5
    s = s.masked_fill(~vis[None, :, None], -float("inf"))
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(top), torch.zeros_like(top), top)).masked_fill(~vis[None, :, None], 0.0)
    l = p.sum(-1, keepdim=True)
    p = p / torch.where(l == 0, torch.ones_like(l), l)
    o = torch.stack([torch.einsum("hgn,hnd->hgd", p[:, i][..., vis[i]], v[:, vis[i]]) for i in range(n)], 1)
    return o.permute(1, 0, 2, 3).reshape(n, QH, d)


def check_tree(b, pool, q, out, seen, new=None):
    at, worst, out = 0, 0.0, out.cpu().double()
    for s, (n, m) in enumerate(zip(b.lens, b.new if new is None else new)):
        if not m:
            continue
        k, v = dequantised(pool, b.table[s], n)
        want = attend64(q[at:at + m].cpu(), k, v, n - m, seen[s])
        got = out[at:at + m]
        assert torch.equal(torch.isfinite(got), torch.isfinite(want)), f"sequence {s}: not finite elsewhere"
        worst = max(worst, float(((got - want).abs() - RTOL * want.abs()).nan_to_num(0.0).max()))
        at += m
    assert worst <= ATOL, worst


def run_tree(tq, b, QH, seen, seed=1, rubbish=True, pool=None, **kw):
    if pool is None:
        pool = b.pool(tq)
        b.fill(tq, pool)
    max_new = max(max(b.new), 1)
    words = -(-max_new // 32) + 1
    masks = np.zeros((b.total + b.pad_rows, words), np.int32)
    at = 0
    for m in seen:
        n = len(m)
        wide = np.zeros((n, 32 * words), bool)
        wide[:, n:] = rubbish  # bits behind the sequence's new tokens
        wide[:, :n] = m
        masks[at:at + n] = pack(wide, words)
        at += n
    q = b.queries(QH, seed)
    out = tq.tq_paged_tree_attention(pool, b.pages(tq), b.dev(b.starts), q.cuda(), dev(masks), max_new, **kw)
    return pool, q, out


TREES = [  # head_dim, key and value bits, group, page, new tokens: the specialised, generic and wide kernels
    (128, 8, 3, 8, 64, 4), (128, 4, 3, 8, 32, 3), (128, 8, 4, 5, 16, 7), (128, 4, 2, 16, 128, 2), (64, 8, 4, 4, 16, 5),
    (64, 4, 3, 8, 48, 9), (256, 8, 3, 4, 32, 4), (256, 4, 4, 16, 64, 3), (512, 8, 3, 2, 16, 6), (128, 5, 5, 3, 80, 8),
    (64, 2, 8, 2, 16, 12), (256, 5, 2, 5, 48, 11), (512, 4, 5, 4, 32, 9), (128, 8, 3, 1, 64, 40), (64, 8, 3, 3, 64, 33),
    (128, 8, 3, 8, 64, 40), (64, 4, 2, 8, 16, 70), (128, 4, 3, 4, 48, 65), (128, 5, 2, 16, 16, 33), (64, 8, 8, 16, 32, 129),
    (256, 8, 4, 4, 128, 33), (512, 2, 2, 1, 16, 50), (128, 8, 3, 2, 64, 64), (128, 4, 4, 3, 32, 37), (64, 8, 2, 5, 16, 25),
    (256, 4, 3, 2, 64, 64),
]


@pytest.mark.parametrize("kind", ["tree", "any"])
@pytest.mark.parametrize("d,kb,vb,G,page,new", TREES)
def test_tree_attention(cuda, d, kb, vb, G, page, new, kind):
    """Up to `new` tokens a sequence: fewer in some, as many as rows in others, lengths around stages and tiles."""
    lens = [1, 2, new, new + 1, 64, 65, 0, 127 + new, 128 + new, 129, 777]
    b = Batch(lens, [min(n, 1 + (i * 7 + new) % new) if i != 8 else min(n, new) for i, n in enumerate(lens)], H=2, d=d, kb=kb, vb=vb,
              page=page, seed=new)
    seen = tree_masks(b, kind)
    pool, q, out = run_tree(cuda, b, 2 * G, seen)
    check_tree(b, pool, q, out, seen)
    assert cuda.tq_device_error() == 0


@pytest.mark.parametrize("d,kb,vb,G,new", [(128, 8, 3, 8, 8), (128, 4, 3, 4, 64), (64, 8, 4, 8, 40), (256, 8, 4, 4, 16), (128, 8, 3, 8, 1)])
def test_a_chain_is_causal(cuda, d, kb, vb, G, new):
    """Masks of a chain give what the causal call gives, each within its tolerance of the same value."""
    b = Batch([3000, 500, new], [new, max(1, new // 2), new], H=2, d=d, kb=kb, vb=vb, page=64)
    pool, q, out = run_tree(cuda, b, 2 * G, tree_masks(b, "chain"))
    causal = cuda.tq_paged_attention(pool, b.pages(cuda), b.dev(b.starts), q.cuda(), max(b.new))
    err = (out.double() - causal.double()).abs() - 2 * RTOL * causal.double().abs()
    assert float(err.max()) <= 2 * ATOL


@pytest.mark.parametrize("d,kb,G,new", [(128, 8, 8, 6), (128, 8, 8, 40), (64, 4, 4, 64), (256, 4, 4, 9), (512, 8, 2, 5), (128, 5, 4, 12)])
def test_hidden_rows_hold_anything(cuda, d, kb, G, new):
    """NaN and infinities in new rows that a token does not see never reach it; a token that sees nothing gives zeros."""
    b = Batch([300, new], [new, new], H=2, d=d, kb=kb, vb=3, page=32)
    pool = b.pool(cuda)
    b.fill(cuda, pool)
    bad = [1, new - 1]
    seen = [np.zeros((n, n), bool) for n in b.new]
    for m in seen:
        for i in range(len(m)):
            m[i, [j for j in range(len(m)) if j not in bad and (j + i) % 3 == 0]] = True
    seen[1][0] = False  # a whole sequence of new tokens, and one that sees none of them
    for s, n in enumerate(b.lens):
        for j in bad:
            row = n - new + j
            page, slot = b.table[s, row // 32], row % 32
            for t, x in ((pool.k_scale, 0x7C00), (pool.k_zero, 0x7E00), (pool.v_scale, 0x7E00 if j == 1 else 0x7C00)):
                t[int(page), :, int(slot)] = x
    _, q, out = run_tree(cuda, b, 2 * G, seen, pool=pool)
    assert bool(torch.isfinite(out).all())
    assert bool((out[b.starts[1]] == 0).all())
    check_tree(b, pool, q, out, seen)


def test_tree_outputs_streams_and_padding(cuda):
    """Rows behind the last sequence keep what they held; another stream, given workspace and output; q in strides."""
    b = Batch([100, 40], [9, 20], H=2, d=128, kb=8, vb=3, page=32, pad_rows=5)
    seen = tree_masks(b, "tree")
    out = torch.full((b.total + 5, 16, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    pool, q, got = run_tree(cuda, b, 16, seen, out=out)
    assert got is out and bool((out[b.total:] == 7).all())
    check_tree(b, pool, q, out, seen)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    _, _, other = run_tree(cuda, b, 16, seen, pool=pool, stream=s)
    s.synchronize()
    assert torch.equal(other[:b.total], out[:b.total])
    wide = torch.zeros(b.total + 5, 32, 128, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:24] = q.cuda()
    masks = dev(pack(np.concatenate([np.pad(m, ((0, 0), (0, 32 - len(m)))) for m in seen] + [np.zeros((5, 32), bool)]), 1))
    again = cuda.tq_paged_tree_attention(pool, b.pages(cuda), b.dev(b.starts), wide[:, 8:24], masks, 20)
    assert torch.equal(again[:b.total], out[:b.total])


def test_more_tokens_than_the_bound_are_reported(cuda):
    b = Batch([100, 40], [9, 20], H=2, d=128, kb=8, vb=3, page=32)
    pool = b.pool(cuda)
    b.fill(cuda, pool)
    out = torch.full((29, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    masks = torch.full((29, 1), -1, dtype=torch.int32, device="cuda")
    cuda.tq_paged_tree_attention(pool, b.pages(cuda), b.dev(b.starts), b.queries(4).cuda(), masks, 10, out=out)
    assert cuda.tq_device_error() == cuda.TQ_DEVICE_ERR_LENGTH
    assert bool((out[9:] == 7).all())  # that sequence gets no results


# ------------------------------------------------------------------ page tables
class TableModel:
    """What tq_page_table_update says, in Python."""

    def __init__(self, rng, seqs, width, page, pages):
        self.page, self.width = page, width
        self.table = np.full((seqs, width), -1, np.int64)
        self.free = list(rng.permutation(pages))
        self.lens = [0] * seqs

    def update(self, want):
        c = lambda n: -(-n // self.page)  # noqa: E731
        free, table = list(self.free), self.table.copy()
        for s, (a, b) in enumerate(zip(self.lens, want)):
            free += [int(x) for x in table[s, c(b):c(a)]]
        for s, (a, b) in enumerate(zip(self.lens, want)):
            for i in range(c(a), c(b)):
                if not free:
                    return False
                table[s, i] = free.pop()
        self.free, self.table, self.lens = free, table, list(want)
        return True


@pytest.mark.parametrize("seqs,page,width", [(1, 16, 4), (7, 32, 40), (200, 16, 9), (1025, 48, 5), (3000, 16, 3)])
def test_tables_follow_the_lengths(cuda, seqs, page, width):
    """Sequences that grow, shrink, begin and end, in place, for many steps; a step that the pool has no pages for
    changes nothing."""
    rng = np.random.default_rng(seqs)
    most, pages = width * page, max(2, seqs * width * 2 // 3)
    m = TableModel(rng, seqs, width, page, pages)
    pool = cuda.Cache(pages, 1, 64, page, k_bits=2, v_bits=2)
    table = cuda.PageTable(dev(m.table), dev(m.lens), most)
    free = dev(m.free + [-7] * 3)
    count = dev([len(m.free)])
    full = 0
    for step in range(24):
        want = [int(rng.integers(0, most + 1)) if rng.random() < 0.15 else 0 if rng.random() < 0.1 else
                int(np.clip(n + rng.integers(-20, 40), 0, most)) for n in m.lens]
        if step == 20:
            want = [most] * seqs  # more than there is (but for the smallest pools)
        new = [int(rng.integers(0, n + 1)) for n in want]
        before = list(m.lens)
        good = m.update(want)
        starts = cuda.tq_page_table_update(pool, table, dev(want), free, count, new_tokens=dev(new))
        err = cuda.tq_device_error()
        full += not good
        assert err == (0 if good else cuda.TQ_DEVICE_ERR_FULL)
        assert table.seq_lens.tolist() == (want if good else before)
        assert starts.tolist() == ([0] + np.cumsum(new).tolist() if good else [0] * (seqs + 1))
        assert int(count) == len(m.free) and free.tolist()[:len(m.free)] == [int(x) for x in m.free]
        for s, n in enumerate(m.lens):
            k = -(-n // page)
            assert np.array_equal(table.pages[s, :k].cpu().numpy(), m.table[s, :k])
    assert full > 0


def test_table_update_out_of_place_and_bad_values(cuda):
    pool = cuda.Cache(8, 1, 64, 16, k_bits=2, v_bits=2)
    pages, old = dev([[5, 1, -1], [2, -1, -1]]), dev([20, 16])
    table = cuda.PageTable(pages, old, 48)
    free, count, out, left = dev([0, 3, 4, 6, 7, 9]), dev([5]), dev([-1, -1]), dev([-1])
    call = lambda want, **kw: cuda.tq_page_table_update(pool, table, dev(want), free, count, lens_out=out, free_count_out=left, **kw)  # noqa: E731
    assert call([0, 48]) is None  # two pages given back to a stack with room for one
    assert cuda.tq_device_error() == cuda.TQ_DEVICE_ERR_FULL and out.tolist() == [20, 16] and int(left) == 5
    free = dev([0, 3, 4, 6, 7, 9, 9])
    for _ in range(2):  # nothing that the call reads is written: the same again
        assert call([0, 48]) is None
        assert out.tolist() == [0, 48] and int(left) == 5 and free.tolist() == [0, 3, 4, 6, 7, 5, 1]
        assert pages.tolist() == [[5, 1, -1], [2, 1, 5]] and old.tolist() == [20, 16] and int(count) == 5
    assert cuda.tq_device_error() == 0
    free, before = dev([0, 3, 4, 6, 7, 9]), pages.tolist()
    for want, kw, code in (([-1, 16], {}, 4), ([20, 49], {}, 4), ([20, 16], dict(new_tokens=dev([21, 0])), 4),
                           ([20, 16], dict(new_tokens=dev([0, -1])), 4)):
        starts = call(want, **kw)
        assert cuda.tq_device_error() == code
        assert out.tolist() == [20, 16] and int(left) == 5 and pages.tolist() == before and free.tolist() == [0, 3, 4, 6, 7, 9]
        assert starts is None or starts.tolist() == [0, 0, 0]
    count.fill_(7)  # more than the stack holds
    call([20, 16])
    assert cuda.tq_device_error() == cuda.TQ_DEVICE_ERR_FULL and int(left) == 7
    count.fill_(6)  # no room for the two pages given back
    call([0, 16])
    assert cuda.tq_device_error() == cuda.TQ_DEVICE_ERR_FULL and int(left) == 6
    pages[0, 1] = 8  # no page of this pool
    count.fill_(4)
    call([16, 16])
    assert cuda.tq_device_error() == cuda.TQ_DEVICE_ERR_PAGE and int(left) == 5


# ------------------------------------------------------------------ layouts
@pytest.mark.parametrize("seqs,page,most", [(1, 16, 1), (5, 32, 70), (40, 48, 33), (300, 16, 9)])
def test_layout(cuda, seqs, page, most):
    rng = np.random.default_rng(seqs + most)
    lens = [int(x) for x in rng.integers(0, 200, seqs)]
    new = [min(n, int(rng.integers(0, most + 1))) for n in lens]
    lens[0], new[0] = most + 3, most
    if seqs > 1:
        lens[1], new[1] = 2, min(4, most)  # more new tokens than rows
    b = Batch([max(lens)] * seqs, [0] * seqs, H=1, d=64, kb=2, vb=2, page=page)
    pool = b.pool(cuda)
    table = cuda.PageTable(dev(b.table), dev(lens), max(lens))
    starts, total = dev(np.cumsum([0] + new)), sum(new)
    parents = [random_parents(rng, n) for n in new]
    pad = 3
    flat = dev([p for t in parents for p in t] + [0] * pad)
    pos, slots, masks = cuda.tq_paged_layout(pool, table, starts, total + pad, parents=flat, max_new=most)
    rows, line, none = cuda.tq_paged_layout(pool, table, starts, total + pad)
    assert none is None and torch.equal(line, slots) and cuda.tq_device_error() == 0
    at = 0
    for s, n in enumerate(new):
        up = ancestors(parents[s])
        for i in range(n):
            row = lens[s] - n + i
            assert int(rows[at]) == (row if row >= 0 else -1)
            assert int(slots[at]) == (int(b.table[s, row // page]) * page + row % page if row >= 0 else -1)
            depth = lens[s] - n + len(up[i]) - 1
            assert int(pos[at]) == (depth if depth >= 0 else -1)
            seen = np.zeros((1, most), bool)
            seen[0, up[i]] = True
            assert masks[at].tolist() == pack(seen, -(-most // 32))[0].tolist()
            at += 1
    for x in (pos, rows, slots):
        assert x[total:].tolist() == [-1] * pad
    assert not bool(masks[total:].any())
    only = cuda.tq_paged_layout(pool, table, starts, total, parents=flat[:total].contiguous(), max_new=most, want_positions=False,
                                want_slots=False)
    assert only[:2] == (None, None) and torch.equal(only[2], masks[:total])


def test_layout_of_bad_trees_and_pages(cuda):
    pool = cuda.Cache(4, 1, 64, 16, k_bits=2, v_bits=2)
    table = cuda.PageTable(dev([[0, 9], [1, 2]]), dev([20, 30]), 32)
    starts = dev([0, 6, 9])
    parents = dev([-1, 0, 5, -2, 3, 4, -1, 0, 1])
    pos, slots, masks = cuda.tq_paged_layout(pool, table, starts, 9, parents=parents, max_new=6)
    assert cuda.tq_device_error() == cuda.TQ_DEVICE_ERR_TREE | cuda.TQ_DEVICE_ERR_PAGE
    assert masks[:, 0].tolist() == [1, 3, 4, 8, 24, 56, 1, 3, 7]  # a bad parent is a root's
    assert pos.tolist() == [14, 15, 14, 14, 15, 16, 27, 28, 29]
    assert slots.tolist() == [14, 15, -1, -1, -1, -1, 43, 44, 45]
    pos, slots, masks = cuda.tq_paged_layout(pool, table, starts, 9, parents=dev([-1] * 9), max_new=5)
    assert cuda.tq_device_error() == cuda.TQ_DEVICE_ERR_LENGTH  # six tokens
    assert pos.tolist()[:6] == [-1] * 6 and slots.tolist()[:6] == [-1] * 6 and masks.tolist() == [[0]] * 6 + [[1], [2], [4]]


def test_layout_of_starts_out_of_order(cuda):
    """Starts that fall: what is read stays within the tokens, the fault is recorded, sequences in order have their places."""
    seqs, total = 40, 400
    starts = np.arange(0, 10 * seqs + 1, 10)
    starts[20], starts[21] = 390, 15
    pool = cuda.Cache(seqs * 4, 1, 64, 16, k_bits=2, v_bits=2)
    table = cuda.PageTable(dev(np.arange(seqs * 4).reshape(seqs, 4)), dev([50] * seqs), 64)
    parents = np.tile(np.arange(-1, 9), seqs)
    for n in (10, 400):
        pos, slots, masks = cuda.tq_paged_layout(pool, table, dev(starts), total, parents=dev(parents), max_new=n)
        assert cuda.tq_device_error() & cuda.TQ_DEVICE_ERR_LENGTH
        assert pos[:100].tolist() == list(range(40, 50)) * 10 and masks[:100, 0].tolist() == [2 ** (i + 1) - 1 for i in range(10)] * 10


def test_layout_of_fewer_tokens_than_parents(cuda):
    """Parents kept for the largest batch: the first `total` count, none of them too; a shorter tensor is refused."""
    pool = cuda.Cache(8, 1, 64, 16, k_bits=2, v_bits=2)
    table = cuda.PageTable(dev(np.arange(8).reshape(2, 4)), dev([20, 9]), 64)
    parents = dev([-1, 0, 0, -1, 0, 7, 7, 7])
    pos, slots, masks = cuda.tq_paged_layout(pool, table, dev([0, 3, 5]), 5, parents=parents, max_new=3)
    assert pos.tolist() == [17, 18, 18, 7, 8] and slots.tolist() == [17, 18, 19, 71, 72] and masks.tolist() == [[1], [3], [5], [1], [3]]
    for few in (parents, parents[:0]):
        pos, slots, masks = cuda.tq_paged_layout(pool, table, dev([0, 0, 0]), 0, parents=few, max_new=3)
        assert pos.shape == (0,) and slots.shape == (0,) and masks.shape == (0, 1)
    assert cuda.tq_device_error() == 0
    with pytest.raises(ValueError):
        cuda.tq_paged_layout(pool, table, dev([0, 3, 5]), 5, parents=parents[:4], max_new=3)
    with pytest.raises(ValueError):
        cuda.tq_paged_layout(pool, table, dev([0, 3, 5]), 5, parents=parents[::2][:4], max_new=3)
    with pytest.raises(ValueError):
        cuda.tq_paged_layout(pool, table, dev([0, 3, 5]), 4, parents=parents.long(), max_new=3)


# ------------------------------------------------------------------ rotary
# Bounds: sine and cosine within 2 steps of 2^-24 (what the part left out adds one rounding), the scale and the
# two products and their sum one each: 6 steps of 2^-24 of (|a| + |b|) scale; then one rounding of the type.
ROTARY = [(64, 64), (128, 128), (128, 64), (128, 96), (128, 32), (256, 256), (256, 10), (512, 512), (512, 130), (64, 2), (128, 124), (64, 20)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", ROTARY)
def test_rotary(cuda, d, rot, interleaved, dtype):
    for tokens, QH, H, top in ((1, 8, 8, 1), (5, 7, 1, 1 << 20), (33, 40, 8, (1 << 31) - 1), (700, 3, 1, 4096)):
        g = torch.Generator(device="cuda").manual_seed(tokens)
        x = torch.randn(tokens, QH + 2 * H, d, generator=g, device="cuda").to(dtype)
        q, k = x[:, :QH], x[:, QH:QH + H]
        pos = torch.randint(0, top, (tokens,), generator=g, device="cuda", dtype=torch.int32)
        if tokens > 4:
            pos[3] = -1
        w, _ = cuda.tq_rotary_frequencies(rot)
        outs = [torch.full(t.shape, 7.0, dtype=dtype, device="cuda") for t in (q, k)]
        got = cuda.tq_rotary(pos, dev(w, torch.float64), q, k, interleaved=interleaved, scale=1.25, q_out=outs[0], k_out=outs[1])
        t = pos.cpu().numpy()[:, None].astype(np.float64) * w
        c, s = (torch.from_numpy(f(t))[:, None] * 1.25 for f in (np.cos, np.sin))
        for a, b in ((q, got[0]), (k, got[1])):
            y, b = a.cpu().double(), b.cpu().double()
            i = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
            want, size = y.clone(), torch.zeros_like(y)
            want[..., i[0]], want[..., i[1]] = y[..., i[0]] * c - y[..., i[1]] * s, y[..., i[0]] * s + y[..., i[1]] * c
            size[..., i[0]] = size[..., i[1]] = (y[..., i[0]].abs() + y[..., i[1]].abs()) * 1.25
            if tokens > 4:
                assert bool((b[3] == 7).all())  # of no sequence
                want[3], size[3] = 7.0, 0.0
            bound = torch.finfo(dtype).eps / 2 * want.abs() + 6 * 2.0 ** -24 * size * (1 + torch.finfo(dtype).eps)
            assert bool(((b - want).abs() <= bound).all()), float(((b - want).abs() - bound).max())
        # in place, and one of the two
        qq, kk = q.clone(), x.clone()
        cuda.tq_rotary(pos, dev(w, torch.float64), qq, kk[:, QH:QH + H], interleaved=interleaved, scale=1.25, q_out=qq, k_out=kk[:, QH:QH + H])
        live = pos >= 0
        assert torch.equal(qq[live], got[0][live]) and torch.equal(kk[:, QH:QH + H][live], got[1][live])
        assert torch.equal(qq[~live], q[~live]) and torch.equal(kk[:, :QH], x[:, :QH])
        none, only = cuda.tq_rotary(pos, dev(w, torch.float64), None, k, interleaved=interleaved, scale=1.25)
        assert none is None and torch.equal(only[live], got[1][live])


def test_rotary_by_zero_and_heads_before_tokens(cuda):
    """Position 0 leaves the vectors as they are; [heads][tokens][d] storage."""
    x = torch.randn(8, 50, 128, device="cuda").bfloat16().transpose(0, 1)
    w = dev(cuda.tq_rotary_frequencies(128)[0], torch.float64)
    out, _ = cuda.tq_rotary(torch.zeros(50, dtype=torch.int32, device="cuda"), w, x)
    assert torch.equal(out, x)
    pos = torch.arange(50, device="cuda", dtype=torch.int32)
    assert torch.equal(cuda.tq_rotary(pos, w, x)[0], cuda.tq_rotary(pos, w, x.contiguous())[0])
    empty, _ = cuda.tq_rotary(pos[:0], w, x[:0])
    assert empty.shape == (0, 8, 128)


# ------------------------------------------------------------------ verification
def verify64(parents, tokens, p, r, u, last):
    """One sequence, by the definition: (path, next)."""
    clean = lambda x: np.where(np.isfinite(x) & (x > 0), x, 0.0).astype(np.float64)  # noqa: E731
    n, V = p.shape
    if n == 0:
        return [], -1
    path, gone, C, M = [0], [], 0.0, 1.0

    def left():
        x = clean(p[path[-1]])
        if r is not None:
            return np.maximum(x - C * clean(r[path[-1]]), 0.0)
        x[gone] = 0.0
        return x

    while True:
        for c in range(path[-1] + 1, n):
            if parents[c] != path[-1] or not 0 <= tokens[c] < V:
                continue
            x = tokens[c]
            if np.float64(u[c]) * (clean(r[path[-1]])[x] if r is not None else 1.0) * M < left()[x]:
                path.append(c)
                gone, C, M = [], 0.0, 1.0
                break
            if r is not None:
                C += M
                M = left().sum()
            else:
                M -= left()[x]
                gone.append(x)
        else:
            break
    s = np.cumsum(left())
    return path, int((s <= np.float64(last) * s[-1]).sum())


def check_verify(tq, news, V, draft, dtype=torch.float32, seed=0, pad=0, stride=0, edit=None, sharp=2.0):
    rng = np.random.default_rng(seed)
    total = sum(news) + pad
    x = sharp * rng.standard_normal((total, V))
    soft = lambda z: np.exp(z - z.max(-1, keepdims=True)) / np.exp(z - z.max(-1, keepdims=True)).sum(-1, keepdims=True)  # noqa: E731
    p, r = soft(x), soft(x + 0.7 * rng.standard_normal((total, V)))

    def rows(a):
        wide = torch.full((total, V + stride), float("nan"), dtype=dtype, device="cuda")
        wide[:, stride // 2:stride // 2 + V] = torch.from_numpy(a).to(dtype)
        return wide[:, stride // 2:stride // 2 + V]

    parents = [random_parents(rng, n) for n in news]
    starts = np.cumsum([0] + list(news))
    tokens = np.zeros(total, np.int64)
    for s, t in enumerate(parents):
        for i, up in enumerate(t):
            tokens[starts[s] + i] = rng.choice(V, p=r[starts[s] + max(up, 0)])
    u, last = rng.random(total, dtype=np.float32), rng.random(len(news), dtype=np.float32)
    if edit:
        edit(p, r, tokens, parents, u, last, starts)
    pt, rt = rows(p), rows(r) if draft else None
    flat = [a for t in parents for a in t] + [0] * pad
    path, kept, nxt = tq.tq_verify_drafts(dev(starts), dev(flat), dev(tokens), pt, rt, dev(u, torch.float32), dev(last, torch.float32),
                                          max(max(news), 1))
    p64 = pt.float().cpu().numpy()
    r64 = rt.float().cpu().numpy() if draft else None
    for s, n in enumerate(news):
        at = slice(starts[s], starts[s] + n)
        way, token = verify64(parents[s], tokens[at], p64[at], r64[at] if draft else None, u[at], last[s])
        assert int(kept[s]) == len(way) and path[s].tolist() == way + [-1] * (path.shape[1] - len(way)), s
        assert int(nxt[s]) == token, (s, int(nxt[s]), token)
    return kept


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("V", [1, 2, 3, 7, 8, 31, 33, 127, 128, 129, 1000, 4099, 32000, 70001])
def test_verify(cuda, V, draft, dtype):
    news = [5, 1, 0, 12, 33, 2] if V < 5000 else [4, 1, 9]
    kept = check_verify(cuda, news, V, draft, dtype, seed=V)
    check_verify(cuda, news, V, draft, dtype, seed=V + 1, pad=3, stride=3)  # rows at odd offsets
    assert cuda.tq_device_error() == 0
    if V >= 128 and draft:
        assert int(kept.max()) > 1  # some drafts are accepted (fixed ones of so many tokens are hardly ever)


@pytest.mark.parametrize("draft", [True, False])
def test_verify_edges(cuda, draft):
    """Rows of one token, of nothing, with NaN, infinities and negative entries; numbers of 0 and just below 1; many
    rejections at one node; the same token twice."""
    def one(p, r, tokens, parents, u, last, starts):
        p[:] = 0.0
        p[:, 5] = 1.0
        r[:] = 0.0
        r[:, 5] = 1.0
        tokens[:] = 5

    def nothing(p, r, tokens, parents, u, last, starts):
        p[:] = 0.0

    def dirt(p, r, tokens, parents, u, last, starts):
        p[:, 3], p[:, 9], p[:, 11] = np.nan, np.inf, -1.0
        r[:, 3], r[:, 7], r[:, 12] = 0.2, np.nan, np.inf
        tokens[::3] = 3

    def ends(p, r, tokens, parents, u, last, starts):
        u[::2], u[1::2] = 0.0, np.float32(1) - np.float32(2.0 ** -24)
        last[::2], last[1::2] = 0.0, np.float32(1) - np.float32(2.0 ** -24)

    def star(p, r, tokens, parents, u, last, starts):
        for t in parents:
            t[1:] = [0] * (len(t) - 1)
        u[:] = 0.999

    def twice(p, r, tokens, parents, u, last, starts):
        star(p, r, tokens, parents, u, last, starts)
        tokens[:] = tokens[0]

    def all_of_it(p, r, tokens, parents, u, last, starts):
        star(p, r, tokens, parents, u, last, starts)
        tokens[:] = np.arange(len(tokens)) % p.shape[1]

    for edit in (one, nothing, dirt, ends, star, twice, all_of_it):
        for V in (40, 600):
            check_verify(cuda, [20, 3, 1, 8, 70], V, draft, edit=edit, seed=V)
    assert cuda.tq_device_error() == 0


def test_verify_bad_trees(cuda):
    """A parent or a token out of range keeps its node, and those behind it, from being reached."""
    V = 50
    p = torch.full((8, V), 1.0 / V, device="cuda")
    args = lambda parents, tokens, starts: (dev(starts), dev(parents), dev(tokens), p, None, torch.zeros(8, device="cuda"),  # noqa: E731
                                            torch.zeros(2, device="cuda"), 6)
    path, kept, nxt = cuda.tq_verify_drafts(*args([-1, 3, 1, 0, 3, 4, -1, 0], [0, 1, 2, -5, 1, 2, 0, V], [0, 6, 8]))
    assert cuda.tq_device_error() == cuda.TQ_DEVICE_ERR_TREE
    assert kept.tolist() == [1, 1] and nxt.tolist() == [0, 0] and path[:, 1:].eq(-1).all()
    path, kept, nxt = cuda.tq_verify_drafts(*args([-1] + [0] * 7, [1] * 8, [0, 7, 8]))  # seven tokens, of six
    assert cuda.tq_device_error() == cuda.TQ_DEVICE_ERR_LENGTH | cuda.TQ_DEVICE_ERR_TREE  # (the second one's root is its own parent)
    assert kept.tolist() == [0, 1] and nxt.tolist() == [-1, 0] and path[0].eq(-1).all()


def test_verify_follows_the_target(cuda):
    """Drafts and random numbers of many sequences: the first token behind node 0 comes out as the target has it, whatever
    the draft's distribution (each count within 5.5 standard deviations; 8 x 2 counts)."""
    S, V = 40000, 4
    g = torch.Generator(device="cuda").manual_seed(11)
    p = torch.tensor([0.45, 0.3, 0.2, 0.05], device="cuda")
    r = torch.tensor([0.1, 0.25, 0.25, 0.4], device="cuda")
    for draft in (True, False):
        # two children of node 0 each: drawn from r, or two fixed tokens
        kids = torch.multinomial(r.expand(S, V), 2, replacement=True, generator=g) if draft else torch.tensor([[3, 1]], device="cuda").expand(S, 2)
        tokens = torch.cat([torch.zeros(S, 1, device="cuda", dtype=torch.long), kids], 1).to(torch.int32)
        parents = torch.tensor([[-1, 0, 0]], device="cuda", dtype=torch.int32).expand(S, 3).contiguous()
        rows = lambda x: x.expand(3 * S, V).contiguous()  # noqa: E731
        path, kept, nxt = cuda.tq_verify_drafts(torch.arange(0, 3 * S + 1, 3, device="cuda", dtype=torch.int32), parents.flatten(), tokens.flatten(),
                                                rows(p), rows(r) if draft else None, torch.rand(3 * S, generator=g, device="cuda"),
                                                torch.rand(S, generator=g, device="cuda"), 3)
        first = torch.where(kept > 1, tokens.gather(1, path[:, 1:2].long().clamp(min=0))[:, 0], nxt)
        counts = torch.bincount(first.long(), minlength=V).double().cpu()
        want = p.double().cpu() * S
        assert bool(((counts - want).abs() <= 5.5 * (want * (1 - p.double().cpu())).sqrt()).all()), (counts, want)


# ------------------------------------------------------------------ kept rows
@pytest.mark.parametrize("d,kb,vb,page", [(128, 8, 3, 64), (64, 2, 3, 16), (64, 4, 5, 48), (256, 5, 2, 32), (512, 8, 8, 16), (128, 4, 4, 256)])
def test_keep(cuda, d, kb, vb, page):
    """Paths of every kind: none, all, a few far apart, long ones whose rows overlap; other rows stay as they are."""
    rng = np.random.default_rng(d + kb)
    new = [1, 9, 40, 150, 7, 0, 33, 5, 64]
    lens = [1, 9, 60, 400, 7, 20, 100, 300, 64]
    b = Batch(lens, new, H=3, d=d, kb=kb, vb=vb, page=page)
    pool = b.pool(cuda)
    for t in pool.planes():
        t.copy_(torch.randint(0, 100, t.shape, device="cuda", dtype=torch.int32).to(t.dtype))
    paths = [[0], [0, 2, 4, 8], list(range(1, 40)), sorted(rng.choice(150, 100, replace=False).tolist()), [], [],
             sorted(rng.choice(33, 20, replace=False).tolist()), list(range(5)), list(range(0, 64, 2))]
    path = np.full((len(lens), 150), -1)
    for s, p in enumerate(paths):
        path[s, :len(p)] = p
    before = [rows_of(pool, b.table[s], n) for s, n in enumerate(lens)]
    others = [t.clone() for t in pool.planes()]
    table = b.pages(cuda)
    left = cuda.tq_paged_keep(pool, table, b.dev(b.starts), dev(path), dev([len(p) for p in paths]))
    assert cuda.tq_device_error() == 0
    assert left.tolist() == [n - m + len(p) for n, m, p in zip(lens, new, paths)]
    assert table.seq_lens.tolist() == lens
    moved = torch.zeros(b.num_pages, page, dtype=torch.bool)
    for s, (n, m, p) in enumerate(zip(lens, new, paths)):
        for got, was in zip(rows_of(pool, b.table[s], n), before[s]):
            want = was.copy()
            for k, i in enumerate(p):
                want[:, n - m + k] = was[:, n - m + i]
                moved[int(b.table[s, (n - m + k) // page]), (n - m + k) % page] = True
            assert np.array_equal(got, want), s
    for t, was in zip(pool.planes(), others):
        assert torch.equal(t.transpose(1, 2)[~moved.cuda()], was.transpose(1, 2)[~moved.cuda()])


def test_keep_refuses_bad_paths(cuda):
    b = Batch([20, 20, 20, 20, 20, 8], [5] * 6, H=2, d=64, kb=4, vb=3, page=16)
    pool = b.pool(cuda)
    b.fill(cuda, pool)
    was = [t.clone() for t in pool.planes()]
    path = dev([[0, 0, 1, -1, -1], [0, 5, -1, -1, -1], [2, 1, -1, -1, -1], [-1, 1, -1, -1, -1], [0, 1, 2, 3, 4], [0, 1, 2, 3, 4]])
    left = cuda.tq_paged_keep(pool, b.pages(cuda), b.dev(b.starts), path, dev([3, 2, 2, 2, 6, -1]))
    assert cuda.tq_device_error() == cuda.TQ_DEVICE_ERR_TREE
    assert left.tolist() == b.lens and all(torch.equal(x, y) for x, y in zip(pool.planes(), was))


# ------------------------------------------------------------------ a step of all of them
class Server:
    """A batch that drafts trees step after step: the tensors of a step are the same ones every time, so that a step can
    be captured once and replayed."""

    def __init__(self, tq, seqs=6, nodes=7, H=2, G=4, d=128, V=300, page=16, pages=64, seed=0):
        self.tq, self.S, self.N, self.V = tq, seqs, nodes, V
        rng = np.random.default_rng(seed)
        self.pool = tq.Cache(pages, H, d, page, k_bits=8, v_bits=3)
        self.table = tq.PageTable(torch.full((seqs, 12), -1, dtype=torch.int32, device="cuda"),
                                  torch.zeros(seqs, dtype=torch.int32, device="cuda"), 12 * page)
        self.free, self.count = dev(rng.permutation(pages)), dev([pages])
        self.lens, self.new = dev([0] * seqs), dev([0] * seqs)
        self.total = seqs * nodes  # (a batch padded to its largest size)
        t = self.total
        self.starts, self.left = dev([0] * (seqs + 1)), dev([0] * seqs)
        self.parents, self.tokens = dev([-1] * t), dev([0] * t)
        bf = lambda *s: torch.zeros(*s, device="cuda", dtype=torch.bfloat16)  # noqa: E731
        self.q, self.k, self.v = bf(t, H * G, d), bf(t, H, d), bf(t, H, d)
        self.u, self.last = torch.zeros(t, device="cuda"), torch.zeros(seqs, device="cuda")
        self.target, self.draft = (torch.zeros(t, V, device="cuda") for _ in range(2))
        self.freqs = dev(tq.tq_rotary_frequencies(d)[0], torch.float64)
        self.out = {}

    def step(self):
        tq, o = self.tq, self.out
        tq.tq_page_table_update(self.pool, self.table, self.lens, self.free, self.count, new_tokens=self.new, starts=self.starts)
        o["pos"], o["slots"], o["masks"] = tq.tq_paged_layout(self.pool, self.table, self.starts, self.total, parents=self.parents,
                                                              max_new=self.N)
        o["q"], o["k"] = tq.tq_rotary(o["pos"], self.freqs, self.q, self.k)
        tq.tq_paged_append(self.pool, self.table, self.starts, o["k"], self.v)
        o["att"] = tq.tq_paged_tree_attention(self.pool, self.table, self.starts, o["q"], o["masks"], self.N)
        o["path"], o["kept"], o["next"] = tq.tq_verify_drafts(self.starts, self.parents, self.tokens, self.target, self.draft, self.u,
                                                              self.last, self.N)
        tq.tq_paged_keep(self.pool, self.table, self.starts, o["path"], o["kept"], lens_out=self.left, total=self.total)
        # rejected rows' pages go back at once
        tq.tq_page_table_update(self.pool, self.table, self.left, self.free, self.count)


@pytest.mark.parametrize("captured", [False, True])
def test_a_step_of_drafted_tokens(cuda, captured):
    """Tables, positions, rotary, append, tree attention, verification and kept rows, step after step, some sequences
    ending and others beginning: what the cache holds is what appending the accepted tokens alone would have left."""
    rng = np.random.default_rng(7)
    sv = Server(cuda)
    S, N, V, d = sv.S, sv.N, sv.V, 128
    accepted = [[] for _ in range(S)]  # (position, k, v) of every kept row
    graph = None
    for step in range(9):
        have = [len(a) for a in accepted]
        new = [0 if step % 4 == s % 4 == 3 else int(rng.integers(1, N + 1)) for s in range(S)]
        for s in range(S):
            if have[s] > 30:  # ends; its row of the table begins a new sequence
                accepted[s], have[s] = [], 0
        ended = [n == 0 for n in have]
        if any(ended) and step:
            sv.lens.copy_(dev(have))  # shorter, and the rest as they are
            cuda.tq_page_table_update(sv.pool, sv.table, sv.lens, sv.free, sv.count)
        starts = np.cumsum([0] + new)
        parents = [random_parents(rng, n, wide=2) for n in new]
        flat = np.full(sv.total, -1)
        flat[:starts[-1]] = [p for t in parents for p in t]
        sv.lens.copy_(dev([a + b for a, b in zip(have, new)]))
        sv.new.copy_(dev(new))
        sv.parents.copy_(dev(flat))
        for t in (sv.q, sv.k, sv.v):
            t.copy_(torch.from_numpy(rng.standard_normal(tuple(t.shape), dtype=np.float32)))
        x = 1.5 * rng.standard_normal((sv.total, V))
        soft = lambda z: (np.exp(z) / np.exp(z).sum(-1, keepdims=True)).astype(np.float32)  # noqa: E731
        p, r = soft(x), soft(x + 0.5 * rng.standard_normal(x.shape))
        tokens = np.array([rng.choice(V, p=r[i].astype(np.float64) / r[i].astype(np.float64).sum()) for i in range(sv.total)])
        u, last = rng.random(sv.total, dtype=np.float32), rng.random(S, dtype=np.float32)
        sv.target.copy_(torch.from_numpy(p))
        sv.draft.copy_(torch.from_numpy(r))
        sv.tokens.copy_(dev(tokens))
        sv.u.copy_(torch.from_numpy(u))
        sv.last.copy_(torch.from_numpy(last))
        if not captured:
            sv.step()
        elif graph is None:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                sv.step()
            graph.replay()
        else:
            graph.replay()
        assert cuda.tq_device_error() == 0
        o = {k: t.cpu() for k, t in sv.out.items()}
        table = sv.table.pages.cpu().numpy()
        at = 0
        for s, n in enumerate(new):
            up = ancestors(parents[s])
            for i in range(n):
                assert int(o["pos"][at + i]) == have[s] + len(up[i]) - 1
            way, token = verify64(parents[s], tokens[at:at + n], p[at:at + n], r[at:at + n], u[at:at + n], last[s])
            assert o["path"][s].tolist()[:len(way)] == way and int(o["kept"][s]) == len(way) and int(o["next"][s]) == token
            accepted[s] += [(o["k"][at + i], sv.v[at + i].cpu()) for i in way]
            at += n
        assert sv.table.seq_lens.tolist() == [len(a) for a in accepted]
        used = sum(-(-len(a) // 16) for a in accepted)
        assert int(sv.count) == 64 - used  # every page is accounted for
        held = [int(x) for s, a in enumerate(accepted) for x in table[s, :-(-len(a) // 16)]] + sv.free[:int(sv.count)].tolist()
        assert sorted(held) == list(range(64))
        for s, a in enumerate(accepted):  # the rows are those of an append of the accepted tokens alone
            if not a:
                continue
            c = cuda.Cache(1, 2, d, len(a), k_bits=8, v_bits=3)
            k, v = (torch.stack([y[i] for y in a], 1)[None].cuda() for i in (0, 1))
            cuda.tq_encode_append(c, k, v, 0)
            for got, ref in zip(rows_of(sv.pool, table[s], len(a)), c.planes()):
                assert np.array_equal(got, ref[0, :, :len(a)].cpu().numpy()), (step, s)
    assert max(len(a) for a in accepted) > 8


def test_tree_attention_of_the_step_matches_its_branches(cuda):
    """Every path from the root to a node, appended alone to a copy of the cache, gives the node the same attention."""
    b = Batch([90], [8], H=2, d=128, kb=8, vb=3, page=16)
    parents = [-1, 0, 0, 1, 1, 2, 3, 5]
    seen = [np.zeros((8, 8), bool)]
    for i, up in enumerate(ancestors(parents)):
        seen[0][i, up] = True
    pool, q, out = run_tree(cuda, b, 8, seen)
    for i, up in enumerate(ancestors(parents)):
        up = up[::-1]
        alone = Batch([82 + len(up)], [len(up)], H=2, d=128, kb=8, vb=3, page=16)
        rows = list(range(82)) + [82 + j for j in up]
        alone.k, alone.v = [b.k[0][rows]], [b.v[0][rows]]
        p2 = alone.pool(cuda)
        alone.fill(cuda, p2)
        causal = cuda.tq_paged_attention(p2, alone.pages(cuda), alone.dev(alone.starts), q[up].contiguous().cuda(), len(up))
        err = (out[i].double() - causal[-1].double()).abs() - 2 * RTOL * causal[-1].double().abs()
        assert float(err.max()) <= 2 * ATOL


def test_two_graphs_of_trees_with_workspaces_of_their_own(cuda):
    """Captured calls on two streams, replayed together, each with its own workspace."""
    runs = []
    for seed in (1, 2):
        b = Batch([900, 40, 300], [6, 40, 20], H=2, d=128, kb=8, vb=3, page=32, seed=seed)
        seen = tree_masks(b, "tree", seed)
        pool, q, want = run_tree(cuda, b, 16, seen)
        masks = dev(np.concatenate([pack(np.pad(m, ((0, 0), (0, 64 - len(m)))), 2) for m in seen]))
        need = cuda.tq_paged_tree_attention_workspace_bytes(pool, b.pages(cuda), 16, b.total, 40)
        runs.append((b, pool, b.pages(cuda), b.dev(b.starts), q.cuda(), masks, torch.empty(need, dtype=torch.uint8, device="cuda"), want,
                     torch.empty_like(want)))
    torch.cuda.synchronize()
    graphs = []
    for b, pool, pages, starts, q, masks, ws, _, out in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(4):
                cuda.tq_paged_tree_attention(pool, pages, starts, q, masks, 40, out=out, workspace=ws)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for *_, want, out in runs:
        assert torch.equal(out, want)
    assert cuda.tq_device_error() == 0
