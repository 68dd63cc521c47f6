"""A step of drafted tokens at sizes and in shapes that the small tests do not reach."""
import numpy as np
import pytest
import torch

from pagedtest import ATOL, RTOL, Batch, dequantised
from test_drafts_gpu import TableModel, ancestors, check_verify, dev, pack, random_parents, tree_masks
from test_tree_ranges_gpu import check_numbers

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("wide", [1, 3, 7, 40])
def test_verify_rejects_and_accepts_in_turn(cuda, wide, draft, dtype):
    """Level after level `wide` children are rejected and the next one is accepted: what is crossed out at a node counts for
    it alone, whether its children stand among 32 nodes with others' or behind them; some rejected tokens come twice."""
    levels = 200 // (wide + 1)

    def edit(p, r, tokens, parents, u, last, starts):
        rng = np.random.default_rng(wide)
        for s, t in enumerate(parents):
            cur, j = 0, 1
            while j < len(t):
                kids = range(j, min(j + wide + 1, len(t)))
                for c in kids:
                    row, back = starts[s] + cur, c < j + wide
                    x = rng.integers(0, 40) if back else rng.integers(40, 500)
                    t[c], tokens[starts[s] + c] = cur, x
                    u[starts[s] + c] = np.float32(1) - np.float32(2.0 ** -24) if back else 0.0
                    if draft:  # (without draft probabilities the number alone rejects: no token has all of the probability)
                        r[row, x] = r[row, x] if back else 0.0
                        p[row, x] = r[row, x] / 2 if back else p[row, x]
                cur, j = kids[-1], j + wide + 1

    kept = check_verify(cuda, [1 + levels * (wide + 1), 33, 65, 2], 500, draft, dtype, seed=wide, edit=edit)
    assert int(kept[0]) == 1 + levels
    assert cuda.tq_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("draft", [True, False])
def test_verify_of_a_large_vocabulary(cuda, draft, dtype):
    check_verify(cuda, [5, 1, 9, 0, 2], 131072, draft, dtype, seed=3)
    check_verify(cuda, [4, 7], 150001, draft, dtype, seed=4, pad=1, stride=5)  # rows at odd offsets
    assert cuda.tq_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,d,rot,QH,H", [(4097, 128, 128, 5, 1), (4098, 128, 64, 8, 2), (4099, 64, 64, 3, 3), (5000, 256, 192, 2, 1),
                                               (4097, 512, 512, 1, 1), (4097, 128, 36, 3, 1)])
def test_rotary_of_many_tokens(cuda, tokens, d, rot, QH, H, interleaved, dtype):
    """Several tokens a block, the last block's short; positions below 0 among them.  Bounds as in test_rotary: 6 steps of
    2^-24 of (|a| + |b|) scale, then one rounding of the type."""
    assert tokens >= 16 * torch.cuda.get_device_properties(0).multi_processor_count
    g = torch.Generator(device="cuda").manual_seed(tokens + rot)
    x = torch.randn(tokens, QH + H, d, generator=g, device="cuda").to(dtype)
    q, k = x[:, :QH], x[:, QH:]
    pos = torch.randint(0, 1 << 20, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    pos[[0, 6, tokens // 2, tokens - 2]] = -1
    live = pos >= 0
    w = dev(cuda.tq_rotary_frequencies(rot)[0], torch.float64)
    outs = [torch.full(t.shape, 7.0, dtype=dtype, device="cuda") for t in (q, k)]
    cuda.tq_rotary(pos, w, q, k, interleaved=interleaved, scale=0.75, q_out=outs[0], k_out=outs[1])
    t = pos.double()[:, None] * w
    c, s = torch.cos(t)[:, None] * 0.75, torch.sin(t)[:, None] * 0.75
    i = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    for a, b in ((q, outs[0]), (k, outs[1])):
        y, want = a.double(), a.double()
        size = torch.zeros_like(y)
        want[..., i[0]], want[..., i[1]] = y[..., i[0]] * c - y[..., i[1]] * s, y[..., i[0]] * s + y[..., i[1]] * c
        size[..., i[0]] = size[..., i[1]] = (y[..., i[0]].abs() + y[..., i[1]].abs()) * 0.75
        bound = torch.finfo(dtype).eps / 2 * want.abs() + 6 * 2.0 ** -24 * size * (1 + torch.finfo(dtype).eps)
        assert bool(((b.double() - want).abs() <= bound)[live].all())
        assert bool((b[~live] == 7).all())
    # in place, both in one tensor
    y = x.clone()
    cuda.tq_rotary(pos, w, y[:, :QH], y[:, QH:], interleaved=interleaved, scale=0.75, q_out=y[:, :QH], k_out=y[:, QH:])
    assert torch.equal(y[live], torch.cat(outs, 1)[live]) and torch.equal(y[~live], x[~live])


@pytest.mark.parametrize("seqs,moving", [(1, 1), (5, 3), (40, 40), (1030, 7)])
def test_long_moves_of_pages(cuda, seqs, moving):
    """Sequences that gain or give back up to a thousand pages in a call, while others grow by a row."""
    rng = np.random.default_rng(seqs)
    page, width = 16, 1100
    pages = moving * 1000 + seqs + 50
    m = TableModel(rng, seqs, width, page, pages)
    pool = cuda.Cache(pages, 1, 64, page, k_bits=2, v_bits=2)
    table = cuda.PageTable(dev(m.table), dev(m.lens), width * page)
    free, count = dev(m.free + [-7] * 3), dev([len(m.free)])
    long = rng.choice(seqs, moving, replace=False)
    for step, most in enumerate((1000, 0, 1000, 257, 1000, 258, 513, 1, 1000, 0)):
        want = [min(n + 1, 16) if s not in long else n for s, n in enumerate(m.lens)]
        for s in long:
            want[s] = most * page - (int(rng.integers(0, page)) if most else 0) if (s + step) % 3 or step < 2 else want[s]
        assert m.update(want)
        cuda.tq_page_table_update(pool, table, dev(want), free, count)
        assert cuda.tq_device_error() == 0 and table.seq_lens.tolist() == want
        assert int(count) == len(m.free) and free.tolist()[:len(m.free)] == [int(x) for x in m.free]
        at = table.pages.cpu().numpy()
        for s, n in enumerate(m.lens):
            k = -(-n // page)
            assert np.array_equal(at[s, :k], m.table[s, :k]), (step, s)
    assert free.tolist()[pages:] == [-7] * 3


@pytest.mark.parametrize("seqs,most,big", [(1023, 3, 3), (1024, 3, 3), (2500, 2, 40), (3, 40, 1500), (6, 9, 3100)])
def test_layout_of_many_sequences_and_large_trees(cuda, seqs, most, big):
    """More sequences than starts stand on the chip, trees of more nodes than parents do."""
    rng = np.random.default_rng(seqs)
    new = [int(x) for x in rng.integers(0, most + 1, seqs)]
    new[seqs // 2] = big
    lens = [n + int(x) for n, x in zip(new, rng.integers(0, 40, seqs))]
    page, width = 16, -(-max(lens) // 16)
    table = rng.permutation(seqs * width).reshape(seqs, width)
    pool = cuda.Cache(seqs * width, 1, 64, page, k_bits=2, v_bits=2)
    pages = cuda.PageTable(dev(table), dev(lens), max(lens))
    parents = [random_parents(rng, n, wide=3) for n in new]
    starts, total = np.cumsum([0] + new), sum(new)
    pos, slots, masks = cuda.tq_paged_layout(pool, pages, dev(starts), total, parents=dev([x for t in parents for x in t]), max_new=big)
    rows, line, _ = cuda.tq_paged_layout(pool, pages, dev(starts), total)
    assert cuda.tq_device_error() == 0 and torch.equal(line, slots)
    want_pos, want_row, want_slot, want_mask = [], [], [], []
    for s, n in enumerate(new):
        for i, up in enumerate(ancestors(parents[s])):
            row = lens[s] - n + i
            want_pos.append(lens[s] - n + len(up) - 1)
            want_row.append(row)
            want_slot.append(int(table[s, row // page]) * page + row % page)
            seen = np.zeros((1, big), bool)
            seen[0, up] = True
            want_mask.append(pack(seen, -(-big // 32))[0])
    assert pos.tolist() == want_pos and rows.tolist() == want_row and slots.tolist() == want_slot
    assert np.array_equal(masks.cpu().numpy(), np.stack(want_mask))


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("shape", ["chain", "star", "any"])
def test_verify_of_the_largest_trees(cuda, shape, draft):
    def edit(p, r, tokens, parents, u, last, starts):
        if shape == "any":
            return
        for s, t in enumerate(parents):
            for i in range(1, len(t)):
                t[i] = i - 1 if shape == "chain" else 0
                if shape == "chain":
                    u[starts[s] + i] = 0.0  # (accepted)

    kept = check_verify(cuda, [1024, 3, 1000], 300, draft, seed=8, edit=edit)
    assert shape != "chain" or kept.tolist()[0] > 30
    assert cuda.tq_device_error() == 0


@pytest.mark.parametrize("d,kb,vb,H,G,new", [(128, 8, 3, 2, 8, 6), (64, 4, 3, 1, 48, 5), (256, 8, 4, 4, 5, 7), (128, 4, 4, 1, 128, 1)])
def test_trees_of_many_sequences(cuda, d, kb, vb, H, G, new):
    """Seventy sequences on the kernel whose rows are dequantised on the chip, odd groups of q-heads, queries within a
    wider tensor, masks with more words than the tokens need."""
    rng = np.random.default_rng(G)
    lens = [int(x) for x in rng.integers(0, 300, 70)]
    b = Batch(lens, [min(n, int(rng.integers(0, new + 1))) for n in lens], H=H, d=d, kb=kb, vb=vb, page=48, seed=3, width=-(-4096 // 48))
    b.new[lens.index(max(lens))] = new
    b.starts = np.concatenate([[0], np.cumsum(b.new)]).astype(np.int32)
    b.total = int(b.starts[-1])
    seen = tree_masks(b, "any")
    masks = np.concatenate([pack(np.pad(m, ((0, 0), (0, 96 - m.shape[1])), constant_values=True), 3) for m in seen])
    pool = b.pool(cuda)
    b.fill(cuda, pool)
    q = b.queries(H * G)
    wide = torch.full((b.total, H * G + 3, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 2:-1] = q.cuda()
    out = cuda.tq_paged_tree_attention(pool, b.pages(cuda, max_len=4096), b.dev(b.starts), wide[:, 2:-1], dev(masks), new)
    assert cuda.tq_device_error() == 0
    check_numbers(b, pool, q, out, seen)


def test_large_trees_that_find_no_room_for_their_rows(cuda):
    """Trees of 512 columns over three sequences whose expanded rows pass what the workspace has for them (8 GiB): the last
    one's go to the kernel without.  One prefix of 512 rows, repeated; the plain implementation counts each row."""
    S, H, G, d, P, n, new = 3, 8, 8, 128, 128, 1 << 19, 64
    b = Batch([512], [0], H=H, d=d, kb=8, vb=3, page=P, spare=0, seed=6)
    pool = b.pool(cuda)
    b.fill(cuda, pool)
    lens = [n - 41 * s for s in range(S)]
    pages = cuda.PageTable(b.dev(np.tile(b.table[0, :4], (S, n // 512)).astype(np.int32)), b.dev(np.array(lens, np.int32)), n)
    need = cuda.tq_paged_tree_attention_workspace_bytes(pool, pages, H * G, S * new, new)
    assert (8 << 30) < need < S * n * H * 6 * d
    rng = np.random.default_rng(4)
    masks = rng.integers(-(1 << 31), 1 << 31, (S * new, 2)).astype(np.int32)
    q = b.queries(H * G, total=S * new)
    out = cuda.tq_paged_tree_attention(pool, pages, dev(np.arange(0, S * new + 1, new)), q.cuda(), dev(masks), new).cpu().double()
    assert cuda.tq_device_error() == 0
    torch.cuda.empty_cache()
    k, v = (torch.from_numpy(x).double() for x in dequantised(pool, b.table[0], 512))
    for s in range(S):
        before = lens[s] - new
        for i in (0, 31, new - 1):
            times = torch.tensor([(before - r + 511) // 512 for r in range(512)], dtype=torch.float64)
            for j in range(new):
                if masks[s * new + i, j // 32] >> (j % 32) & 1:
                    times[(before + j) % 512] += 1
            x = torch.einsum("hgd,hnd->hgn", q[s * new + i].double().view(H, G, d), k) * d ** -0.5
            p = torch.exp(x - x.amax(-1, keepdim=True)) * times
            want = torch.einsum("hgn,hnd->hgd", p / p.sum(-1, keepdim=True), v).reshape(H * G, d)
            assert float(((out[s * new + i] - want).abs() - RTOL * want.abs()).max()) <= ATOL, (s, i)
