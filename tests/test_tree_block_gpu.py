"""Attention of trees on the kernel whose rows are dequantised on the chip (more columns than one pass of the split kernel,
bounds of 2^20 rows x kv-heads x columns and more): its column counts, tile and slot ends, ranges and outliers."""
import numpy as np
import pytest
import torch

from pagedtest import ATOL, RTOL, Batch, dequantised, rows_of
from test_drafts_gpu import check_tree, dev, pack, tree_masks

pytestmark = pytest.mark.gpu

BOUND = 1 << 14  # rows of a sequence, as the host is told


def attend(tq, b, QH, seen, q=None, pool=None, **kw):
    if pool is None:
        pool = b.pool(tq)
        b.fill(tq, pool)
    new, words = max(b.new), -(-max(b.new) // 32)
    masks = np.concatenate([pack(np.pad(m, ((0, 0), (0, 32 * words - m.shape[1]))), words) for m in seen])
    q = b.queries(QH) if q is None else q
    out = tq.tq_paged_tree_attention(pool, b.pages(tq, max_len=BOUND), b.dev(b.starts), q.cuda(), dev(masks), new, **kw)
    return pool, q, out


def batch(lens, new, d, kb, vb, page, seed=0, H=2):
    return Batch(lens, new, H=H, d=d, kb=kb, vb=vb, page=page, seed=seed, width=-(-BOUND // page))


SHAPES = [  # head_dim, key and value bits, group, page, most new tokens
    (128, 8, 3, 8, 64, 3), (128, 4, 3, 8, 16, 4), (128, 8, 4, 8, 48, 5), (128, 4, 2, 8, 256, 8), (128, 8, 2, 4, 32, 9),
    (128, 4, 4, 1, 64, 33), (128, 8, 3, 3, 80, 43), (128, 5, 3, 8, 64, 8), (128, 8, 8, 8, 64, 16), (128, 2, 5, 8, 16, 40),
    (128, 8, 3, 8, 128, 48), (64, 8, 3, 8, 64, 3), (64, 4, 4, 16, 32, 4), (64, 8, 2, 8, 16, 8), (64, 4, 3, 5, 48, 25),
    (64, 8, 4, 12, 64, 21), (64, 2, 2, 8, 64, 9), (64, 8, 3, 8, 64, 48), (256, 8, 4, 4, 64, 3), (256, 4, 3, 8, 16, 4),
    (256, 8, 2, 8, 48, 5), (256, 4, 4, 4, 128, 17), (256, 8, 3, 8, 32, 33), (256, 5, 8, 4, 64, 12), (256, 8, 4, 16, 64, 40),
]


@pytest.mark.parametrize("kind", ["tree", "any"])
@pytest.mark.parametrize("d,kb,vb,G,page,new", SHAPES)
def test_shapes(cuda, d, kb, vb, G, page, new, kind):
    """Up to `new` tokens a sequence, lengths around tiles of 64 and 128 rows, one sequence with more segments than one."""
    lens = [new, new + 1, 63 + new, 64, 128, 129, 0, 127 + new, 1500, 256, 2]
    b = batch(lens, [min(n, 1 + (i * 5 + new) % new) if i else new for i, n in enumerate(lens)], d, kb, vb, page, seed=new)
    seen = tree_masks(b, kind)
    pool, q, out = attend(cuda, b, 2 * G, seen)
    check_tree(b, pool, q, out, seen)
    assert cuda.tq_device_error() == 0


@pytest.mark.parametrize("d,kb,vb,G,new", [(128, 8, 3, 8, 4), (128, 4, 4, 8, 14), (64, 8, 3, 8, 20), (256, 4, 3, 4, 11), (128, 5, 5, 8, 8)])
def test_long_runs(cuda, d, kb, vb, G, new):
    """One prefix of 512 rows repeated up to 131072: runs of more tiles than stay in one accumulator, on every CTA.  The
    plain implementation counts each row of the prefix as often as it is seen."""
    S, H, P, n = 8, 8, 128, 131072
    b = Batch([512], [0], H=H, d=d, kb=kb, vb=vb, page=P, spare=0, seed=5)
    pool = b.pool(cuda)
    b.fill(cuda, pool)
    lens = [n - 37 * s for s in range(S)]
    pages = cuda.PageTable(b.dev(np.tile(b.table[0, :4], (S, n // 512)).astype(np.int32)), b.dev(np.array(lens, np.int32)), n)
    rng = np.random.default_rng(3)
    masks = rng.integers(0, 1 << 20, (S * new, 1)).astype(np.int32)
    q = b.queries(H * G, total=S * new)
    starts = b.dev(np.arange(0, S * new + 1, new).astype(np.int32))
    out = cuda.tq_paged_tree_attention(pool, pages, starts, q.cuda(), dev(masks), new).cpu().double()
    assert cuda.tq_device_error() == 0
    k, v = (torch.from_numpy(x).double() for x in dequantised(pool, b.table[0], 512))
    worst = 0.0
    for s in range(S):
        before = lens[s] - new
        for i in (0, new - 1):
            times = torch.tensor([(before - r + 511) // 512 for r in range(512)], dtype=torch.float64)
            for j in range(new):
                if masks[s * new + i, 0] >> j & 1:
                    times[(before + j) % 512] += 1
            x = torch.einsum("hgd,hnd->hgn", q[s * new + i].double().view(H, G, d), k) * d ** -0.5
            p = torch.exp(x - x.amax(-1, keepdim=True)) * times
            want = torch.einsum("hgn,hnd->hgd", p / p.sum(-1, keepdim=True), v).reshape(H * G, d)
            worst = max(worst, float(((out[s * new + i] - want).abs() - RTOL * want.abs()).max()))
    assert worst <= ATOL, worst


@pytest.mark.parametrize("power", [0, 26, 116])
@pytest.mark.parametrize("d,kb,G", [(128, 8, 8), (64, 4, 8), (256, 8, 4), (128, 5, 8)])
def test_queries_of_any_size(cuda, d, kb, G, power):
    """Finite scores of any size: with rows whose scores differ by more than what fp32 leaves of them, the weights are
    those of the ordinary query's largest score.  (Queries along one key each, of integers that the codes hold.)"""
    new = 9
    b = batch([400, 90], [new, new], d, kb, 3, 64, seed=4)
    for s in range(2):
        for t in range(len(b.k[s])):
            b.k[s][t] = 0.0
            b.k[s][t, :, 32 * (t % (d // 32)):32 * (t % (d // 32)) + 32] = torch.where(torch.arange(32) % 2 == 0, 1.0, -1.0) * (1 + t % 3)
    q = torch.zeros(2 * new, 2 * G, d)
    q[:, :, 0:32] = torch.where(torch.arange(32) % 2 == 0, 1.0, -1.0) * 4.0
    q = (q * 2.0 ** power).to(torch.bfloat16)
    seen = tree_masks(b, "tree")
    pool, _, out = attend(cuda, b, 2 * G, seen, q=q)
    assert cuda.tq_device_error() == 0
    # scores are 128 x 2^power / sqrt(d) x 1, 2, 3 or 0: the rows of the largest share the weight from power 26 on
    check_tree(b, pool, q, out, seen)


@pytest.mark.parametrize("d,kb,vb,G,new", [(128, 8, 3, 8, 9), (128, 4, 3, 8, 16), (64, 8, 4, 8, 9), (256, 8, 3, 4, 20), (128, 2, 5, 8, 9)])
def test_far_outliers(cuda, d, kb, vb, G, new):
    """Rows with keys of up to 2^20 that all queries point away from: no weight of theirs is left, and the other rows of
    their tile keep their precision; rows with values of 2^-14 beside them, and groups far from zero."""
    b = batch([new + 400, 200], [new, new], d, kb, vb, 64, seed=9)
    way = np.where(np.arange(d) % 2, 1.0, -1.0).astype(np.float32)
    q = b.queries(2 * G).float()
    q = q + torch.from_numpy(way) * (4.0 - (q * torch.from_numpy(way)).mean(-1, keepdim=True))
    q = q.to(torch.bfloat16)
    for s in range(2):
        for t, size in ((3, 2.0 ** 20), (64, 2.0 ** 14), (150, 2.0 ** 18)):
            b.k[s][t] = (torch.from_numpy(-size * way) * (1 + 0.25 * torch.rand(2, 1))).to(torch.bfloat16)
        b.v[s][8:16] = b.v[s][8:16] * 2.0 ** -14
        b.k[s][20:24, :, 32:64] = (2.0 + 2.0 ** -7 * torch.rand(4, 2, 32)).to(torch.bfloat16)  # zero points in the hundreds
    seen = tree_masks(b, "tree")
    pool, _, out = attend(cuda, b, 2 * G, seen, q=q)
    check_tree(b, pool, q, out, seen)
    assert cuda.tq_device_error() == 0


@pytest.mark.parametrize("d,kb,G,new", [(128, 8, 8, 9), (64, 4, 8, 30), (256, 4, 4, 20), (128, 5, 8, 12), (128, 8, 8, 4)])
def test_hidden_rows_hold_anything(cuda, d, kb, G, new):
    """NaN, infinities and the largest finite scales in new rows that a token does not see never reach it; one that sees
    a value row that is not finite gets what is not finite; one that sees nothing gives zeros."""
    b = batch([300, new], [new, new], d, kb, 3, 32)
    pool = b.pool(cuda)
    b.fill(cuda, pool)
    bad = {1: 0x7E00, new - 1: 0x7C00, 2: 0x7BFF}
    seen = [np.zeros((n, n), bool) for n in b.new]
    for m in seen:
        for i in range(len(m)):
            m[i, [j for j in range(len(m)) if j not in bad and (j + i) % 3 == 0]] = True
    seen[1][0] = False
    for s, n in enumerate(b.lens):
        for j, x in bad.items():
            row = n - new + j
            for t in (pool.k_scale, pool.k_zero, pool.v_scale):
                t[int(b.table[s, row // 32]), :, int(row % 32)] = x
    _, q, out = attend(cuda, b, 2 * G, seen, pool=pool)
    assert bool(torch.isfinite(out).all()) and bool((out[b.starts[1]] == 0).all())
    check_tree(b, pool, q, out, seen)
    # the same rows' values alone, seen by some
    page, slot = b.table[0, (300 - new + 1) // 32], (300 - new + 1) % 32
    pool.k_scale[int(page), :, int(slot)] = pool.k_scale[int(b.table[0, 0]), :, 0]
    pool.k_zero[int(page), :, int(slot)] = 0
    seen[0][0, 1] = True
    _, q, out = attend(cuda, b, 2 * G, seen, pool=pool)
    assert not bool(torch.isfinite(out[0]).any()) and bool(torch.isfinite(out[1:]).all())
    assert cuda.tq_device_error() == 0


def test_bad_pages_and_lengths_are_reported(cuda):
    b = batch([300, 500], [9, 9], 128, 8, 3, 64)
    seen = tree_masks(b, "tree")
    pool, q, want = attend(cuda, b, 16, seen)
    good = b.table.copy()
    b.table[0, 2] = b.num_pages
    _, _, out = attend(cuda, b, 16, seen, pool=pool)
    assert cuda.tq_device_error() == cuda.TQ_DEVICE_ERR_PAGE
    assert torch.equal(out[9:], want[9:])  # the other sequence's results
    b.table = good
    out = torch.full_like(want, 7.0)
    masks = dev(np.concatenate([pack(np.pad(m, ((0, 0), (0, 23))), 1) for m in seen]))
    cuda.tq_paged_tree_attention(pool, b.pages(cuda, lens=[300, BOUND + 1], max_len=BOUND), b.dev(b.starts), q.cuda(), masks, 8, out=out)
    assert cuda.tq_device_error() & cuda.TQ_DEVICE_ERR_LENGTH
    assert bool((out == 7).all())  # nine new tokens, eight of which the call was told of


def test_negative_scale_and_two_streams(cuda):
    b = batch([700, 64, 1000], [6, 20, 13], 128, 8, 3, 64, seed=2)
    seen = tree_masks(b, "any")
    pool, q, out = attend(cuda, b, 16, seen, softmax_scale=-0.07)
    at = 0
    for s, (n, m) in enumerate(zip(b.lens, b.new)):
        k, v = dequantised(pool, b.table[s], n)
        vis = torch.ones(m, n, dtype=torch.bool)
        vis[:, n - m:] = torch.from_numpy(seen[s])
        x = torch.einsum("mhgd,hnd->hmgn", q[at:at + m].double().view(m, 2, 8, 128), torch.from_numpy(k).double()) * -0.07
        p = torch.softmax(x.masked_fill(~vis[None, :, None], -float("inf")), -1)
        want = torch.einsum("hmgn,hnd->hmgd", p, torch.from_numpy(v).double()).permute(1, 0, 2, 3).reshape(m, 16, 128)
        assert float(((out[at:at + m].cpu().double() - want).abs() - RTOL * want.abs()).max()) <= ATOL
        at += m
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        outs.append(attend(cuda, b, 16, seen, pool=pool, softmax_scale=-0.07, stream=s)[2])
    torch.cuda.synchronize()
    assert all(torch.equal(x, out) for x in outs)
    assert cuda.tq_device_error() == 0


@pytest.mark.parametrize("d,kb,vb,G,new", [(128, 8, 3, 8, 5), (128, 8, 3, 8, 50), (64, 4, 3, 4, 7), (256, 8, 4, 4, 20), (128, 5, 5, 8, 9),
                                           (512, 8, 3, 2, 6)])
@pytest.mark.parametrize("bound", [None, BOUND])
def test_a_workspace_may_hold_anything(cuda, d, kb, vb, G, new, bound):
    """NaN in all of it, then what another call left there: the same output, with sequences of no rows, of no new
    tokens, and tokens that see nothing, whose partial sums count for nothing."""
    lens = [new, 0, 700, 40 + new, 129, 1500]
    b = Batch(lens, [new, 0, new // 2, 1, 0, new], H=2, d=d, kb=kb, vb=vb, page=64, seed=d, width=-(-BOUND // 64))
    seen = tree_masks(b, "any")
    words = -(-new // 32)
    masks = dev(np.concatenate([pack(np.pad(m, ((0, 0), (0, 32 * words - m.shape[1]))), words) for m in seen]))
    pool = b.pool(cuda)
    b.fill(cuda, pool)
    pages, q = b.pages(cuda, max_len=bound), b.queries(2 * G)
    need = cuda.tq_paged_tree_attention_workspace_bytes(pool, pages, 2 * G, b.total, new)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    outs = [cuda.tq_paged_tree_attention(pool, pages, b.dev(b.starts), q.cuda(), masks, new, workspace=ws) for _ in range(2)]
    assert cuda.tq_device_error() == 0 and torch.equal(*outs)
    check_tree(b, pool, q, outs[0], seen)


@pytest.mark.parametrize("d,kb,vb,H,page,rows", [(128, 8, 3, 2, 64, 1 << 26), (64, 4, 2, 1, 16, (1 << 31) + 4096)])
def test_trees_far_into_a_large_pool(cuda, d, kb, vb, H, page, rows):
    """Planes of more than 2^32 bytes, and a pool of more than 2^31 rows: trees on every kernel, slots and kept rows at
    its last pages."""
    per_row = d * kb // 8 + d * vb // 8 + 3 * (d // 32) * 2
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < rows * per_row + (8 << 30):
        pytest.skip("not enough device memory")
    lens, width, G = [300, 17, 0, 200, 64], -(-BOUND // page), 8
    pages = rows // (H * page)
    pool = cuda.Cache(pages, H, d, page, k_bits=kb, v_bits=vb)
    for new, bound in (([2, 1, 0, 1, 2], 320), ([8, 17, 0, 3, 5], BOUND), ([60, 1, 0, 33, 64], BOUND)):  # split, block, wide
        b = Batch(lens, new, H=H, d=d, kb=kb, vb=vb, page=page, seed=13, spare=0, width=width)
        b.table = b.table + (pages - b.num_pages)
        b.fill(cuda, pool)
        seen = tree_masks(b, "tree")
        words = -(-max(new) // 32)
        masks = dev(np.concatenate([pack(np.pad(m, ((0, 0), (0, 32 * words - m.shape[1]))), words) for m in seen]))
        table, q = b.pages(cuda, max_len=bound), b.queries(H * G)
        out = cuda.tq_paged_tree_attention(pool, table, b.dev(b.starts), q.cuda(), masks, max(new))
        check_tree(b, pool, q, out, seen)
        _, slots, _ = cuda.tq_paged_layout(pool, table, b.dev(b.starts), b.total)
        at = [int(b.table[s, r // page]) * page + r % page for s, n in enumerate(lens) for r in range(n - new[s], n)]
        assert slots.tolist() == at
        before = [rows_of(pool, b.table[s], n) for s, n in enumerate(lens)]
        path = [list(range(0, n, 2)) for n in new]
        ids = np.full((5, max(new)), -1, np.int32)
        for s, x in enumerate(path):
            ids[s, :len(x)] = x
        cuda.tq_paged_keep(pool, table, b.dev(b.starts), dev(ids), dev([len(x) for x in path]))
        for s, (n, x) in enumerate(zip(lens, path)):
            for got, was in zip(rows_of(pool, b.table[s], n), before[s]):
                want = was.copy()
                want[:, n - new[s]:n - new[s] + len(x)] = was[:, [n - new[s] + i for i in x]]
                assert np.array_equal(got, want), s
    assert cuda.tq_device_error() == 0
    del pool
    torch.cuda.empty_cache()
