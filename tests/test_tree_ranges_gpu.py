"""Attention of trees over keys, values and queries of unlike sizes, every comparison among finite numbers: key groups
far from zero, outliers, scores of any size, on the kernel whose rows are dequantised on the chip."""
import numpy as np
import pytest
import torch

from pagedtest import ATOL, RTOL, dequantised
from test_drafts_gpu import tree_masks
from test_tree_block_gpu import attend, batch

pytestmark = pytest.mark.gpu


def check_numbers(b, pool, q, out, seen, lost=0.0):
    """As check_tree, but for the reference, which has to be finite everywhere; `lost` is what a score's sum may lose
    of its products' sizes (a score error e moves an output by e times the weighted distance of the values at most)."""
    at, worst, out = 0, -1.0, out.cpu().double()
    for s, (n, m) in enumerate(zip(b.lens, b.new)):
        if not m:
            continue
        k, v = (torch.from_numpy(x).double() for x in dequantised(pool, b.table[s], n))
        x = q[at:at + m].cpu().double()
        QH, d = x.shape[1:]
        vis = torch.ones(m, n, dtype=torch.bool)
        vis[:, max(0, n - m):] = torch.from_numpy(seen[s][:, max(0, m - n):])
        for h in range(QH):
            kh, vh = k[h * k.shape[0] // QH], v[h * k.shape[0] // QH]
            z = (x[:, h] @ kh.T * d ** -0.5).masked_fill(~vis, -float("inf"))
            some = vis.any(-1, keepdim=True)
            p = torch.exp(z - torch.where(some, z.amax(-1, keepdim=True), 0.0)).masked_fill(~vis, 0.0)
            p = p / torch.where(some, p.sum(-1, keepdim=True), 1.0)
            want, got = p @ vh, out[at:at + m, h]
            assert bool(torch.isfinite(want).all()), "the reference is not finite"
            assert bool(torch.isfinite(got).all()), "not finite"
            bound = ATOL + RTOL * want.abs()
            if lost:
                size = (x[:, h].abs() @ kh.abs().T * d ** -0.5).masked_fill(~vis, 0.0).amax(-1, keepdim=True)
                bound = bound + lost * size * torch.stack([p[i] @ (vh - want[i]).abs() for i in range(m)])
            worst = max(worst, float(((got - want).abs() - bound).max()))
        at += m
    assert at > 0 and worst <= 0.0, worst


def zeros_of(b, pool, s, group):
    """The zero points of a group of a sequence's keys."""
    P = pool.capacity
    pages = torch.from_numpy(b.table[s, :-(-b.lens[s] // P)].astype(np.int64)).cuda()
    z = pool.k_zero.view(torch.float16)[pages][..., group].transpose(1, 2).reshape(-1, pool.num_kv_heads)
    return z[:b.lens[s]].float().cpu()


def page_0_to(b, s):
    """The pool's first page becomes sequence s's first one."""
    was = b.table[s, 0]
    b.table = np.where(b.table == 0, -1, b.table)
    b.table[b.table == was] = 0
    b.table[b.table == -1] = was


OFFSETS = [(kb, offset) for kb in (8, 4) for offset in ((16.0, 64.0, 200.0) if kb == 8 else (64.0, 200.0, 400.0))]


@pytest.mark.parametrize("kb,offset", OFFSETS)
@pytest.mark.parametrize("d,vb,G,new", [(128, 3, 8, 9), (128, 4, 8, 40), (128, 2, 8, 4), (64, 3, 8, 9), (64, 4, 4, 40), (256, 3, 4, 9),
                                        (256, 4, 4, 40), (256, 2, 1, 12)])
def test_keys_with_an_offset(cuda, d, vb, G, new, kb, offset):
    """One group of 32 key channels far from zero, as keys of trained models have them: zero points on both sides of
    what a half-precision sum of code and zero point holds.  The first page of the pool belongs to another sequence, whose
    rows hold other codes.  A score's sum goes through d / 16 products whose sums lose 2^-20 each."""
    b = batch([900, 333, 40], [new, new, min(new, 40)], d, kb, vb, 64, seed=71)
    page_0_to(b, 2)
    for s in range(3):
        # (4-bit groups spread wide enough that none of them rounds to one value)
        b.k[s][:, :, 32:64] = (b.k[s][:, :, 32:64].float() * (1.5 if kb == 4 else 1.0) + offset).to(torch.bfloat16)
    b.k[2] = (-3.0 * b.k[2].float()).to(torch.bfloat16)
    seen = tree_masks(b, "tree")
    pool, q, out = attend(cuda, b, 2 * G, seen)
    z = torch.cat([zeros_of(b, pool, s, 1) for s in range(2)]).abs()
    assert bool(torch.isfinite(z).all())
    if (kb, offset) in ((8, 64.0), (8, 200.0), (4, 400.0)):
        assert float((z > 896).float().mean()) > 0.25
    check_numbers(b, pool, q, out, seen, lost=d / 16 * 2.0 ** -20)
    assert cuda.tq_device_error() == 0


@pytest.mark.parametrize("d,kb,vb,G,new", [(128, 8, 3, 8, 9), (128, 4, 3, 8, 16), (128, 8, 3, 8, 4), (64, 8, 4, 8, 9), (256, 8, 3, 4, 20),
                                           (128, 2, 5, 8, 9), (256, 4, 2, 4, 4)])
def test_far_outliers(cuda, d, kb, vb, G, new):
    """Rows with keys of up to 2^20 (what a half-precision scale of their width holds) that all queries point away from: no
    weight of theirs is left, and the other rows of their tile keep their precision; rows with values of 2^-14 beside
    them, and groups far from zero."""
    b = batch([new + 400, 200], [new, new], d, kb, vb, 64, seed=9)
    rng = np.random.default_rng(17)
    way = np.where(np.arange(d) % 2, 1.0, -1.0).astype(np.float32)
    q = b.queries(2 * G).float()
    q = q + torch.from_numpy(way) * (4.0 - (q * torch.from_numpy(way)).mean(-1, keepdim=True))
    q = q.to(torch.bfloat16)
    top = {8: 20, 4: 18, 2: 16}[kb]
    for s in range(2):
        for t, size in ((3, 2.0 ** top), (64, 2.0 ** 14), (150, 2.0 ** (top - 2))):
            b.k[s][t] = (torch.from_numpy(-size * way) * torch.from_numpy(1 + 0.25 * rng.random((2, 1), np.float32))).to(torch.bfloat16)
        b.v[s][8:16] = b.v[s][8:16] * 2.0 ** -14
        b.k[s][20:24, :, 32:64] = torch.from_numpy(2.0 + 2.0 ** -4 * rng.random((4, 2, 32), np.float32)).to(torch.bfloat16)
    seen = tree_masks(b, "tree")
    pool, _, out = attend(cuda, b, 2 * G, seen, q=q)
    if kb == 8:
        z = zeros_of(b, pool, 0, 1).abs()
        assert bool((z[20:24] > 896).all()) and bool((z[30:60] < 896).all())
    check_numbers(b, pool, q, out, seen)
    assert cuda.tq_device_error() == 0


@pytest.mark.parametrize("power", [0, 26, 116])
@pytest.mark.parametrize("d,kb,G,new", [(128, 8, 8, 3), (128, 8, 8, 6), (128, 8, 8, 9), (128, 4, 8, 40), (64, 4, 8, 3), (64, 8, 8, 9),
                                        (256, 8, 4, 9), (256, 4, 4, 20), (128, 5, 8, 8)])
def test_queries_of_any_size(cuda, d, kb, G, new, power):
    """Finite scores of any size: where they differ by more than what fp32 leaves of them, the rows of the largest share
    the weight.  (Keys of one of three sizes in the queries' group, so that scores are equal or far apart; a negative
    query's largest score is the smallest key's.)"""
    b = batch([400, 90], [new, new], d, kb, 3, 64, seed=4)
    sign = torch.where(torch.arange(d) % 2 == 0, 1.0, -1.0)
    for s in range(2):
        size = torch.ones(len(b.k[s]), 2, d)
        size[:, :, :32] = 1.0 + (torch.arange(len(b.k[s])) % 3)[:, None, None]
        b.k[s] = (size * sign).to(torch.bfloat16)
    q = torch.zeros(2 * new, 2 * G, d)
    q[:, :, :32] = 4.0 * sign[:32]
    q[:, 1::2] = -q[:, 1::2]
    q = (q * 2.0 ** power).to(torch.bfloat16)
    seen = tree_masks(b, "tree")
    pool, _, out = attend(cuda, b, 2 * G, seen, q=q)
    assert cuda.tq_device_error() == 0
    check_numbers(b, pool, q, out, seen)


@pytest.mark.parametrize("d,kb,vb,G,new,bound", [
    (128, 8, 3, 8, 2, 64), (128, 5, 5, 3, 6, 64), (512, 8, 3, 2, 6, 64), (128, 8, 3, 8, 5, 1 << 14), (128, 4, 3, 8, 33, 1 << 14),
    (64, 8, 4, 8, 9, 1 << 14), (256, 8, 4, 4, 40, 1 << 14), (128, 5, 5, 8, 12, 1 << 14), (128, 8, 3, 8, 60, 1 << 14), (64, 4, 2, 16, 40, 1 << 14)])
def test_more_new_tokens_than_rows(cuda, d, kb, vb, G, new, bound):
    """Lengths below the number of new tokens, on every kernel: those in front stand before the first row, tokens see of
    the rows that are there what their masks name."""
    lens = [1, new // 2 + 1, max(1, new - 1), new, new + 1, 0]
    b = batch(lens, [new] * 5 + [0], d, kb, vb, 16)
    seen = tree_masks(b, "any")
    pool = b.pool(cuda)
    b.fill(cuda, pool)
    words = -(-new // 32)
    masks = np.zeros((b.total, words), np.uint32)
    at = 0
    for m in seen:
        for row in m:
            for j in np.flatnonzero(row):
                masks[at, j // 32] |= np.uint32(1) << np.uint32(j % 32)
            at += 1
    q = b.queries(2 * G)
    out = cuda.tq_paged_tree_attention(pool, b.pages(cuda, max_len=bound), b.dev(b.starts), q.cuda(),
                                       torch.from_numpy(masks.view(np.int32)).cuda(), new)
    assert cuda.tq_device_error() == 0
    check_numbers(b, pool, q, out, seen)
