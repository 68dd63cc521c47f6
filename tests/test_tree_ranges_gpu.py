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
