"""Shared helpers of the paged-cache tests: batches in pages, and the plain
implementation (the oracle's rows, attention in binary64)."""
import numpy as np
import torch

import oracle

# An attention output is rounded once to bf16 (half a step: 2^-8 of the value).
# Before that, keys, values (centroid times rms) and probabilities carry at most
# three f16 roundings of 2^-11 each; independent and signed, they leave an error
# per output of rms at most 2^-11 sqrt(sum p^2 v^2) <= 2^-11 max|v|, with values
# of unit variance (|v| < 4.2 over the few thousand rows here, and the score
# errors they meet of the same size): six such deviations are 2^-11 * 4.2 / 6.8
# * 6 < 2e-3, the absolute tolerance of the contiguous calls as well.
ATOL, RTOL = 2e-3, 2.0 ** -8


class Batch:
    """Sequences of the given lengths, the last new[s] rows of each to be appended, in shuffled pages."""

    def __init__(self, lens, new, H, d, kb, vb, page, seed=0, spare=2, width=None, device="cuda", pad_rows=0):
        self.lens, self.new, self.H, self.d, self.kb, self.vb, self.page = list(lens), list(new), H, d, kb, vb, page
        rng = np.random.default_rng(seed)
        counts = [-(-n // page) for n in lens]
        self.num_pages = sum(counts) + spare
        order = rng.permutation(self.num_pages).astype(np.int32)
        # a bound of the lengths that lets chunks of 128 columns take the kernels of long chunks (4 Mi rows x kv-heads x
        # columns in all); a bound given with pages() may be closer
        self.bound = max(max(lens), 1, -(-(1 << 22) // (128 * H * len(lens))))
        self.width = width or -(-self.bound // page)
        self.table = np.zeros((len(lens), self.width), np.int32)
        at = 0
        for s, c in enumerate(counts):
            self.table[s, :c] = order[at:at + c]
            at += c
        self.starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.total = int(self.starts[-1])
        scale = np.exp(0.5 * rng.standard_normal((H, d))).astype(np.float32)
        self.k = [self._bf16(rng.standard_normal((n, H, d), dtype=np.float32) * scale) for n in lens]
        self.v = [self._bf16(rng.standard_normal((n, H, d), dtype=np.float32)) for n in lens]
        self.rng, self.device, self.pad_rows = rng, device, pad_rows

    @staticmethod
    def _bf16(x):
        return torch.from_numpy(x).to(torch.bfloat16)

    def tokens(self, rows, new):
        """Ragged [total][H][d]: the last new[s] rows of every sequence."""
        parts = [x[len(x) - n:] for x, n in zip(rows, new)]
        return torch.cat(parts + [torch.zeros(self.pad_rows, self.H, self.d, dtype=torch.bfloat16)])

    def dev(self, x):
        return torch.from_numpy(np.ascontiguousarray(x)).to(self.device)

    def pool(self, tq):
        return tq.Cache(self.num_pages, self.H, self.d, self.page, k_bits=self.kb, v_bits=self.vb, device=self.device)

    def pages(self, tq, lens=None, max_len=None):
        lens = self.lens if lens is None else lens
        return tq.PageTable(self.dev(self.table), self.dev(np.array(lens, np.int32)), max_len or min(self.bound, self.width * self.page))

    def fill(self, tq, pool, lens=None):
        """Append every row, as one chunk of each sequence."""
        lens = self.lens if lens is None else lens
        starts = self.dev(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
        cut = lambda rows: torch.cat([x[:n] for x, n in zip(rows, lens)]).to(self.device)  # noqa: E731
        tq.tq_paged_append(pool, self.pages(tq, lens), starts, cut(self.k), cut(self.v))

    def planes(self, s, n=None):
        """The oracle's cache of sequence s (its first n rows)."""
        n = self.lens[s] if n is None else n
        p = oracle.Planes(1, self.H, self.d, self.kb, self.vb, max(16, -(-n // 16) * 16))
        if n:
            bits = lambda x: x[:n].transpose(0, 1).contiguous()[None].view(torch.int16).numpy().view(np.uint16)  # noqa: E731
            oracle.encode(p, bits(self.k[s]), bits(self.v[s]))
        return p

    def queries(self, QH, seed=1, total=None):
        rng = np.random.default_rng(1000 + seed)
        return self._bf16(1.3 * rng.standard_normal(((self.total if total is None else total) + self.pad_rows, QH, self.d),
                                                    dtype=np.float32))


def rows_of(pool, table_row, n):
    """The first n rows of a sequence out of the pool's planes: [H][n][row] numpy arrays."""
    P = pool.capacity
    idx = torch.as_tensor(np.asarray(table_row[: -(-n // P)], dtype=np.int64))
    return [t[idx.to(t.device)].transpose(0, 1).flatten(1, 2)[:, :n].cpu().numpy() for t in pool.planes()]


def dequantised(pool, table_row, n, sign_seed=42):
    """K and V (fp32, [H][n][d]) of a sequence's rows as the pool holds them, by the oracle."""
    p = oracle.Planes(1, pool.num_kv_heads, pool.head_dim, pool.k_bits, pool.v_bits, max(16, -(-n // 16) * 16),
                      sign_seed=sign_seed)
    for dst, src in zip(p.arrays(), rows_of(pool, table_row, n)):
        dst[0, :, :n] = src if src.dtype == dst.dtype else src.view(dst.dtype)
    k, v = oracle.decode(p, 0, n)
    return k[0], v[0]


def attention64(q, k, v, first, scale=None):
    """q [M][QH][d] at positions first .. first + M - 1 over k, v [H][n][d]: binary64."""
    q = q.double()
    M, QH, d = q.shape
    H, n = k.shape[:2]
    k, v = torch.from_numpy(k).double(), torch.from_numpy(v).double()
    s = torch.einsum("mhgd,hnd->hmgn", q.view(M, H, QH // H, d), k) * (d ** -0.5 if scale is None else scale)
    hide = torch.arange(n)[None] > torch.arange(first, first + M)[:, None]
    s = s.masked_fill(hide[None, :, None], -float("inf"))
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    p = p.masked_fill(hide[None, :, None], 0.0)
    l = p.sum(-1, keepdim=True)
    p = p / torch.where(l == 0, torch.ones_like(l), l)
    # a hidden row is no part of the sum, whatever it holds
    seen = torch.where((~hide).any(0)[None, :, None], v, torch.zeros_like(v))
    if torch.isfinite(seen).all():
        o = torch.einsum("hmgn,hnd->hmgd", p, seen)
    else:
        o = torch.stack([torch.einsum("hgn,hnd->hgd", p[:, i, :, :max(0, first + i + 1)], v[:, :max(0, first + i + 1)])
                         for i in range(M)], 1)
    return o.permute(1, 0, 2, 3).reshape(M, QH, d)


def check_attention(batch, pool, q, out, lens=None, new=None, scale=None, sign_seed=42):
    """Every sequence's outputs against the plain implementation on the rows the pool holds."""
    lens, new = batch.lens if lens is None else lens, batch.new if new is None else new
    at, worst = 0, 0.0
    out = out.cpu().double()
    for s, (n, m) in enumerate(zip(lens, new)):
        if not m:
            continue
        if n:
            k, v = dequantised(pool, batch.table[s], n, sign_seed)
            want = attention64(q[at:at + m].cpu(), k, v, n - m, scale)
        else:
            want = torch.zeros(m, q.shape[1], q.shape[2], dtype=torch.float64)
        got = out[at:at + m]
        # Not finite together.  A value row with an infinite rms is +-inf in every rotated dim, and its
        # un-rotation is inf - inf = NaN except in a dim whose signs happen to agree with all of them;
        # chunks on the wide kernel give NaN there as well (the header says so).
        assert torch.equal(torch.isfinite(got), torch.isfinite(want)), f"sequence {s}: not finite elsewhere"
        err = (got - want).abs() - RTOL * want.abs()
        worst = max(worst, float(err.nan_to_num(0.0).max()))
        at += m
    assert worst <= ATOL, worst
