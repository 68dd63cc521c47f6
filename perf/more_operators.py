"""Cases, plain forms and exact values of the operators of a speculative serving step.

A step over a paged cache (a pool of packed pages, a page table, ragged new tokens: sequence s owns rows
[starts[s], starts[s + 1]) of the token tensors, its last positions) goes through

  tables     the wanted lengths come in; pages that sequences no longer need go back to a stack of free ones, pages
             that they lack are taken from it, and every new token gets its position and its slot; drafted tokens that
             form trees also the mask of their ancestors
  rotary     q and k turned by the angles of their positions
  tree       attention of the drafted tokens over their sequence's rows and their own ancestors
  verify     the drafted tokens against the target's probabilities, from given random numbers
  keep       the accepted path's rows moved together behind the sequence's own

Formulas (P: page size; a tree's node i has parent[i] < i among its sequence's new tokens, -1 at the root):
  tables     pages(n) = ceil(n / P); released entries are pushed in (sequence, page) order, lacking ones popped in that
             order; position = length - new + depth in the tree (in the row order without trees); slot = page P +
             position of the row mod P; mask bit j of token i: j is i or an ancestor of it
  rotary     (a, b) -> m (a cos t - b sin t, a sin t + b cos t), t = position * frequency of the pair
  tree       softmax(q k^T / sqrt(d) over the rows before the new ones and those whose mask bit is set) v
  verify     at an accepted node with target row p and draft row r, its children in index order: one of token x with
             number u is accepted where u r(x) M < max(p(x) - C r(x), 0), C = 0 and M = 1 at first; a rejected one sets
             C += M, M = sum max(p - C r, 0).  Without draft probabilities u M < p(x), and a rejected x sets M -= p(x),
             p(x) = 0.  The next token is the first v whose running sum of what is left passes its number times the sum
  keep       row (length - new + path[k]) -> row (length - new + k), k below the count kept
"""
import functools
import math
import random

import numpy as np
import torch

own = False
SEED = 42  # of the value sign vector


# ------------------------------------------------------------------ cases
def listed():
    cache = dict(kv_heads=8, q_heads=64, d=128, k_bits=8, v_bits=3, page=64, layout=1)
    tables = dict(kind="tables", page=64, layout=1)
    tree = dict(cache, kind="tree")
    return [
        # a decode step's bookkeeping: every sequence one token on, a few ended and a few begun
        dict(tables, name="tables decode step", seqs=64, len_lo=1, len_hi=8192, new_lo=1, new_hi=1, begin=4, end=4, trees=False),
        # the same where every sequence drafts a tree, the last step's rejected tokens given back
        dict(tables, name="tables 256 trees", seqs=256, len_lo=100, len_hi=32768, new_lo=20, new_hi=64, begin=8, end=8, trees=True),
        # a decode step's queries and keys
        dict(kind="rotary", name="rotary decode", tokens=64, q_heads=64, kv_heads=8, d=128, rot=128, interleaved=False,
             f32=False, top=32768, scaling="none", fused=True),
        # a prompt's, in pairs, half the head turned, a context stretched beyond what the model was made for
        dict(kind="rotary", name="rotary prompt 8191", tokens=8191, q_heads=32, kv_heads=8, d=128, rot=64, interleaved=True,
             f32=False, top=131072, scaling="yarn", fused=True),
        # one user, a short context, a small tree: the smallest verification
        dict(tree, name="tree one short", seqs=1, len_lo=500, len_hi=500, new_lo=16, new_hi=16, q_heads=32),
        # long contexts, a few drafted tokens each
        dict(tree, name="tree 32 long, 8 nodes", seqs=32, len_lo=24577, len_hi=32769, new_lo=5, new_hi=8),
        # trees of 64, ragged contexts: hundreds of columns to a kv-head
        dict(tree, name="tree 16 x 64 nodes k4v3", seqs=16, len_lo=500, len_hi=8192, new_lo=40, new_hi=64, k_bits=4, page=32),
        # wide heads, 4-bit values, few q-heads to a kv-head
        dict(tree, name="tree d256 k8v4", seqs=6, len_lo=900, len_hi=16384, new_lo=9, new_hi=25, d=256, kv_heads=4,
             q_heads=16, v_bits=4, page=128),
        # chains of four drafted tokens with the draft model's probabilities, a small vocabulary
        dict(kind="verify", name="verify chains 32000", seqs=16, new_lo=5, new_hi=5, vocab=32000, draft=True, bf16=False,
             chain=True, layout=1),
        # trees without draft probabilities, a large vocabulary, the largest batch
        dict(kind="verify", name="verify trees 131072", seqs=64, new_lo=8, new_hi=32, vocab=131072, draft=False, bf16=False,
             chain=False, layout=1),
        # accepted paths of a verification step moved together
        dict(cache, kind="keep", name="keep 32", seqs=32, len_lo=500, len_hi=8192, new_lo=5, new_hi=16, most=5),
        # large trees and a large batch, wide heads
        dict(cache, kind="keep", name="keep 256 x 64 nodes d256", seqs=256, len_lo=100, len_hi=1024, new_lo=40, new_hi=64,
             most=12, d=256, kv_heads=4, v_bits=4, page=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("tables", "rotary", "tree", "tree", "verify", "keep"))
    c = dict(kind=kind)
    if kind == "rotary":
        d = rng.choice((64, 128, 128, 256, 512))
        kv = rng.choice((1, 2, 4, 8))
        c.update(d=d, kv_heads=kv, q_heads=kv * rng.choice((1, 2, 3, 4, 5, 7, 8)), rot=rng.choice((d, d, d // 2, 2 * rng.randint(1, d // 2))),
                 interleaved=rng.random() < 0.5, f32=rng.random() < 0.3, top=_log(rng, 16, 1000000),
                 scaling=rng.choice(("none", "none", "linear", "ntk", "yarn")), fused=rng.random() < 0.5)
        c["tokens"] = _log(rng, 1, min(16384, 4.0e7 / (d * (c["q_heads"] + kv))))
        return c
    if kind == "verify":
        c.update(seqs=_log(rng, 1, 64), vocab=_log(rng, 2, 131072), draft=rng.random() < 0.5, bf16=rng.random() < 0.3,
                 chain=rng.random() < 0.4, layout=rng.randrange(1 << 30))
        hi = _log(rng, 1, max(2, min(64, 2.0e8 / (c["vocab"] * c["seqs"]))))
        c.update(new_lo=rng.choice((1, max(1, hi // 2), hi)), new_hi=hi)
        return c
    c.update(page=16 * rng.choice((1, 2, 3, 4, 5, 8, 16)), layout=rng.randrange(1 << 30))
    if kind == "tables":
        c["seqs"] = _log(rng, 1, 512)
        hi = _log(rng, 2, max(3, min(65536, 8.0e6 / c["seqs"])))
        trees = rng.random() < 0.5
        c.update(len_lo=rng.choice((0, 1, hi // 2)), len_hi=hi, begin=rng.randint(0, 3), end=rng.randint(0, 3), trees=trees,
                 new_lo=rng.choice((0, 1)), new_hi=min(hi, _log(rng, 1, 128 if trees else max(2, 1.0e5 / c["seqs"]))))
        return c
    d = rng.choice((64, 128, 128, 256))
    kv = rng.choice((1, 2, 4, 8))
    c.update(kv_heads=kv, q_heads=kv * rng.choice((1, 2, 3, 4, 5, 7, 8, 12, 16)), d=d, k_bits=rng.choice((8, 8, 4, 4, 2, 5)),
             v_bits=rng.choice((3, 3, 4, 2)))
    if kind == "keep":
        c["seqs"] = _log(rng, 1, 256)
        hi = _log(rng, 2, max(3, min(2048, 2.0e8 / (kv * d * c["seqs"]))))
        new = min(hi, rng.randint(1, 96))
        c.update(len_lo=max(1, hi // rng.choice((1, 4))), len_hi=hi, new_lo=max(1, new // rng.choice((1, 3))), new_hi=new,
                 most=rng.randint(1, 16))
        return c
    # the fp32 window of K and V of the plain form, and its scores
    c["seqs"] = _log(rng, 1, 48)
    hi = _log(rng, 1, max(2, min(32768, 6.0e8 / (kv * d * c["seqs"]))))
    new = min(hi, _log(rng, 1, max(2, min(128, 6.0e8 / (c["seqs"] * c["q_heads"] * hi)))))
    c.update(len_lo=max(1, hi // rng.choice((1, 3, 10))), len_hi=hi, new_lo=max(1, new // rng.choice((1, 3))), new_hi=new)
    return c


@functools.lru_cache(64)
def _shape(key):
    """Rows and new tokens of every sequence, a matter of the case alone."""
    case = dict(key)
    r = random.Random(case["layout"])
    lens, new = [], []
    for _ in range(case["seqs"]):
        n = r.randint(case["len_lo"], case["len_hi"]) if "len_lo" in case else 1 << 30
        m = min(n, r.randint(case["new_lo"], case["new_hi"]))
        lens.append(n)
        new.append(m)
    return lens, new


def lengths(case):
    return _shape(tuple(sorted(case.items())))


def trees(case):
    """The parents of every sequence's nodes: chains, or trees of two to eight children a node, level after level."""
    _, new = lengths(case)
    r = random.Random(case["layout"] + 1)
    out = []
    for n in new:
        wide = r.choice((2, 4, 8))
        out.append([-1 if i == 0 else (i - 1 if case.get("chain") else max(0, (i - 1) // wide - r.randint(0, 1))) for i in range(n)])
    return out


def paths(case):
    """Kept nodes: some that stay where they are, then some from behind all places that are written (so that a second
    pass over the same rows moves the same ones)."""
    _, new = lengths(case)
    r = random.Random(case["layout"] + 2)
    out = []
    for n in new:
        k = r.randint(1, min(n, case["most"]))
        stay = r.randint(1, k)
        stay = max(stay, 2 * k - n)  # the others have to fit behind
        out.append(list(range(stay)) + sorted(r.sample(range(k, n), k - stay)))
    return out


def tables_before(case):
    """The lengths that the tables held before the step: of a sequence that begins none, of one that ends its old rows."""
    lens, new = (list(x) for x in lengths(case))
    r = random.Random(case["layout"] + 3)
    old = [max(0, n - m + (r.randint(0, m) if case["trees"] else 0)) for n, m in zip(lens, new)]  # rejected rows still there
    order = r.sample(range(len(lens)), len(lens))
    for s in order[:case["begin"]]:
        old[s] = 0
    for s in order[case["begin"]:case["begin"] + case["end"]]:
        old[s], lens[s], new[s] = lens[s], 0, 0
    return old, lens, new


def row_bytes(case):
    d = case["d"]
    return d * case["k_bits"] // 8 + 3 * (d // 32) * 2 + d * case["v_bits"] // 8


def work(case):
    if case["kind"] == "rotary":
        size, heads = 4 if case["f32"] else 2, case["q_heads"] + case["kv_heads"]
        return {"bytes": case["tokens"] * (heads * case["d"] * 2 * size + 4), "flops": case["tokens"] * (heads * case["rot"] * 3 + case["rot"] * 10)}
    if case["kind"] == "tables":
        old, lens, new = tables_before(case)
        count = lambda n: -(-n // case["page"])  # noqa: E731
        moved = sum(abs(count(a) - count(b)) for a, b in zip(old, lens))
        words = -(-max(max(new), 1) // 32) if case["trees"] else 0
        return {"bytes": 4 * (4 * len(lens) + 2 + 2 * moved) + sum(new) * (4 + 8 + 4 * words + (4 if words else 0)), "flops": 8 * (len(lens) + sum(new))}
    lens, new = lengths(case)
    total = sum(new)
    if case["kind"] == "verify":  # one row of each distribution, at least, of every sequence
        rows = 2 if case["draft"] else 1
        return {"bytes": len(new) * case["vocab"] * rows * (2 if case["bf16"] else 4) + 16 * total, "flops": len(new) * case["vocab"] * (1 + 2 * (rows - 1))}
    if case["kind"] == "keep":
        rows = sum(k != i for p in paths(case) for k, i in enumerate(p))
        back = total * case["kv_heads"] * (row_bytes(case) + 4 * case["d"])
        return {"bytes": rows * case["kv_heads"] * 2 * row_bytes(case) + back, "flops": total * case["kv_heads"] * case["d"] * (math.log2(case["d"]) + 8)}
    d, QH = case["d"], case["q_heads"]
    seen = 0
    for n, parents in zip(lens, trees(case)):
        depth = []
        for p in parents:
            depth.append(0 if p < 0 else depth[p] + 1)
        seen += len(parents) * (n - len(parents)) + sum(depth) + len(parents)
    ints = 4 * (sum(-(-n // case["page"]) for n in lens) + 2 * len(lens) + 1 + total * -(-max(new) // 32))
    return {"bytes": sum(n for n, m in zip(lens, new) if m) * case["kv_heads"] * row_bytes(case) + total * QH * d * 4 + ints, "flops": seen * QH * 4 * d}


# ------------------------------------------------------------------ tables of the codec
@functools.lru_cache(None)
def sign_vector(d):
    """+-1 by the top bit of SplitMix64's outputs."""
    mask, out = (1 << 64) - 1, []
    for i in range(d):
        z = (SEED + (i + 1) * 0x9E3779B97F4A7C15) & mask
        z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & mask
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & mask
        out.append(-1.0 if (z ^ (z >> 31)) >> 63 else 1.0)
    return out


@functools.lru_cache(None)
def codebook(bits):
    """Lloyd-Max centroids and boundaries of a unit normal: every centroid the mean of its cell, every boundary a midpoint."""
    def means(c):
        b = np.concatenate([[-np.inf], (c[1:] + c[:-1]) / 2, [np.inf]])
        pdf = np.exp(-b * b / 2) / math.sqrt(2 * math.pi)
        # mass of a cell from the tail on its own side of zero
        tail = np.array([0.5 * math.erfc(abs(x) / math.sqrt(2)) for x in b])
        lo, hi = b[:-1], b[1:]
        mass = np.where(lo >= 0, tail[:-1] - tail[1:], np.where(hi <= 0, tail[1:] - tail[:-1], 1 - tail[:-1] - tail[1:]))
        return (pdf[:-1] - pdf[1:]) / mass

    n = 1 << bits
    c = np.linspace(-2.5, 2.5, n) if n > 4 else np.linspace(-1.5, 1.5, n)
    for _ in range(300):
        c = means(c)
    for _ in range(8):  # Newton on c - means(c)
        f = c - means(c)
        jac = np.stack([((c + e) - means(c + e) - (c - e) + means(c - e)) / 2e-5 for e in 1e-5 * np.eye(n)], axis=1)
        c = c - np.linalg.solve(jac, f)
    c = (c - c[::-1]) / 2
    return c.tolist(), ((c[1:] + c[:-1]) / 2).tolist()


# the context that a model was made for, and by how much it is stretched
SCALING = dict(base=10000.0, factor=8.0, original=16384, fast=32.0, slow=1.0)


def frequencies(rot, scaling):
    """Angle per position of every pair, and the size of the turned vectors, in 64 bits."""
    base, f = SCALING["base"], SCALING["factor"]
    if scaling == "ntk":  # the slowest pair stretched by the factor, the fastest left as it is
        base *= f ** (rot / max(rot - 2, 1))
    w = base ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if scaling == "linear":
        w = w / f
    if scaling == "yarn":  # pairs of many turns in the original context left, those of few stretched, a ramp between
        at = lambda turns: rot * math.log(SCALING["original"] / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(SCALING["fast"])), 0), min(math.ceil(at(SCALING["slow"])), rot - 1)
        ramp = np.clip((np.arange(rot // 2) - lo) / max(hi - lo, 0.001), 0, 1)
        return w / f * ramp + w * (1 - ramp), 0.1 * math.log(f) + 1
    return w, 1.0


# ------------------------------------------------------------------ inputs
def _dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x)).to(dtype).cuda()


def _starts(new):
    return _dev(np.cumsum([0] + list(new)))


def _flat(parts):
    return [x for p in parts for x in p]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 17)
    return dict(rotary=_prepare_rotary, tables=_prepare_tables, verify=_prepare_verify, tree=_prepare_cache,
                keep=_prepare_cache)[case["kind"]](case, g)


def _prepare_rotary(case, g):
    d, H, QH, n = case["d"], case["kv_heads"], case["q_heads"], case["tokens"]
    dtype = torch.float32 if case["f32"] else torch.bfloat16
    pos = torch.randint(0, case["top"], (n,), generator=g, device="cuda", dtype=torch.int32)
    if case["fused"]:  # slices of the projection's output
        x = torch.randn(n, QH + 2 * H, d, generator=g, device="cuda").to(dtype)
        q, k = x[:, :QH], x[:, QH:QH + H]
    else:
        q, k = (torch.randn(n, h, d, generator=g, device="cuda").to(dtype) for h in (QH, H))
    w, scale = frequencies(case["rot"], case["scaling"])
    if own:
        import rotated_kv_cache_gb300 as tq

        w, scale = tq.tq_rotary_frequencies(case["rot"], base=SCALING["base"], scaling=case["scaling"], factor=SCALING["factor"],
                                            original_len=SCALING["original"], fast=SCALING["fast"], slow=SCALING["slow"])
    return dict(case=dict(case), pos=pos, q=q, k=k, freqs=_dev(w, torch.float64), scale=scale)


def _prepare_tables(case, g):
    old, lens, new = tables_before(case)
    P = case["page"]
    counts = [-(-n // P) for n in old]
    most = max(max(max(old), max(lens)), 1)
    width = -(-most // P)
    capacity = sum(-(-max(a, b) // P) for a, b in zip(old, lens)) + 5
    order = torch.randperm(capacity, generator=g, device="cuda").to(torch.int32)
    first, col = np.cumsum([0] + counts), np.arange(width)[None, :]
    at = _dev(np.where(col < np.array(counts)[:, None], first[:-1, None] + col, capacity - 1), torch.long)
    table = torch.where(_dev(col < np.array(counts)[:, None], torch.bool), order[at], torch.full_like(order[at], -1))
    free = torch.full((capacity,), -1, dtype=torch.int32, device="cuda")
    left = capacity - int(first[-1])
    free[:left] = order[int(first[-1]):]
    s = dict(case=dict(case), table=table, old=_dev(old), lens=_dev(lens), new=_dev(new), free=free, count=_dev([left]),
             total=sum(new), max_len=most, max_new=max(max(new), 1), lens_out=_dev(old), count_out=_dev([0]),
             starts=torch.zeros(len(lens) + 1, dtype=torch.int32, device="cuda"), parents=None)
    if case["trees"]:
        s["parents"] = _dev(_flat(t[:n] for t, n in zip(trees(case), new)) or [0])
    if own:  # the pool's handle and the table; the row planes are not touched: the narrowest there are
        import rotated_kv_cache_gb300 as tq

        s["pool"] = tq.Cache(capacity, 1, 64, P, k_bits=2, v_bits=2)
        s["pages"] = tq.PageTable(table, s["old"], most)
        s["after"] = tq.PageTable(table, s["lens_out"], most)
    return s


def _prepare_verify(case, g):
    _, new = lengths(case)
    total, V, S = sum(new), case["vocab"], len(new)
    dtype = torch.bfloat16 if case["bf16"] else torch.float32
    parents = trees(case)
    # a model's probabilities: a few likely tokens and a long tail; the draft's are near them
    target = torch.empty(total, V, dtype=dtype, device="cuda")
    draft = torch.empty(total, V, dtype=dtype, device="cuda")
    step = max(1, int(1.0e8) // V)
    for i in range(0, total, step):
        m = min(step, total - i)
        x = 2.5 * torch.randn(m, V, generator=g, device="cuda")
        target[i:i + m] = torch.softmax(x, -1).to(dtype)
        draft[i:i + m] = torch.softmax(x + 0.7 * torch.randn(m, V, generator=g, device="cuda"), -1).to(dtype)
    starts = np.cumsum([0] + new)
    rows = _dev(_flat([max(p, 0) + int(a) for p in t] for t, a in zip(parents, starts)) or [0], torch.long)
    # drafted tokens drawn from their parent's draft row
    tokens = torch.cat([torch.multinomial(draft[rows[i:i + step]].float(), 1, generator=g)[:, 0] for i in range(0, total, step)])
    s = dict(case=dict(case), starts=_starts(new), parents=_dev(_flat(parents)), tokens=tokens.to(torch.int32), target=target,
             draft=draft if case["draft"] else None, u=torch.rand(total, generator=g, device="cuda"),
             last=torch.rand(S, generator=g, device="cuda"), max_new=max(max(new), 1))
    return s


def _prepare_cache(case, g):
    lens, new = lengths(case)
    S, H, QH, d, P = len(lens), case["kv_heads"], case["q_heads"], case["d"], case["page"]
    counts = [-(-n // P) for n in lens]
    width, used = max(1, max(counts)), sum(counts)
    pool_pages = used + 3
    # pages handed out in no order, as a pool that has served others does
    order = torch.randperm(pool_pages, generator=g, device="cuda").to(torch.int32)
    first, col = np.cumsum([0] + counts), np.arange(width)[None, :]
    table = order[_dev(np.where(col < np.array(counts)[:, None], first[:-1, None] + col, 0), torch.long)].contiguous()
    s = dict(case=dict(case), table=table, lens=_dev(lens), starts=_starts(new), max_len=max(max(lens), 1),
             max_new=max(max(new), 1), total=sum(new))
    # channels of unlike sizes, a few of them large, as keys of trained models have
    size = torch.exp(0.4 * torch.randn(H, 1, d, generator=g, device="cuda"))
    size[:, :, :: max(1, d // 4)] *= 4.0
    shift = 0.5 * torch.randn(H, 1, d, generator=g, device="cuda") * size

    def rows(shape, keys):
        x = torch.randn(shape, generator=g, device="cuda")
        return (x * size + shift if keys else x).to(torch.bfloat16)

    planes = dict(k_codes=torch.zeros(pool_pages, H, P, d * case["k_bits"] // 8, dtype=torch.uint8, device="cuda"),
                  k_scale=torch.zeros(pool_pages, H, P, d // 32, dtype=torch.float16, device="cuda"),
                  k_zero=torch.zeros(pool_pages, H, P, d // 32, dtype=torch.float16, device="cuda"),
                  v_codes=torch.zeros(pool_pages, H, P, d * case["v_bits"] // 8, dtype=torch.uint8, device="cuda"),
                  v_scale=torch.zeros(pool_pages, H, P, d // 32, dtype=torch.float16, device="cuda"))
    step = max(1, int(6e7) // (H * P * d))
    for p0 in range(0, pool_pages, step):  # the rows that are there already
        n = min(step, pool_pages - p0)
        for name, x in zip(("k_codes", "k_scale", "k_zero"), encode_keys(rows((n, H, P, d), True), case["k_bits"])):
            planes[name][p0:p0 + n] = x
        for name, x in zip(("v_codes", "v_scale"), encode_values(rows((n, H, P, d), False), case["v_bits"])):
            planes[name][p0:p0 + n] = x
    s.update(planes)
    if own:
        import rotated_kv_cache_gb300 as tq

        s["pool"] = tq.Cache.from_planes(s["k_codes"], s["k_scale"], s["k_zero"], s["v_codes"], s["v_scale"], head_dim=d,
                                         k_bits=case["k_bits"], v_bits=case["v_bits"], sign_seed=SEED)
        s["pages"] = tq.PageTable(table, s["lens"], s["max_len"])
    if case["kind"] == "keep":
        chosen = paths(case)
        path = np.full((S, s["max_new"]), -1)
        for i, p in enumerate(chosen):
            path[i, :len(p)] = p
        s.update(path=_dev(path), kept=_dev([len(p) for p in chosen]), lens_out=_dev(lens))
        return s
    sharp = torch.exp(0.5 * torch.randn(1, QH, 1, generator=g, device="cuda")) / (size.mean() * 2)
    s["q"] = (torch.randn(s["total"], QH, d, generator=g, device="cuda") * 1.5 * sharp).to(torch.bfloat16)
    words = -(-s["max_new"] // 32)
    masks = np.zeros((s["total"], words), np.uint32)
    at = 0
    for t in trees(case):  # bit j of token i: j is i or an ancestor of it
        for i, p in enumerate(t):
            if p >= 0:
                masks[at + i] = masks[at + p]
            masks[at + i, i // 32] |= np.uint32(1 << (i % 32))
        at += len(t)
    s["masks"] = _dev(masks.view(np.int32))
    if own:  # the workspace that a serving loop keeps
        need = tq.tq_paged_tree_attention_workspace_bytes(s["pool"], s["pages"], QH, s["total"], s["max_new"])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms
@functools.lru_cache(None)
def _sylvester(d):
    h = torch.ones(1, 1)
    for _ in range(d.bit_length() - 1):
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)])
    return h.cuda()


@functools.lru_cache(None)
def _constants(d, bits):
    c, b = codebook(bits)
    return tuple(torch.tensor(x, dtype=torch.float32, device="cuda") for x in (sign_vector(d), c, b))


def pack(codes, bits):
    """[..., d] codes -> [..., d bits / 8] bytes, little-endian."""
    if bits == 8:
        return codes.to(torch.uint8)
    *lead, d = codes.shape
    w = codes.reshape(*lead, d // 8, 8).to(torch.int64) << (bits * torch.arange(8, device=codes.device))
    w = w.sum(-1, keepdim=True)  # 8 codes are `bits` whole bytes
    return ((w >> (8 * torch.arange(bits, device=codes.device))) & 255).reshape(*lead, d * bits // 8).to(torch.uint8)


def unpack(packed, bits):
    if bits == 8:
        return packed.to(torch.int32)
    *lead, n = packed.shape
    w = packed.reshape(*lead, n // bits, bits).to(torch.int64) << (8 * torch.arange(bits, device=packed.device))
    w = w.sum(-1, keepdim=True)
    return ((w >> (bits * torch.arange(8, device=packed.device))) & ((1 << bits) - 1)).reshape(*lead, n * 8 // bits).to(torch.int32)


def encode_keys(x, bits):
    x = x.float().unflatten(-1, (-1, 32))
    hi, lo = x.amax(-1, keepdim=True), x.amin(-1, keepdim=True)
    scale = (hi - lo) / torch.full_like(hi, 254.0 if bits == 8 else 2.0 ** bits - 1)
    zero = torch.round((hi + lo) / (2 * scale)) if bits == 8 else torch.round(lo / scale)
    codes = torch.round(x / scale - zero)
    codes = codes.clamp(-127, 127) if bits == 8 else codes.clamp(0, 2.0 ** bits - 1)
    codes = (codes.to(torch.int32) & 255 if bits == 8 else codes.to(torch.int32)).flatten(-2)
    return pack(codes, bits), scale[..., 0].half(), zero[..., 0].half()


def encode_values(x, bits):
    d = x.shape[-1]
    signs, _, bounds = _constants(d, bits)
    y = ((x.float() * signs) @ _sylvester(d) * (1 / math.sqrt(d))).unflatten(-1, (-1, 32))
    rms = torch.sqrt((y * y).mean(-1, keepdim=True))
    codes = torch.searchsorted(bounds, (y / (rms + 1e-8)).contiguous()).flatten(-2)
    return pack(codes, bits), rms[..., 0].half()


def decode_keys(codes, scale, zero, bits):
    c = unpack(codes, bits)
    c = torch.where(c > 127, c - 256, c) if bits == 8 else c
    x = (c.float().unflatten(-1, (-1, 32)) + zero.float()[..., None]) * scale.float()[..., None]
    return x.flatten(-2)


def decode_values(codes, scale, bits, d):
    signs, centroids, _ = _constants(d, bits)
    x = (centroids[unpack(codes, bits).long()].unflatten(-1, (-1, 32)) * scale.float()[..., None]).flatten(-2)
    return (x @ _sylvester(d)) * (1 / math.sqrt(d)) * signs


def plain_rotary(state):
    c, rot = state["case"], state["case"]["rot"]
    t = state["pos"].double()[:, None] * state["freqs"]
    cos, sin = ((f(t) * state["scale"]).float()[:, None] for f in (torch.cos, torch.sin))
    out = []
    for x in (state["q"], state["k"]):
        y = x.float()
        if c["interleaved"]:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        else:
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        out.append(torch.cat([turned, y[..., rot:]], -1).to(x.dtype))
    return tuple(out)


def plain_tables(state):
    c, P = state["case"], state["case"]["page"]
    table, free = state["table"], state["free"]
    S, width = table.shape
    pages = lambda n: ((n + P - 1) // P)[:, None]  # noqa: E731
    old, want = pages(state["old"].long()), pages(state["lens"].long())
    col = torch.arange(width, device="cuda")
    give, take = (col >= want) & (col < old), (col >= old) & (col < want)
    order = lambda m: (m.flatten().cumsum(0) - 1).view(S, width)  # noqa: E731
    count, cap = state["count"].long(), free.shape[0]
    stack = torch.cat([free, free[:1]])  # one place for what moves nowhere
    stack = stack.scatter(0, torch.where(give, count + order(give), cap).flatten(), table.flatten())
    top = count + give.sum()
    table = torch.where(take, stack[torch.where(take, top - 1 - order(take), 0)], table)
    starts = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), state["new"].long().cumsum(0)])
    out = [table, state["lens"].clone(), starts.to(torch.int32), stack[:cap], (top - take.sum()).to(torch.int32)]
    # places of the new tokens
    row = torch.arange(state["total"], device="cuda")
    seq = torch.searchsorted(starts[1:], row, right=True)
    node, before = row - starts[seq], (state["lens"] - state["new"]).long()[seq]
    pos = before + node
    slots = table.long()[seq, pos // P] * P + pos % P
    if state["parents"] is None:
        return (*out, pos.to(torch.int32), slots)
    M = state["max_new"]
    parents = state["parents"].long()[:state["total"]]
    up = torch.eye(M, device="cuda").repeat(S, 1, 1)
    up[seq, node, torch.where(parents < 0, node, parents)] = 1.0
    for _ in range(M.bit_length()):  # up to 2, 4, 8, ... steps towards the root
        up = ((up @ up) > 0).float()
    seen = up[seq, node] > 0  # [total][M]
    pos = before + seen.sum(-1) - 1
    words = -(-M // 32)
    seen = torch.nn.functional.pad(seen, (0, words * 32 - M)).view(-1, words, 32).long()
    masks = (seen << torch.arange(32, device="cuda")).sum(-1)
    return (*out, pos.to(torch.int32), slots, masks.to(torch.int32))


def plain_tree(state):
    c = state["case"]
    H, QH, d, M, P = c["kv_heads"], c["q_heads"], c["d"], state["max_new"], c["page"]
    S, L, G = state["table"].shape[0], state["max_len"], c["q_heads"] // c["kv_heads"]

    def window(name):  # [S][H][max_len][row]
        x = state[name][state["table"].long()]
        return x.transpose(1, 2).flatten(2, 3)[:, :, :L]

    k = decode_keys(window("k_codes"), window("k_scale"), window("k_zero"), c["k_bits"])
    v = decode_values(window("v_codes"), window("v_scale"), c["v_bits"], d)
    row, starts = torch.arange(state["total"], device="cuda"), state["starts"].long()
    seq = torch.searchsorted(starts[1:], row, right=True)
    node = row - starts[seq]
    q = torch.zeros(S, M, H, G, d, device="cuda")
    q[seq, node] = state["q"].float().unflatten(1, (H, G))
    bits = ((state["masks"].long()[..., None] >> torch.arange(32, device="cuda")) & 1).flatten(-2)[:, :M] > 0
    before = (state["lens"].long() - (starts[1:] - starts[:-1]))[seq][:, None]
    at = torch.arange(L, device="cuda")[None] - before  # a row's place among the new ones
    ahead = torch.gather(bits, 1, at.clamp(0, M - 1))
    seen = torch.zeros(S, M, L, dtype=torch.bool, device="cuda")
    seen[seq, node] = (at < 0) | ((at < M) & ahead)
    s = q.permute(0, 2, 1, 3, 4).flatten(2, 3) @ k.transpose(2, 3) * (1 / math.sqrt(d))  # [S][H][M G][L]
    s = s.unflatten(2, (M, G)).masked_fill_(~seen[:, None, :, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1)[..., None]
    o = (p.flatten(2, 3) @ v).unflatten(2, (M, G)) / torch.where(total == 0, torch.ones_like(total), total)
    return o.permute(0, 2, 1, 3, 4).flatten(2, 3)[seq, node].to(torch.bfloat16)


def plain_verify(state):
    """One node after another in index order, all sequences together: a node whose parent is the last accepted one is
    looked at, which goes through a node's children in order and then through those of the accepted one."""
    S, M, V = state["last"].shape[0], state["max_new"], state["case"]["vocab"]
    starts = state["starts"].long()
    n, seqs = starts[1:] - starts[:-1], torch.arange(S, device="cuda")
    cur, count = torch.zeros_like(n), (n > 0).long()
    path = torch.full((S, M), -1, dtype=torch.long, device="cuda")
    path[:, 0] = torch.where(n > 0, 0, -1)
    C, mass = torch.zeros(S, dtype=torch.double, device="cuda"), torch.ones(S, dtype=torch.double, device="cuda")
    rows = lambda x, at: x[(starts[:-1] + at).clamp(max=x.shape[0] - 1)]  # noqa: E731
    gone = torch.full((S, M), V, device="cuda")  # rejected tokens (V: none), without draft probabilities

    def rest():  # what is left of the current nodes' target rows
        p = rows(state["target"], cur).double()
        if state["draft"] is None:
            return torch.nn.functional.pad(p, (0, 1)).scatter(1, gone, 0.0)[:, :V]
        return (p - C[:, None] * rows(state["draft"], cur).double()).clamp(min=0)

    def at(name, x):  # the current row's entry of a token
        return state[name][(starts[:-1] + cur).clamp(max=state[name].shape[0] - 1), x].double()

    for j in range(1, M):
        child = (j < n) & (rows(state["parents"], j).long() == cur)
        x, u = rows(state["tokens"], j).long(), rows(state["u"], j).double()
        p = at("target", x)
        if state["draft"] is None:
            r = torch.where((gone == x[:, None]).any(1), 0.0, p)
            yes = child & (u * mass < r)
            mass = torch.where(child & ~yes, mass - r, mass)
            gone[:, j] = torch.where(child & ~yes, x, V)
            gone = torch.where(yes[:, None], V, gone)
        else:
            t = at("draft", x)
            yes = child & (u * t * mass < (p - C * t).clamp(min=0))
            C = torch.where(child & ~yes, C + mass, C)
            mass = torch.where(child & ~yes, rest().sum(-1), mass)
        cur = torch.where(yes, j, cur)
        path[seqs, count.clamp(max=M - 1)] = torch.where(yes, j, path[seqs, count.clamp(max=M - 1)])
        count = count + yes
        C, mass = torch.where(yes, 0.0, C), torch.where(yes, 1.0, mass)
    run_sum = rest().cumsum(-1)
    goal = state["last"].double()[:, None] * run_sum[:, -1:]
    token = (run_sum <= goal).sum(-1)
    return path.to(torch.int32), count.to(torch.int32), torch.where(n > 0, token, -1).to(torch.int32)


def plain_keep(state):
    c, P, M = state["case"], state["case"]["page"], state["max_new"]
    starts, lens = state["starts"].long(), state["lens"].long()
    before = lens - (starts[1:] - starts[:-1])
    S, k = lens.shape[0], torch.arange(M, device="cuda")
    live = k < state["kept"][:, None]
    source = torch.where(live, state["path"].long(), 0)  # beyond the kept ones: the first, which stays where it is
    line = torch.arange(S, device="cuda")[:, None]

    def place(at):
        pos = before[:, None] + at
        return state["table"].long()[line, pos // P].flatten(), (pos % P).flatten()

    (page, slot), (to_page, to_slot) = place(source), place(torch.where(live, k, 0))
    for name in ("k_codes", "k_scale", "k_zero", "v_codes", "v_scale"):
        state[name][to_page, :, to_slot] = state[name][page, :, slot]  # all read before the first is written
    row = torch.arange(state["total"], device="cuda")
    seq = torch.searchsorted(starts[1:], row, right=True)
    pos = before[seq] + row - starts[seq]
    page, slot = state["table"].long()[seq, pos // P], pos % P
    pick = lambda name: state[name][page, :, slot]  # noqa: E731  [total][H][row]
    return (decode_keys(pick("k_codes"), pick("k_scale"), pick("k_zero"), c["k_bits"]).to(torch.bfloat16),
            decode_values(pick("v_codes"), pick("v_scale"), c["v_bits"], c["d"]).to(torch.bfloat16),
            (before + state["kept"]).to(torch.int32))


# ------------------------------------------------------------------ one pass
def run(state):
    kind = state["case"]["kind"]
    if not own:
        return dict(rotary=plain_rotary, tables=plain_tables, verify=plain_verify, tree=plain_tree, keep=plain_keep)[kind](state)
    import rotated_kv_cache_gb300 as tq

    if kind == "rotary":
        return tq.tq_rotary(state["pos"], state["freqs"], state["q"], state["k"], interleaved=state["case"]["interleaved"],
                            scale=state["scale"])
    if kind == "tables":
        tq.tq_page_table_update(state["pool"], state["pages"], state["lens"], state["free"], state["count"], new_tokens=state["new"],
                                lens_out=state["lens_out"], starts=state["starts"], free_count_out=state["count_out"])
        placed = tq.tq_paged_layout(state["pool"], state["after"], state["starts"], state["total"], parents=state["parents"],
                                    max_new=state["max_new"])
        out = (state["table"], state["lens_out"], state["starts"], state["free"], state["count_out"])
        return out + (placed if state["parents"] is not None else placed[:2])
    if kind == "verify":
        return tq.tq_verify_drafts(state["starts"], state["parents"], state["tokens"], state["target"], state["draft"], state["u"],
                                   state["last"], state["max_new"])
    if kind == "tree":
        return tq.tq_paged_tree_attention(state["pool"], state["pages"], state["starts"], state["q"], state["masks"],
                                          state["max_new"], workspace=state["workspace"])
    # keep, and the new rows as they are then (their places behind the kept ones among them)
    tq.tq_paged_keep(state["pool"], state["pages"], state["starts"], state["path"], state["kept"], lens_out=state["lens_out"])
    return *tq.tq_paged_decode(state["pool"], state["pages"], state["starts"], state["total"]), state["lens_out"]


# ------------------------------------------------------------------ exact values
def _butterfly(x):
    """Sylvester's transform of the last axis over sqrt(d), in 64 bits."""
    d, h = x.shape[-1], 1
    while h < d:
        x = x.reshape(*x.shape[:-1], d // (2 * h), 2, h) if x.shape[-1] == d else x
        a, b = x[..., 0, :], x[..., 1, :]
        x = torch.stack([a + b, a - b], dim=-2).reshape(*a.shape[:-2], d)
        h *= 2
    return x / math.sqrt(d)


def _bits_of(packed, bits):
    """Codes of little-endian packed rows, bit by bit."""
    bit = (packed[..., None].to(torch.int16) >> torch.arange(8, device=packed.device)) & 1
    bit = bit.flatten(-2).unflatten(-1, (-1, bits)).double()
    return (bit * 2.0 ** torch.arange(bits, device=packed.device)).sum(-1)


def _exact_rows(state, page, slot):
    """64-bit K and V of pool rows: [n][H][d]."""
    c = state["case"]
    group = lambda name: state[name][page, :, slot].double().repeat_interleave(32, -1)  # noqa: E731
    code = _bits_of(state["k_codes"][page, :, slot], c["k_bits"])
    code = code - 256 * (code > 127) if c["k_bits"] == 8 else code
    k = (code + group("k_zero")) * group("k_scale")
    cen = torch.tensor(codebook(c["v_bits"])[0], dtype=torch.float64, device="cuda")
    y = cen[_bits_of(state["v_codes"][page, :, slot], c["v_bits"]).long()] * group("v_scale")
    return k, _butterfly(y) * torch.tensor(sign_vector(c["d"]), dtype=torch.float64, device="cuda")


def _exact_rotary(state):
    rot, out = state["case"]["rot"], []
    turn = state["scale"] * torch.exp(1j * (state["pos"].double()[:, None, None] * state["freqs"]))  # m e^(i t)
    for x in (state["q"], state["k"]):
        y = x.double()
        if state["case"]["interleaved"]:
            z = torch.view_as_complex(y[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * turn
            y[..., :rot] = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * turn
            y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
        out.append(y)
    return tuple(out)


def _exact_tables(state):
    c, P = state["case"], state["case"]["page"]
    table, free = state["table"].cpu().numpy().copy(), state["free"].cpu().numpy().copy()
    old, lens, new = tables_before(c)
    top, starts = int(state["count"]), [0]
    for s in range(len(lens)):
        for i in range(-(-lens[s] // P), -(-old[s] // P)):
            free[top] = table[s, i]
            top += 1
    for s in range(len(lens)):
        for i in range(-(-old[s] // P), -(-lens[s] // P)):
            top -= 1
            table[s, i] = free[top]
        starts.append(starts[-1] + new[s])
    pos, slots, masks = [], [], []
    words = -(-state["max_new"] // 32)
    for s, parents in enumerate(trees(c)):
        up = []
        for i in range(new[s]):
            row = lens[s] - new[s] + i
            slots.append(int(table[s, row // P]) * P + row % P)
            up.append([i] + (up[parents[i]] if parents[i] >= 0 else []))
            pos.append(lens[s] - new[s] + len(up[-1]) - 1 if c["trees"] else row)
            masks.append([sum(1 << (j % 32) for j in up[-1] if j // 32 == w) for w in range(words)] if c["trees"] else [])
    out = [_dev(table), _dev(lens), _dev(starts), _dev(free), _dev([top]), _dev(pos), _dev(np.array(slots, np.int64), torch.int64)]
    if c["trees"]:
        out.append(_dev(np.array(masks, np.uint32).reshape(-1, words).view(np.int32)))
    return tuple(out)


def _exact_verify(state):
    c = state["case"]
    _, new = lengths(c)
    tokens, u, last = (state[k].cpu().tolist() for k in ("tokens", "u", "last"))
    path, kept, token, at = [], [], [], 0
    for s, parents in enumerate(trees(c)):
        here, way, C, mass, gone = 0, [0], 0.0, 1.0, []
        row = lambda name: state[name][at + here].double()  # noqa: E731, B023

        def left():
            p = row("target").clone()  # noqa: B023
            if c["draft"]:
                return torch.relu(p - C * row("draft"))  # noqa: B023
            p[gone] = 0.0  # noqa: B023
            return p

        while True:
            for j in [i for i, p in enumerate(parents) if p == here and i > 0]:
                x = tokens[at + j]
                chance = float(left()[x])
                if u[at + j] * (float(row("draft")[x]) if c["draft"] else 1.0) * mass < chance:
                    here, C, mass, gone = j, 0.0, 1.0, []
                    way.append(j)
                    break
                if c["draft"]:
                    C += mass
                    mass = float(left().sum())
                else:
                    mass -= chance
                    gone.append(x)
            else:
                break
        run_sum = torch.cumsum(left(), 0)
        token.append(int(torch.searchsorted(run_sum, last[s] * run_sum[-1], right=True)))
        path.append(way + [-1] * (state["max_new"] - len(way)))
        kept.append(len(way))
        at += new[s]
    return _dev(path), _dev(kept), _dev(token)


def _exact_keep(state):
    c, P = state["case"], state["case"]["page"]
    lens, new = lengths(c)
    k, v, table = [], [], state["table"].cpu().numpy()
    for s, way in enumerate(paths(c)):
        base = lens[s] - new[s]
        at = np.array([base + (way[i] if i < len(way) else i) for i in range(new[s])])
        rows = _exact_rows(state, _dev(table[s, at // P], torch.long), _dev(at % P, torch.long))
        k.append(rows[0])
        v.append(rows[1])
    return torch.cat(k), torch.cat(v), _dev([n - m + len(p) for n, m, p in zip(lens, new, paths(c))])


def _exact_tree(state):
    c = state["case"]
    lens, _ = lengths(c)
    H, G, P, d = c["kv_heads"], c["q_heads"] // c["kv_heads"], c["page"], c["d"]
    out, at = [], 0
    for s, (n, parents) in enumerate(zip(lens, trees(c))):
        m = len(parents)
        pos = torch.arange(n, device="cuda")
        parts = [_exact_rows(state, state["table"][s].long()[x // P], x % P) for x in pos.split(4096)]
        k, v = (torch.cat([p[i] for p in parts]) for i in (0, 1))
        seen = np.zeros((m, n), bool)
        for i, p in enumerate(parents):
            seen[i, :n - m] = True
            if p >= 0:
                seen[i] |= seen[p]
            seen[i, n - m + i] = True
        seen = _dev(seen, torch.bool)
        o = torch.empty(m, H * G, d, dtype=torch.float64, device="cuda")
        for h in range(H):
            q = state["q"][at:at + m, h * G:(h + 1) * G].double()
            x = (q.flatten(0, 1) @ k[:, h].T / math.sqrt(d)).unflatten(0, (m, G))
            x = torch.where(seen[:, None], x, torch.full_like(x, -math.inf))
            o[:, h * G:(h + 1) * G] = (torch.softmax(x, -1).flatten(0, 1) @ v[:, h]).unflatten(0, (m, G))
        out.append(o)
        at += m
    return torch.cat(out)


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        state = prepare(case, seed)
    finally:
        own = kept
    return dict(rotary=_exact_rotary, tables=_exact_tables, verify=_exact_verify, tree=_exact_tree, keep=_exact_keep)[case["kind"]](state)
