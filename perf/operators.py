"""Cases, plain forms and exact values of the paged-cache operators.

A paged cache is one pool of packed pages (page_size token rows of every
kv-head each) and, per batch, a page table: for every sequence the list of its
pages and its length.  New tokens are ragged: sequence s owns rows
[starts[s], starts[s + 1]) of the token tensors, its last starts[s + 1] -
starts[s] positions.  Three operators work on it:

  append     quantise the new tokens' K and V into their pages (run reads the
             rows back in the same pass, the update-and-fetch form)
  fetch      read the last rows of every sequence back as K and V
  attention  causal attention of the new tokens over their sequence's rows,
             one token each (decode), a few (verification) or a long chunk

Formulas, for a row x of head_dim d in groups of 32:
  keys    8 bits: s = (max - min) / 254, z = round((max + min) / (2 s)),
          c = clip(round(x / s - z), -127, 127); b in {2, 4, 5} bits:
          s = (max - min) / (2^b - 1), z = round(min / s),
          c = clip(round(x / s - z), 0, 2^b - 1); s and z stored as fp16;
          k = (c + z) s
  values  y = H (x * signs) / sqrt(d), rms = sqrt(mean(y^2)) per group (fp16),
          c = #{boundaries < y / (rms + 1e-8)}; v = signs * H (centroid[c] rms)
          / sqrt(d), H the Sylvester matrix
  out     softmax(q k^T * d^-1/2 over positions <= the token's own) v, q-head h
          reading kv-head h / (q_heads / kv_heads); zero where nothing is visible
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
    base = dict(kv_heads=8, q_heads=64, d=128, k_bits=8, v_bits=3, page=64, layout=1, singles=0, empty=0)
    att = dict(base, kind="attention")
    return [
        # a decode step's append: one token of each running sequence, where the call's latency counts
        dict(base, name="append one token each", kind="append", seqs=32, len_lo=1, len_hi=8192, new_lo=1, new_hi=1),
        # prompts of several users prefilled together, ragged, on top of what some of them had
        dict(base, name="append prompts", kind="append", seqs=5, len_lo=3001, len_hi=9000, new_lo=3000, new_hi=8200, page=32),
        # windows handed to a dense attention call in the model's type
        dict(base, name="fetch windows", kind="fetch", seqs=4, len_lo=7000, len_hi=8192, new_lo=8192, new_hi=8192, f32=False),
        # wide heads, 4- and 2-bit codes, read back in fp32 to check or re-encode a cache
        dict(base, name="fetch d256 k4v2 fp32", kind="fetch", seqs=11, len_lo=1, len_hi=3000, new_lo=1, new_hi=3000, d=256,
             kv_heads=4, q_heads=16, k_bits=4, v_bits=2, page=48, f32=True, layout=4),
        # one user, a short context: the smallest decode step
        dict(att, name="decode one short", seqs=1, len_lo=500, len_hi=500, new_lo=1, new_hi=1, q_heads=32),
        # a full decode batch of long contexts (the benchmark's decode step, now in pages and ragged)
        dict(att, name="decode 32 long", seqs=32, len_lo=24577, len_hi=32769, new_lo=1, new_hi=1),
        # continuous batching: contexts of every length, two slots empty, small pages, 4-bit keys
        dict(att, name="decode 64 ragged k4v3", seqs=64, len_lo=1, len_hi=8192, new_lo=1, new_hi=1, q_heads=32, k_bits=4,
             page=16, empty=2),
        # wide heads, 4-bit values, few q-heads to a kv-head
        dict(att, name="decode d256 k8v4", seqs=6, len_lo=900, len_hi=16384, new_lo=1, new_hi=1, d=256, kv_heads=4, q_heads=16,
             v_bits=4, page=128),
        # speculative verification: a few drafted tokens of each sequence
        dict(att, name="verify 4 each", seqs=16, len_lo=500, len_hi=8192, new_lo=2, new_hi=4),
        # a prompt from empty
        dict(att, name="prompt 8191", seqs=1, len_lo=8191, len_hi=8191, new_lo=8191, new_hi=8191, q_heads=32),
        # a chunk of a long document, 4-bit keys
        dict(att, name="chunk 2048 over 32768 k4v3", seqs=1, len_lo=32768, len_hi=32768, new_lo=2048, new_hi=2048, k_bits=4),
        # a mixed batch: decode rows beside prefill chunks, short heads
        dict(att, name="mixed d64", seqs=16, len_lo=300, len_hi=4096, new_lo=200, new_hi=512, singles=13, d=64, q_heads=32,
             v_bits=4, page=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    d = rng.choice((64, 128, 128, 256))
    kv = rng.choice((1, 2, 4, 8))
    c = dict(kind=rng.choice(("append", "fetch", "attention", "attention", "attention")), kv_heads=kv,
             q_heads=kv * rng.choice((1, 2, 3, 4, 5, 7, 8, 12, 16)), d=d, k_bits=rng.choice((8, 8, 4, 4, 2, 5)),
             v_bits=rng.choice((3, 3, 4, 2)), page=16 * rng.choice((1, 2, 3, 4, 5, 8, 16)), layout=rng.randrange(1 << 30),
             singles=0, empty=rng.choice((0, 0, 1, 2)))
    budget = 4.0e9 / (kv * d)  # rows of all sequences that the fp32 plain form holds easily
    if c["kind"] != "attention":
        c["seqs"] = _log(rng, 1, 64)
        hi = _log(rng, 1, max(2, min(8192, 3.0e7 / (kv * d * c["seqs"]))))
        c.update(len_lo=max(1, hi // rng.choice((1, 2, 5))), len_hi=hi, new_lo=1, new_hi=rng.choice((1, hi, hi)))
        if c["kind"] == "fetch":
            c["f32"] = rng.random() < 0.5
        return c
    form = rng.choice(("decode", "decode", "verify", "chunk", "mixed"))
    if form in ("decode", "verify"):
        c["seqs"] = _log(rng, 1, 128)
        hi = _log(rng, 1, max(2, min(65536, 0.2 * budget / c["seqs"])))
        c.update(len_lo=max(1, hi // rng.choice((1, 3, 10))), len_hi=hi, new_lo=1, new_hi=1 if form == "decode" else rng.randint(2, 9))
        return c
    # the fp32 scores of the plain form, padded: seqs * new * q_heads * len elements
    c["seqs"] = rng.randint(1, 2) if form == "chunk" else rng.randint(3, 12)
    c["singles"] = 0 if form == "chunk" else c["seqs"] - rng.randint(1, 2)
    hi = _log(rng, 17, 16384)
    new = min(hi, _log(rng, 10, max(11, min(4096, 1.5e9 / (c["seqs"] * c["q_heads"] * hi)))))
    c.update(len_lo=max(1, hi // rng.choice((1, 2))), len_hi=hi, new_lo=max(1, new // 2), new_hi=new)
    return c


def lengths(case):
    """Rows and new tokens of every sequence, a matter of the case alone."""
    r = random.Random(case["layout"])
    lens, new = [], []
    for s in range(case["seqs"]):
        n = r.randint(case["len_lo"], case["len_hi"])
        m = 1 if s < case["singles"] else min(n, r.randint(case["new_lo"], case["new_hi"]))
        if s >= case["seqs"] - case["empty"] and case["seqs"] > case["empty"]:
            n = m = 0  # a slot without a sequence
        lens.append(n)
        new.append(m)
    return lens, new


def row_bytes(case):
    d = case["d"]
    return d * case["k_bits"] // 8 + 3 * (d // 32) * 2 + d * case["v_bits"] // 8


def work(case):
    lens, new = lengths(case)
    d, H, QH = case["d"], case["kv_heads"], case["q_heads"]
    total, ints = sum(new), 4 * (sum(-(-n // case["page"]) for n in lens) + 2 * len(lens) + 1)
    transform = d * math.log2(d) + 6 * d  # of one value row, with its quantisation or lookup
    if case["kind"] == "append":
        return {"bytes": total * H * (8 * d + row_bytes(case)) + ints, "flops": total * H * (2 * transform + 10 * d)}
    if case["kind"] == "fetch":
        return {"bytes": total * H * (row_bytes(case) + 2 * d * (4 if case["f32"] else 2)) + ints,
                "flops": total * H * (transform + 2 * d)}
    pairs = sum(m * (n - m) + m * (m + 1) // 2 for n, m in zip(lens, new))
    rows = sum(n for n, m in zip(lens, new) if m)
    return {"bytes": rows * H * row_bytes(case) + total * QH * d * 4 + ints, "flops": pairs * QH * 4 * d}


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


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev, g = "cuda", torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 17)
    lens, new = lengths(case)
    S, H, QH, d, P = len(lens), case["kv_heads"], case["q_heads"], case["d"], case["page"]
    counts = [-(-n // P) for n in lens]
    width, used = max(1, max(counts)), sum(counts)
    pool_pages = used + 3
    # pages handed out in no order, as a pool that has served others does
    order = torch.randperm(pool_pages, generator=g, device=dev).to(torch.int32)
    first = np.cumsum([0] + counts)
    col = np.arange(width)[None, :]
    at = np.where(col < np.array(counts)[:, None], first[:-1, None] + col, 0)
    table = order[torch.from_numpy(at).to(dev)].contiguous()
    state = dict(case=dict(case), table=table, lens=torch.tensor(lens, dtype=torch.int32, device=dev),
                 starts=torch.tensor(np.cumsum([0] + new), dtype=torch.int32, device=dev), max_len=max(max(lens), 1),
                 max_new=max(max(new), 1), total=sum(new))
    # channels of unlike sizes, a few of them large, as keys of trained models have
    size = torch.exp(0.4 * torch.randn(H, 1, d, generator=g, device=dev))
    size[:, :, :: max(1, d // 4)] *= 4.0
    shift = 0.5 * torch.randn(H, 1, d, generator=g, device=dev) * size

    def rows(shape, keys):
        x = torch.randn(shape, generator=g, device=dev)
        return (x * size + shift if keys else x).to(torch.bfloat16)

    planes = dict(k_codes=torch.zeros(pool_pages, H, P, d * case["k_bits"] // 8, dtype=torch.uint8, device=dev),
                  k_scale=torch.zeros(pool_pages, H, P, d // 32, dtype=torch.float16, device=dev),
                  k_zero=torch.zeros(pool_pages, H, P, d // 32, dtype=torch.float16, device=dev),
                  v_codes=torch.zeros(pool_pages, H, P, d * case["v_bits"] // 8, dtype=torch.uint8, device=dev),
                  v_scale=torch.zeros(pool_pages, H, P, d // 32, dtype=torch.float16, device=dev))
    step = max(1, int(6e7) // (H * P * d))
    for p0 in range(0, pool_pages, step):  # the rows that are there already
        n = min(step, pool_pages - p0)
        for name, x in zip(("k_codes", "k_scale", "k_zero"), encode_keys(rows((n, H, P, d), True), case["k_bits"])):
            planes[name][p0:p0 + n] = x
        for name, x in zip(("v_codes", "v_scale"), encode_values(rows((n, H, P, d), False), case["v_bits"])):
            planes[name][p0:p0 + n] = x
    state.update(planes)
    if case["kind"] == "append":
        # K and V as a model's projection leaves them: slices of one fused tensor
        fused = torch.cat([rows((H, state["total"], d), True), rows((H, state["total"], d), False)]).transpose(0, 1).contiguous()
        state["k"], state["v"] = fused[:, :H], fused[:, H:]
    if case["kind"] == "attention":
        sharp = torch.exp(0.5 * torch.randn(1, QH, 1, generator=g, device=dev)) / (size.mean() * 2)
        state["q"] = (torch.randn(state["total"], QH, d, generator=g, device=dev) * 1.5 * sharp).to(torch.bfloat16)
    if own:  # the pool and the page table as the framework's handles, and the workspace that a serving loop keeps
        import rotated_kv_cache_gb300 as tq

        pool = tq.Cache.from_planes(state["k_codes"], state["k_scale"], state["k_zero"], state["v_codes"], state["v_scale"],
                                    head_dim=d, k_bits=case["k_bits"], v_bits=case["v_bits"], sign_seed=SEED)
        pages = tq.PageTable(table, state["lens"], state["max_len"])
        state.update(pool=pool, pages=pages)
        if case["kind"] == "attention":
            need = tq.tq_paged_attention_workspace_bytes(pool, pages, QH, state["total"], state["max_new"])
            state["workspace"] = torch.empty(need, dtype=torch.uint8, device=dev)
    return state


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
    levels = torch.full_like(hi, 254.0 if bits == 8 else 2.0 ** bits - 1)  # a tensor: divided by, not multiplied by a reciprocal
    scale = (hi - lo) / levels
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


def _places(state, starts, total):
    """Sequence, position, page and slot of every ragged row, the last rows of each sequence."""
    row = torch.arange(total, device="cuda")
    seq = torch.searchsorted(starts[1:].long(), row, right=True)
    pos = row - starts.long()[seq + 1] + state["lens"].long()[seq]
    P = state["case"]["page"]
    return seq, pos, state["table"].long()[seq, pos // P], pos % P


def plain_fetch(state, dtype):
    c = state["case"]
    _, _, page, slot = _places(state, state["starts"], state["total"])
    pick = lambda name: state[name][page, :, slot]  # noqa: E731  [total][H][row]
    return (decode_keys(pick("k_codes"), pick("k_scale"), pick("k_zero"), c["k_bits"]).to(dtype),
            decode_values(pick("v_codes"), pick("v_scale"), c["v_bits"], c["d"]).to(dtype))


def plain_append(state):
    c = state["case"]
    _, _, page, slot = _places(state, state["starts"], state["total"])
    for name, x in zip(("k_codes", "k_scale", "k_zero"), encode_keys(state["k"], c["k_bits"])):
        state[name][page, :, slot] = x
    for name, x in zip(("v_codes", "v_scale"), encode_values(state["v"], c["v_bits"])):
        state[name][page, :, slot] = x


def plain_attention(state):
    c = state["case"]
    H, QH, d, M = c["kv_heads"], c["q_heads"], c["d"], state["max_new"]
    S, L = state["table"].shape[0], state["max_len"]

    def window(name):  # [S][H][max_len][row]
        x = state[name][state["table"].long()]
        return x.transpose(1, 2).flatten(2, 3)[:, :, :L]

    k = decode_keys(window("k_codes"), window("k_scale"), window("k_zero"), c["k_bits"])
    v = decode_values(window("v_codes"), window("v_scale"), c["v_bits"], d)
    seq, pos, _, _ = _places(state, state["starts"], state["total"])
    at = torch.arange(state["total"], device="cuda") - state["starts"].long()[seq]
    q = torch.zeros(S, M, H, QH // H, d, device="cuda")
    q[seq, at] = state["q"].float().unflatten(1, (H, QH // H))
    where = torch.full((S, M), -1, dtype=torch.long, device="cuda")
    where[seq, at] = pos
    hidden = torch.arange(L, device="cuda") > where[..., None]  # [S][M][L]
    s = q.permute(0, 2, 1, 3, 4).flatten(2, 3) @ k.transpose(2, 3) * (1 / math.sqrt(d))  # [S][H][M G][L]
    s = s.unflatten(2, (M, QH // H)).masked_fill_(hidden[:, None, :, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1)[..., None]
    o = (p.flatten(2, 3) @ v).unflatten(2, (M, QH // H)) / torch.where(total == 0, torch.ones_like(total), total)
    return o.permute(0, 2, 1, 3, 4).flatten(2, 3)[seq, at].to(torch.bfloat16)


# ------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    f32 = bool(case.get("f32"))
    if own:
        import rotated_kv_cache_gb300 as tq

        if case["kind"] == "attention":
            return tq.tq_paged_attention(state["pool"], state["pages"], state["starts"], state["q"], state["max_new"],
                                         workspace=state["workspace"])
        if case["kind"] == "append":
            tq.tq_paged_append(state["pool"], state["pages"], state["starts"], state["k"], state["v"])
        return tq.tq_paged_decode(state["pool"], state["pages"], state["starts"], state["total"],
                                  dtype=torch.float32 if f32 else torch.bfloat16)
    if case["kind"] == "attention":
        return plain_attention(state)
    if case["kind"] == "append":
        plain_append(state)
    return plain_fetch(state, torch.float32 if f32 else torch.bfloat16)


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


def _exact_roundtrip(case, k, v):
    """What the appended rows stand for, from the definition in 64 bits (scales and zeros as stored, in fp16)."""
    bits = case["k_bits"]
    x = k.double().unflatten(-1, (-1, 32))
    hi, lo = x.max(-1, keepdim=True).values, x.min(-1, keepdim=True).values
    span = 254 if bits == 8 else 2 ** bits - 1
    s = (hi - lo) / span
    z = ((hi + lo) / 2 / s).round() if bits == 8 else (lo / s).round()
    code = (x / s - z).round().clamp(*((-127, 127) if bits == 8 else (0, span)))
    k_hat = ((code + z.half().double()) * s.half().double()).flatten(-2)
    sg = torch.tensor(sign_vector(case["d"]), dtype=torch.float64, device="cuda")
    cen, bnd = (torch.tensor(t, dtype=torch.float64, device="cuda") for t in codebook(case["v_bits"]))
    y = _butterfly(v.double() * sg).unflatten(-1, (-1, 32))
    rms = y.pow(2).mean(-1, keepdim=True).sqrt()
    cell = torch.zeros_like(y, dtype=torch.long)
    for b in bnd:
        cell += y / (rms + 1e-8) > b
    return k_hat, _butterfly((cen[cell] * rms.half().double()).flatten(-2)) * sg


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        state = prepare(case, seed)
    finally:
        own = kept
    lens, new = lengths(case)
    H, G, P, d = case["kv_heads"], case["q_heads"] // case["kv_heads"], case["page"], case["d"]
    if case["kind"] == "append":
        parts = [_exact_roundtrip(case, state["k"][i:i + 8192], state["v"][i:i + 8192]) for i in range(0, state["total"], 8192)]
        return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])
    out, at = [], 0
    for s, (n, m) in enumerate(zip(lens, new)):
        pos = torch.arange(n - m if case["kind"] == "fetch" else 0, n if m else 0, device="cuda")
        if not m:
            continue
        parts = [_exact_rows(state, state["table"][s].long()[x // P], x % P) for x in pos.split(4096)]
        k, v = (torch.cat([p[i] for p in parts]) for i in (0, 1))
        if case["kind"] == "fetch":
            out.append((k, v))
            continue
        o = torch.empty(m, H * G, d, dtype=torch.float64, device="cuda")
        for h in range(H):
            for i in range(0, m, 512):  # the rows' own positions are n - m + i
                j = min(m, i + 512)
                q = state["q"][at + i:at + j, h * G:(h + 1) * G].double()
                s_ = (q.flatten(0, 1) @ k[:n - m + j, h].T / math.sqrt(d)).unflatten(0, (j - i, G))
                seen = torch.arange(n - m + j, device="cuda")[None] <= torch.arange(n - m + i, n - m + j, device="cuda")[:, None]
                s_ = torch.where(seen[:, None], s_, torch.full_like(s_, -math.inf))
                o[i:j, h * G:(h + 1) * G] = (torch.softmax(s_, -1).flatten(0, 1) @ v[:n - m + j, h]).unflatten(0, (j - i, G))
        out.append(o)
        at += m
    if case["kind"] == "fetch":
        return torch.cat([k for k, _ in out]), torch.cat([v for _, v in out])
    return torch.cat(out)
