"""The calls of a step of drafted tokens on the host: argument refusals (nothing here launches a kernel; the pointers
are never read), rotary frequencies, and models of the identities that the kernels rest on."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest

from conftest import ROOT
from test_abi_host import _struct
from test_devices_host import fake  # noqa: F401  (fixture)
from test_paged_host import _table, _two

NULL, HEAD_DIM, SHAPE, CAPACITY, ALIGN, WORKSPACE = 1, 2, 4, 5, 6, 7
P = 0x100000
REF = ctypes.byref


def test_tree_attention_refusals(tqlib):
    L = tqlib.lib()
    pool, table = _struct(tqlib, batch=12), _table(tqlib)

    def attend(pool=pool, table=table, q=P, qs=(512, 128), heads=4, total=40, max_new=33, masks=2 * P, words=2, out=3 * P, ws=None,
               nbytes=0):
        return L.tq_paged_tree_attention(REF(pool), REF(table), 4 * P, total, max_new, q, _two(*qs), heads, 1.0, masks, words, out,
                                         ws, nbytes, None)

    assert attend(masks=None) == NULL
    assert attend(words=1) == SHAPE and attend(words=0, max_new=1) == SHAPE and attend(words=-1) == SHAPE
    assert attend(words=1, total=32) == attend()  # no sequence has more tokens than there are
    assert attend(heads=3) == SHAPE and attend(max_new=0) == SHAPE and attend(q=None) == NULL and attend(out=None) == NULL
    assert attend(q=P + 4) == ALIGN and attend(out=P + 8) == ALIGN and attend(qs=(512, 4)) == ALIGN
    assert attend(table=_table(tqlib, max_len=129)) == CAPACITY
    assert attend(masks=2 * P + 2) == ALIGN
    assert attend(total=0) == 0
    size = L.tq_paged_tree_attention_workspace_bytes
    assert size(REF(pool), REF(table), 3, 4, 1) == 0 and size(REF(pool), REF(table), 4, 4, 0) == 0


def test_table_update_refusals(tqlib):
    L = tqlib.lib()
    pool, table = _struct(tqlib, batch=12), _table(tqlib)

    def update(pool=pool, table=table, lens=P, new=2 * P, out=3 * P, starts=4 * P, stack=5 * P, cap=12, count=6 * P, count_out=6 * P):
        return L.tq_page_table_update(REF(pool) if pool is not None else None, REF(table) if table is not None else None, lens, new,
                                      out, starts, stack, cap, count, count_out, None)

    assert update(pool=None) == NULL and update(table=None) == NULL
    for name in ("lens", "out", "stack", "count", "count_out"):
        assert update(**{name: None}) == NULL
    assert update(new=None) == NULL  # starts of what
    assert update(cap=0) == SHAPE and update(cap=1 << 31) == SHAPE
    assert update(table=_table(tqlib, max_len=129)) == CAPACITY
    assert update(pool=_struct(tqlib, capacity=1 << 31)) == SHAPE
    for name, at in dict(lens=P, new=2 * P, out=3 * P, starts=4 * P, stack=5 * P, count=6 * P, count_out=7 * P).items():
        assert update(**{name: at + 2}) == ALIGN, name
    assert update(table=_table(tqlib, pages=P + 1)) == ALIGN and update(table=_table(tqlib, seq_lens=2 * P + 2)) == ALIGN
    for at in (P, 2 * P, 3 * P, table.seq_lens):  # what is read after the starts are written, or written over them
        assert update(lens=P, new=2 * P, out=3 * P, starts=at) == SHAPE


def test_layout_and_keep_refusals(tqlib):
    L = tqlib.lib()
    pool, table = _struct(tqlib, batch=12), _table(tqlib)

    def layout(total=40, parents=P, max_new=33, pos=2 * P, slots=3 * P, masks=4 * P, words=2):
        return L.tq_paged_layout(REF(pool), REF(table), 5 * P, total, parents, max_new, pos, slots, masks, words, None)

    assert layout(parents=None) == NULL  # masks of what
    assert layout(max_new=0) == SHAPE and layout(words=1) == SHAPE and layout(words=0, max_new=1) == SHAPE
    assert layout(total=0) == 0 and layout(pos=None, slots=None, masks=None) == 0
    assert layout(total=-1) == SHAPE
    assert layout(parents=P + 2) == ALIGN and layout(pos=2 * P + 2) == ALIGN and layout(masks=4 * P + 2) == ALIGN
    assert layout(slots=3 * P + 4) == ALIGN
    assert layout(pos=P) == SHAPE and layout(masks=P) == SHAPE and layout(pos=4 * P) == SHAPE  # parents of others are read

    def keep(total=40, max_new=8, path=P, stride=8, kept=2 * P, out=3 * P):
        return L.tq_paged_keep(REF(pool), REF(table), 5 * P, total, max_new, path, stride, kept, out, None)

    assert keep(path=None) == NULL and keep(kept=None) == NULL and keep(out=None) == NULL
    assert keep(max_new=0) == SHAPE and keep(stride=7) == SHAPE
    assert keep(out=table.seq_lens) == SHAPE  # the table's own lengths
    assert keep(out=2 * P) == SHAPE  # the counts
    assert keep(path=P + 2) == ALIGN and keep(kept=2 * P + 1) == ALIGN and keep(out=3 * P + 2) == ALIGN


def test_verify_refusals(tqlib):
    L = tqlib.lib()

    def verify(starts=P, seqs=3, total=12, max_new=4, parents=2 * P, tokens=3 * P, vocab=100, dt=1, target=4 * P, ts=100, draft=5 * P,
               ds=100, u=6 * P, last=7 * P, path=8 * P, stride=4, kept=9 * P, nxt=10 * P):
        return L.tq_verify_drafts(starts, seqs, total, max_new, parents, tokens, vocab, dt, target, ts, draft, ds, u, last, path,
                                  stride, kept, nxt, None)

    for name in ("starts", "parents", "tokens", "target", "u", "last", "path", "kept", "nxt"):
        assert verify(**{name: None}) == NULL
    assert verify(seqs=0) == SHAPE and verify(total=-1) == SHAPE and verify(dt=2) == SHAPE
    assert verify(max_new=0) == SHAPE and verify(max_new=5) == SHAPE  # of a path of 4
    assert verify(max_new=tqlib.TQ_MAX_DRAFT + 1, stride=1 << 20) == SHAPE
    assert verify(vocab=0) == SHAPE and verify(vocab=(1 << 30) + 1, ts=1 << 31, ds=1 << 31) == SHAPE
    assert verify(ts=99) == SHAPE and verify(ds=99) == SHAPE
    assert verify(target=4 * P + 2) == ALIGN and verify(draft=5 * P + 2) == ALIGN
    assert verify(target=4 * P + 1, dt=0) == ALIGN
    for name, at in dict(starts=P, parents=2 * P, tokens=3 * P, u=6 * P, last=7 * P, path=8 * P, kept=9 * P, nxt=10 * P).items():
        assert verify(**{name: at + 2}) == ALIGN, name
    assert verify(kept=10 * P) == SHAPE and verify(path=9 * P) == SHAPE and verify(path=10 * P) == SHAPE


def test_rotary_refusals(tqlib):
    L = tqlib.lib()

    def tensor(x=P, out=2 * P, xs=(512, 128), os=(512, 128), heads=4, reserved=0):
        return tqlib._RotaryStruct(x, out, _two(*xs), _two(*os), heads, reserved)

    def rotary(pos=3 * P, tokens=5, d=128, rot=128, freqs=4 * P, dt=0, q=tensor(), k=None):
        return L.tq_rotary(pos, tokens, d, rot, 0, freqs, 1.0, dt, REF(q) if q is not None else None,
                           REF(k) if k is not None else None, None)

    assert rotary(q=None) == NULL and rotary(pos=None) == NULL and rotary(freqs=None) == NULL
    assert rotary(q=tensor(x=None)) == NULL and rotary(k=tensor(out=None)) == NULL
    assert rotary(d=96) == HEAD_DIM
    assert rotary(rot=0) == SHAPE and rotary(rot=130) == SHAPE and rotary(rot=7) == SHAPE and rotary(tokens=-1) == SHAPE
    assert rotary(dt=5) == SHAPE and rotary(q=tensor(heads=0)) == SHAPE and rotary(q=tensor(reserved=1)) == SHAPE
    assert rotary(q=tensor(xs=(-512, 128))) == SHAPE
    assert rotary(q=tensor(x=P + 8)) == ALIGN and rotary(q=tensor(xs=(512, 132))) == ALIGN
    assert rotary(q=tensor(os=(0, 128))) == SHAPE and rotary(q=tensor(os=(512, 64))) == SHAPE  # outputs upon one another
    assert rotary(q=tensor(os=(256, 128))) == SHAPE and rotary(q=tensor(os=(128, 512))) == SHAPE
    assert rotary(q=tensor(out=P, os=(1024, 128))) == SHAPE  # in place with other strides
    assert rotary(tokens=0) == 0
    assert rotary(pos=3 * P + 2) == ALIGN and rotary(freqs=4 * P + 4) == ALIGN


def test_codes_match_the_header(tqlib):
    text = open(f"{ROOT}/include/tq.h").read()
    assert f"#define TQ_DEVICE_ERR_FULL {tqlib.TQ_DEVICE_ERR_FULL}u" in text
    assert f"#define TQ_DEVICE_ERR_TREE {tqlib.TQ_DEVICE_ERR_TREE}u" in text
    assert f"#define TQ_MAX_DRAFT {tqlib.TQ_MAX_DRAFT}\n" in text
    for name, code in (("PLAIN", "none"), ("LINEAR", "linear"), ("NTK", "ntk"), ("YARN", "yarn")):
        assert f"TQ_ROTARY_{name} = {tqlib.ROTARY_SCALING[code]}" in text


def _frequencies(rot, base, scaling, factor, original, fast, slow):
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (rot / max(rot - 2, 1))
    w = base ** (-2 * i / rot)
    if scaling == "linear":
        return w / factor, 1.0
    if scaling == "yarn":
        # turns of pair i in the original context: original w / (2 pi); the ramp runs over whole pair indices
        pair = lambda turns: rot * np.log(original / (2 * np.pi * turns)) / (2 * np.log(base))  # noqa: E731
        lo, hi = max(np.floor(pair(fast)), 0), min(np.ceil(pair(slow)), rot - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 1e-3), 0, 1)
        return (w / factor) * ramp + w * (1 - ramp), 0.1 * np.log(factor) + 1
    return w, 1.0


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
@pytest.mark.parametrize("rot,base,factor,original", [(128, 1e4, 8.0, 4096), (64, 5e5, 2.5, 8192), (2, 1e4, 4.0, 100), (512, 1e6, 1.0, 1)])
def test_rotary_frequencies(tqlib, rot, base, factor, original, scaling):
    got, scale = tqlib.tq_rotary_frequencies(rot, base, scaling, factor, original, 32.0, 1.0)
    want, size = _frequencies(rot, base, scaling, factor, original, 32.0, 1.0)
    assert got.shape == (rot // 2,) and got[0] > 0
    np.testing.assert_allclose(got, want, rtol=1e-14)
    assert abs(scale - size) <= 2.0 ** -24 * size
    if scaling == "ntk" and rot > 2:  # the slowest pair stretched by the factor, the fastest left
        plain = _frequencies(rot, base, "none", 1.0, 1, 1.0, 1.0)[0]
        assert got[0] == plain[0] and abs(got[-1] * factor / plain[-1] - 1) < 1e-13


@pytest.mark.parametrize("original,fast,slow", [(4, 32.0, 1.0), (1, 1.0, 1.0), (4096, 3000.0, 2000.0), (6, 2.0, 1.0)])
def test_yarn_of_pairs_that_all_turn_too_little(tqlib, original, fast, slow):
    """The first pair turns original / (2 pi) times; where that is below `slow` every pair is divided by the factor."""
    assert original / (2 * np.pi) < slow
    got, _ = tqlib.tq_rotary_frequencies(64, 1e4, "yarn", 8.0, original, fast, slow)
    np.testing.assert_allclose(got, 1e4 ** (-2.0 * np.arange(32) / 64) / 8.0, rtol=1e-14)


def test_rotary_frequency_refusals(tqlib):
    bad = lambda *a, **k: pytest.raises((ValueError, tqlib.TQError))  # noqa: E731
    for args in ((3,), (0,), (514,), (64, 1.0), (64, float("nan")), (64, float("inf"))):
        with bad():
            tqlib.tq_rotary_frequencies(*args)
    for kw in (dict(scaling="other"), dict(scaling="linear", factor=0.5), dict(scaling="ntk", factor=float("nan")),
               dict(scaling="yarn", factor=2.0), dict(scaling="yarn", factor=2.0, original_len=100, fast=1.0, slow=2.0),
               dict(scaling="yarn", factor=2.0, original_len=100, slow=0.0)):
        with bad():
            tqlib.tq_rotary_frequencies(64, 1e4, **kw)


def test_binding_refusals(tqlib):
    """Shapes and types that the binding refuses before the library is reached."""
    import torch

    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    f = lambda *s: torch.zeros(*s)  # noqa: E731
    ok = dict(starts=i32(3), parents=i32(4), tokens=i32(4), target=f(4, 7), draft=None, uniforms=f(4), last=f(2), max_new=2)
    for change in (dict(starts=i32(1)), dict(parents=i32(5)), dict(tokens=i32(4).long()), dict(target=f(4, 14)[:, ::2]),
                   dict(target=f(4)), dict(target=f(4, 7).half()), dict(draft=f(4, 6)), dict(draft=f(4, 7).bfloat16()),
                   dict(uniforms=f(3)), dict(uniforms=f(4).double()), dict(last=f(3)), {}):
        with pytest.raises(ValueError):  # (the last one: not on a CUDA device)
            tqlib.tq_verify_drafts(**{**ok, **change})
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    good = dict(positions=i32(4), freqs=torch.zeros(32, dtype=torch.float64), q=q)
    for change in (dict(q=None), dict(q=q[0]), dict(positions=i32(3)), dict(freqs=f(32)), dict(q=q.half()), dict(k=q[:3]),
                   dict(k=q.float()), dict(k_out=q), dict(q=q.transpose(1, 2)), {}):
        with pytest.raises(ValueError):
            tqlib.tq_rotary(**{**good, **change})


@pytest.mark.parametrize("d,kb,vb", [(64, 8, 3), (128, 4, 4), (128, 5, 8), (256, 8, 4), (256, 2, 5), (512, 8, 3)])
def test_calls_are_set_up_on_every_device(tqlib, fake, d, kb, vb):  # noqa: F811
    """As the other calls: what one device is given the next one is, in the same process."""
    cache = tqlib._CacheStruct(d, kb, vb, 2, 64, 0, 32, P, 2 * P, 3 * P, 4 * P, 5 * P, 42)
    table = tqlib._PageTableStruct(6 * P, 7 * P, 1 << 20, 1 << 20, 0, 3, 0)
    q = tqlib._RotaryStruct(8 * P, 9 * P, _two(16 * d, d), _two(16 * d, d), 16, 0)

    def calls():
        out = {}
        for total, new in ((3, 1), (9, 3), (48, 16), (400, 200)):
            size = fake.tq_paged_tree_attention_workspace_bytes(REF(cache), REF(table), 16, total, new)
            out[f"size {new}"] = 0 if size > 0 else -1
            out[f"tree {new}"] = fake.tq_paged_tree_attention(REF(cache), REF(table), 11 * P, total, new, 8 * P, _two(16 * d, d), 16, 1.0,
                                                              12 * P, 7, 9 * P, 10 * P, 1 << 40, None)
        out["update"] = fake.tq_page_table_update(REF(cache), REF(table), P, 2 * P, 3 * P, 4 * P, 5 * P, 64, 6 * P, 6 * P, None)
        out["layout"] = fake.tq_paged_layout(REF(cache), REF(table), 5 * P, 40, P, 33, 2 * P, 3 * P, 4 * P, 2, None)
        out["keep"] = fake.tq_paged_keep(REF(cache), REF(table), 5 * P, 40, 8, P, 8, 2 * P, 3 * P, None)
        for rot in (d, 6):
            out[f"rotary {rot}"] = fake.tq_rotary(3 * P, 5, d, rot, 0, 4 * P, 1.0, 0, REF(q), None, None)
        for dt in (0, 1):
            out[f"verify {dt}"] = fake.tq_verify_drafts(P, 3, 12, 1024, 2 * P, 3 * P, 100, dt, 4 * P, 100, 5 * P, 100, 6 * P, 7 * P, 8 * P,
                                                        1024, 9 * P, 10 * P, None)
        return out

    for dev in (0, 1, 0, 5):
        fake.fake_set_device(dev)
        got = calls()
        assert set(got.values()) == {0}, (dev, got)


def test_outputs_upon_other_tensors_are_refused(tqlib, fake):  # noqa: F811
    """Whole tensors or their ends: where a call would read what it has written, nothing is launched; tensors side by
    side, and those that may be the same, are taken."""
    pool = _struct(tqlib, batch=12)
    S, total, most = 3, 40, 33
    table = _table(tqlib, pages=20 * P, seq_lens=21 * P)  # 4 pages a row
    fake.fake_set_device(0)

    def update(lens=P, new=2 * P, out=3 * P, starts=4 * P, stack=5 * P, count=6 * P, count_out=7 * P):
        return fake.tq_page_table_update(REF(pool), REF(table), lens, new, out, starts, stack, 12, count, count_out, None)

    for kw in ({}, dict(out=P), dict(out=21 * P), dict(count_out=6 * P), dict(starts=2 * P + 4 * S), dict(starts=P - 4 * (S + 1)),
               dict(out=P + 4 * S), dict(stack=20 * P + 48), dict(out=2 * P), dict(lens=21 * P, out=21 * P)):
        assert update(**kw) == 0, kw
    ends = {P: S, 2 * P: S, 3 * P: S, 5 * P: 12, 6 * P: 1, 7 * P: 1, 20 * P: 12, 21 * P: S}  # words of each
    for at, n in ends.items():
        assert update(starts=at) == SHAPE and update(starts=at + 4 * n - 4) == SHAPE and update(starts=at - 4 * S) == SHAPE, at
        if at not in (5 * P,):
            assert update(stack=at) == SHAPE and update(stack=at - 44) == SHAPE and update(stack=at + 4 * n - 4) == SHAPE, at
    assert update(out=P + 4) == SHAPE and update(out=21 * P - 8) == SHAPE  # partly the lengths
    assert update(out=20 * P + 44) == SHAPE and update(out=7 * P) == SHAPE

    def layout(starts=5 * P, parents=P, pos=2 * P, slots=3 * P, masks=4 * P):
        return fake.tq_paged_layout(REF(pool), REF(table), starts, total, parents, most, pos, slots, masks, 2, None)

    for kw in ({}, dict(pos=P + 4 * total), dict(slots=2 * P + 4 * total), dict(masks=P - 8 * total), dict(starts=3 * P + 8 * total)):
        assert layout(**kw) == 0, kw
    for at, n in {P: total, 5 * P: S + 1, 20 * P: 12, 21 * P: S}.items():
        for name, size in (("pos", 4 * total), ("slots", 8 * total), ("masks", 8 * total)):
            for x in (at, (at + 4 * n - 8) // 8 * 8, at - size + 8):
                assert layout(**{name: x}) == SHAPE, (name, at)
    assert layout(pos=3 * P + 8) == SHAPE and layout(masks=3 * P + 8 * total - 8) == SHAPE and layout(pos=4 * P + 8 * total - 4) == SHAPE

    def keep(path=P, kept=2 * P, out=3 * P):
        return fake.tq_paged_keep(REF(pool), REF(table), 5 * P, total, 8, path, 10, kept, out, None)

    for kw in ({}, dict(out=2 * P + 4 * S), dict(out=P + 4 * 28), dict(kept=3 * P + 4 * S)):
        assert keep(**kw) == 0, kw
    for x in (P, P + 4 * 27, 2 * P + 8, 2 * P - 8, 5 * P + 12, 20 * P + 44, 21 * P, 21 * P + 8):
        assert keep(out=x) == SHAPE, hex(x)

    def verify(path=8 * P, kept=9 * P, nxt=10 * P, draft=5 * P):
        return fake.tq_verify_drafts(P, S, total, 12, 2 * P, 3 * P, 100, 1, 4 * P, 120, draft, 100, 6 * P, 7 * P, path, 12, kept, nxt, None)

    last_row = 4 * (39 * 120 + 99)
    for kw in ({}, dict(kept=8 * P + 4 * 36, nxt=8 * P + 4 * 39), dict(path=4 * P + last_row + 4), dict(nxt=2 * P + 4 * total), dict(draft=None)):
        assert verify(**kw) == 0, kw
    for name, size in (("path", 4 * 36), ("kept", 12), ("nxt", 12)):
        for at, n in {P: 16, 2 * P: 160, 3 * P: 160, 4 * P: last_row + 4, 5 * P: 4 * 40 * 100, 6 * P: 160, 7 * P: 12}.items():
            assert verify(**{name: at}) == SHAPE and verify(**{name: at + n - 4}) == SHAPE and verify(**{name: at - size + 4}) == SHAPE, (name, at)
    assert verify(kept=10 * P + 8) == SHAPE and verify(path=9 * P - 4) == SHAPE and verify(nxt=8 * P + 4 * 35) == SHAPE

    def rotary(x=P, out=2 * P, x2=3 * P, out2=4 * P):
        q, k = (tqlib._RotaryStruct(a, b, _two(512, 128), _two(512, 128), 4, 0) for a, b in ((x, out), (x2, out2)))
        return fake.tq_rotary(5 * P, 5, 128, 128, 0, 6 * P, 1.0, 0, REF(q), REF(k), None)

    assert rotary() == 0 and rotary(out=P, out2=3 * P) == 0
    assert rotary(out=3 * P) == SHAPE and rotary(out2=P) == SHAPE and rotary(out2=2 * P) == SHAPE


# ------------------------------------------------------------------ what the kernels rest on
@pytest.mark.parametrize("seed", range(20))
def test_what_is_left_after_rejections_has_one_factor(seed):
    """max(R - M r, 0), taken again and again, normalised each time, is max(p - C r, 0) up to a factor: in fractions."""
    rng = np.random.default_rng(seed)
    n = int(rng.integers(1, 12))
    p, r = ([Fraction(int(x), 1) for x in rng.integers(0, 20, n)] for _ in range(2))
    if not sum(p) or not sum(r):
        return
    p, r = [x / sum(p) for x in p], [x / sum(r) for x in r]
    left, C, M = list(p), Fraction(0), Fraction(1)
    for _ in range(4):
        rest = [max(a - b, 0) for a, b in zip(left, r)]
        C += M
        M = sum(max(a - C * b, 0) for a, b in zip(p, r))
        if not sum(rest):
            assert M == 0
            return
        left = [x / sum(rest) for x in rest]
        assert left == [max(a - C * b, 0) / M for a, b in zip(p, r)]


def test_rotary_reduction_keeps_the_angle():
    """Turns taken off in two parts: positions of 2^31 lose no more than the product's own rounding (2^-53 of the angle)."""
    rng = np.random.default_rng(5)
    two_pi = (Fraction(6.283185307179586), Fraction(2.4492935982947064e-16))
    pi = Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)
    assert abs(two_pi[0] + two_pi[1] - 2 * pi) < Fraction(1, 10 ** 31)
    for _ in range(200):
        t = float(rng.integers(0, 1 << 31)) * float(10.0 ** -rng.uniform(0, 5))
        k = round(Fraction(t * 0.15915494309189535))
        y = float(Fraction(t) - k * two_pi[0])  # a fused multiply-add rounds once
        y = float(Fraction(y) - k * two_pi[1])
        assert abs(Fraction(y) - (Fraction(t) - 2 * k * pi)) < Fraction(1, 2 ** 50)
        assert abs(y) < 3.2
