"""The binding's views of tensors on the host: no call is made, so CPU tensors stand in for device ones."""
import copy
import io
import pickle

import pytest
import torch


def _cache(tq, **kw):
    return tq.Cache(3, 2, 64, 32, device="cpu", **kw)


def _addresses(cache):
    s = cache.struct()
    return [s.k_codes, s.k_scale, s.k_zero, s.v_codes, s.v_scale]


def test_a_used_cache_copies_and_pickles(tqlib):
    """What works on a fresh cache works on one that calls were made with."""
    c = _cache(tqlib, v_bits=4, sign_seed=7)
    c.k_codes.random_(0, 256)
    c.struct()
    other = copy.deepcopy(c)
    back = pickle.loads(pickle.dumps(c))
    buf = io.BytesIO()
    torch.save(c, buf)
    buf.seek(0)
    for x in (other, back, torch.load(buf, weights_only=False), copy.copy(c)):
        assert (x.batch, x.num_kv_heads, x.head_dim, x.capacity, x.v_bits, x.sign_seed) == (3, 2, 64, 32, 4, 7)
        assert all(torch.equal(a, b) for a, b in zip(x.planes(), c.planes()))
        assert _addresses(x) == [t.data_ptr() for t in x.planes()]


def test_a_cache_follows_its_planes(tqlib):
    """A plane whose storage is replaced in place is passed at its new address."""
    c = _cache(tqlib)
    before = _addresses(c)
    assert before == [t.data_ptr() for t in c.planes()]
    kept = [t.detach() for t in c.planes()]  # (the first storages live on, so that no new one takes their place)
    for name in ("k_codes", "k_scale", "k_zero", "v_codes", "v_scale"):
        t = getattr(c, name)
        t.data = t.clone()
        assert _addresses(c) == [t.data_ptr() for t in c.planes()]
    assert not set(before) & set(_addresses(c)) and [t.data_ptr() for t in kept] == before
    c.v_codes.set_(c.v_codes.clone())
    assert _addresses(c) == [t.data_ptr() for t in c.planes()]
    c.v_scale = c.v_scale.clone()
    c.sign_seed = 9
    assert _addresses(c) == [t.data_ptr() for t in c.planes()] and c.struct().sign_seed == 9
    part = c.batch_slice(1, 2)
    assert _addresses(part) == [t[1:].data_ptr() for t in c.planes()] and part.struct().batch == 2


def test_from_planes_takes_the_planes_it_is_given(tqlib):
    kinds = [(32, torch.uint8), (2, torch.float16), (2, torch.int16), (24, torch.uint8), (2, torch.float16)]
    planes = [torch.zeros(4, 3, 48, n, dtype=t) for n, t in kinds]
    c = tqlib.Cache.from_planes(*planes, head_dim=64, k_bits=4, v_bits=3, sign_seed=5)
    s = c.struct()
    assert (s.head_dim, s.k_bits, s.v_bits, s.num_kv_heads, s.batch, s.capacity, s.sign_seed) == (64, 4, 3, 3, 4, 48, 5)
    assert _addresses(c) == [t.data_ptr() for t in planes]


def _table(tq, monkeypatch, pages, lens, *a, **kw):
    monkeypatch.setattr(tq, "_require_cuda", lambda *t: None)
    return tq.PageTable(pages, lens, *a, **kw)


def test_a_page_table_follows_its_tensors_and_bounds(tqlib, monkeypatch):
    """Bounds set later, and tensors whose storage is replaced in place, reach the library."""
    pool = _cache(tqlib)  # pages of 32 rows
    pages, lens = torch.zeros(2, 5, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    t = _table(tqlib, monkeypatch, pages, lens, page_size=32)
    s = t.struct(pool)
    assert (s.pages, s.seq_lens, s.stride, s.max_len, s.total_len, s.num_seqs) == (
        pages.data_ptr(), lens.data_ptr(), 5, 160, 0, 2)
    t.max_len, t.total_len = 96, 128
    s = t.struct(pool)
    assert (s.max_len, s.total_len) == (96, 128)
    t.max_len = 161
    with pytest.raises(ValueError):
        t.struct(pool)
    t.max_len = 64
    old = (pages.detach(), lens.detach())
    pages.data, lens.data = torch.ones(2, 9, dtype=torch.int32)[:, :3], torch.ones(2, dtype=torch.int32)
    s = t.struct(pool)
    assert (s.pages, s.seq_lens, s.stride, s.num_seqs, s.max_len) == (pages.data_ptr(), lens.data_ptr(), 9, 2, 64)
    t.max_len = 97  # three pages of 32 hold 96
    with pytest.raises(ValueError):
        t.struct(pool)
    t.max_len = 96
    assert t.struct(pool).max_len == 96 and old[0].shape == (2, 5)
    # what a table is refused for when it is made, it is refused for later
    lens.data = torch.ones(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        t.struct(pool)
    lens.data = torch.ones(2, dtype=torch.int32)
    pages.data = torch.zeros(3, 2, dtype=torch.int32).t()
    with pytest.raises(ValueError):
        t.struct(pool)


def test_a_used_page_table_copies_and_pickles(tqlib, monkeypatch):
    pool = _cache(tqlib)
    t = _table(tqlib, monkeypatch, torch.arange(6, dtype=torch.int32).view(2, 3), torch.tensor([7, 9], dtype=torch.int32), 64,
               total_len=16)
    t.struct(pool)
    for x in (copy.deepcopy(t), pickle.loads(pickle.dumps(t)), copy.copy(t)):
        s = x.struct(pool)
        assert (s.pages, s.seq_lens, s.max_len, s.total_len) == (x.pages.data_ptr(), x.seq_lens.data_ptr(), 64, 16)
        assert torch.equal(x.pages, t.pages) and torch.equal(x.seq_lens, t.seq_lens)
