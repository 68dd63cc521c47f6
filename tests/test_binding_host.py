"""The binding's views of tensors on the host: no call is made, so CPU tensors stand in for device ones."""
import copy
import io
import pickle

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
