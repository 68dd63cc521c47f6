"""The library's host code against a stand-in for the CUDA runtime (tests/helpers/fake_cudart.c): what it sets up
on one device it sets up on the next one, in the same process."""
import ctypes
import os
import subprocess

import pytest

from conftest import ROOT


@pytest.fixture()
def fake(tqlib, tmp_path):
    """The library's objects linked with the stand-in, nothing set up yet."""
    from rotated_kv_cache_gb300 import build

    objs = [os.path.join(build.OUT_DIR, os.path.basename(s) + ".o") for s in build.sources()]
    if not all(os.path.exists(o) and os.path.getmtime(o) <= os.path.getmtime(build.LIB) for o in objs):
        build.build(force=True)
    obj, so = str(tmp_path / "fake.o"), str(tmp_path / "libtq_fake.so")
    subprocess.run(["gcc", "-O1", "-fPIC", "-c", os.path.join(ROOT, "tests", "helpers", "fake_cudart.c"), "-o", obj], check=True)
    subprocess.run(["g++", "-shared", "-Wl,--no-undefined", "-Wl,-Bsymbolic", "-o", so, *objs, obj], check=True)
    lib = ctypes.CDLL(so)
    real = tqlib.lib()
    for name in tqlib.EXPORTS:
        getattr(lib, name).argtypes = getattr(real, name).argtypes
        getattr(lib, name).restype = getattr(real, name).restype
    return lib


def _calls(tq, lib, d, kb, vb):
    """One of each call whose kernels need a set-up, on made-up addresses; the statuses by name."""
    page, H, QH, P = 32, 2, 16, 0x100000
    cache = tq._CacheStruct(d, kb, vb, H, 64, 0, page, P, 2 * P, 3 * P, 4 * P, 5 * P, 42)
    table = tq._PageTableStruct(6 * P, 7 * P, 4, 128, 0, 3, 0)
    ref, two, three = ctypes.byref, (ctypes.c_int64 * 2)(2 * d, d), (ctypes.c_int64 * 3)(page * d * H, page * d, d)
    big = 1 << 40
    out = dict(append=lib.tq_encode_append(ref(cache), 8 * P, three, 9 * P, three, 0, page, None),
               decode=lib.tq_decode(ref(cache), 0, page, 0, 8 * P, 9 * P, None),
               attention=lib.tq_decode_attention(ref(cache), 8 * P, QH, page, 1.0, 9 * P, 10 * P, big, None),
               chunk=lib.tq_multi_token_attention(ref(cache), 8 * P, QH, 20, page, 1.0, 9 * P, 10 * P, big, None),
               few=lib.tq_multi_token_attention(ref(cache), 8 * P, QH, 3, page, 1.0, 9 * P, 10 * P, big, None),
               unrotate=lib.tq_unrotate(d, 42, 1, 8 * P, 100, 1, 9 * P, None),
               paged_append=lib.tq_paged_append(ref(cache), ref(table), 11 * P, 3, 8 * P, two, 9 * P, two, None),
               paged_decode=lib.tq_paged_decode(ref(cache), ref(table), 11 * P, 3, 0, 8 * P, 9 * P, None))
    qs = (ctypes.c_int64 * 2)(QH * d, d)
    long = tq._PageTableStruct(6 * P, 7 * P, 1 << 20, 1 << 20, 0, 3, 0)
    for name, t, total, new in (("paged_step", table, 3, 1), ("paged_few", table, 9, 3), ("paged_chunk", long, 400, 200)):
        size = lib.tq_paged_attention_workspace_bytes(ref(cache), ref(t), QH, total, new)
        out[name + " size"] = 0 if size > 0 else -1
        out[name] = lib.tq_paged_attention(ref(cache), ref(t), 11 * P, total, new, 8 * P, qs, QH, 1.0, 9 * P, 10 * P, big, None)
    return out


@pytest.mark.parametrize("d,kb,vb", [(64, 8, 3), (128, 8, 3), (128, 4, 4), (128, 5, 8), (256, 8, 3), (256, 8, 4), (256, 5, 5),
                                     (512, 8, 3), (512, 4, 2)])
def test_every_call_is_set_up_on_every_device(tqlib, fake, d, kb, vb):
    for dev in (0, 1, 0, 5):
        fake.fake_set_device(dev)
        assert set(_calls(tqlib, fake, d, kb, vb).values()) == {0}, (dev, _calls(tqlib, fake, d, kb, vb))
    # and once a device: calls made again on any of them ask for nothing but what the chunk kernels ask every time
    fake.fake_set_device(1)
    before = fake.fake_queries()
    _calls(tqlib, fake, d, kb, vb)
    each = fake.fake_queries() - before
    assert each <= 2
    for dev in (0, 5):
        fake.fake_set_device(dev)
        before = fake.fake_queries()
        _calls(tqlib, fake, d, kb, vb)
        assert fake.fake_queries() - before == each


@pytest.mark.parametrize("d", [64, 128, 256, 512])
def test_widths_follow_one_another(tqlib, fake, d):
    """Kernels that serve several widths keep the opt-in of the largest, whichever was asked for last."""
    for kb, vb in ((8, 8), (2, 2), (8, 8), (5, 4), (4, 2), (8, 5), (8, 8)):
        assert set(_calls(tqlib, fake, d, kb, vb).values()) == {0}, (kb, vb)
