"""Paged cache on the GPU: append and fetch against the contiguous calls (bit
for bit) and the oracle, attention against a plain binary64 implementation."""
import numpy as np
import pytest
import torch

from pagedtest import Batch, check_attention, rows_of

pytestmark = pytest.mark.gpu


def _contiguous(tq, b, s, n=None):
    """Sequence s appended through tq_encode_append into a cache of its own."""
    n = b.lens[s] if n is None else n
    c = tq.Cache(1, b.H, b.d, max(n, 1), k_bits=b.kb, v_bits=b.vb)
    x = [t[s][:n].transpose(0, 1).contiguous()[None].cuda() for t in (b.k, b.v)]
    tq.tq_encode_append(c, x[0], x[1], 0)
    return c


APPENDS = [(128, 8, 3, 64), (128, 4, 3, 16), (128, 5, 8, 48), (64, 8, 4, 32), (64, 4, 2, 16), (64, 2, 3, 80),
           (256, 4, 2, 48), (256, 8, 5, 128), (512, 8, 3, 16), (512, 2, 4, 256)]


@pytest.mark.parametrize("d,kb,vb,page", APPENDS)
def test_append_matches_the_contiguous_append(cuda, d, kb, vb, page):
    """Chunks on top of chunks, ragged, some of one row and some empty: the rows' bytes are those of
    tq_encode_append, and no other row of the pool is written."""
    b = Batch([70, 0, 1, 257, 33, 16], [0] * 6, H=3, d=d, kb=kb, vb=vb, page=page, seed=d + kb)
    pool = b.pool(cuda)
    for t in pool.planes():
        t.fill_(0x5A)
    lens = [0] * 6
    for step in ([1, 0, 1, 100, 16, 15], [69, 0, 0, 156, 17, 0], [0, 0, 0, 1, 0, 1]):
        lens = [a + c for a, c in zip(lens, step)]
        part = lambda rows: torch.cat([x[n - c:n] for x, n, c in zip(rows, lens, step)]).cuda()  # noqa: E731
        starts = b.dev(np.concatenate([[0], np.cumsum(step)]).astype(np.int32))
        cuda.tq_paged_append(pool, b.pages(cuda, lens), starts, part(b.k), part(b.v))
    assert lens == b.lens
    for s, n in enumerate(lens):
        if n:
            want = _contiguous(cuda, b, s)
            for got, ref in zip(rows_of(pool, b.table[s], n), want.planes()):
                assert np.array_equal(got, ref[0, :, :n].cpu().numpy()), s
    written = torch.zeros(b.num_pages, page, dtype=torch.bool)
    for s, n in enumerate(lens):
        for t in range(n):
            written[b.table[s, t // page], t % page] = True
    for t in pool.planes():
        rest = t.transpose(1, 2)[~written.cuda()]
        fill = 0x5A if t.dtype == torch.uint8 else 0x5A
        assert bool((rest == fill).all())
    assert cuda.tq_device_error() == 0


def test_append_strided_views_and_padding(cuda):
    """K and V as slices of one fused projection; tokens behind the last sequence are not read into any page."""
    H, d = 4, 128
    b = Batch([40, 25], [40, 25], H=H, d=d, kb=8, vb=3, page=32, pad_rows=7)
    k, v = b.tokens(b.k, b.new), b.tokens(b.v, b.new)
    k[b.total:] = float("nan")
    fused = torch.cat([k, v], 1).cuda()
    plain, strided = b.pool(cuda), b.pool(cuda)
    starts = b.dev(b.starts)
    cuda.tq_paged_append(plain, b.pages(cuda), starts, k[:b.total].cuda(), v[:b.total].cuda())
    cuda.tq_paged_append(strided, b.pages(cuda), starts, fused[:, :H], fused[:, H:])
    for x, y in zip(plain.planes(), strided.planes()):
        assert torch.equal(x, y)
    # heads before tokens
    hk, hv = (x.transpose(0, 1).contiguous().transpose(0, 1).cuda() for x in (k, v))
    other = b.pool(cuda)
    cuda.tq_paged_append(other, b.pages(cuda), starts, hk, hv)
    for x, y in zip(plain.planes(), other.planes()):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,kb,vb,page", APPENDS)
def test_fetch_matches_the_contiguous_fetch(cuda, d, kb, vb, page, dtype):
    b = Batch([70, 0, 1, 257, 33], [33, 0, 1, 257, 2], H=3, d=d, kb=kb, vb=vb, page=page, seed=d + vb, pad_rows=5)
    pool = b.pool(cuda)
    b.fill(cuda, pool)
    n = b.total + b.pad_rows
    outs = [torch.full((n, b.H, d), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    args = (pool, b.pages(cuda), b.dev(b.starts), n)
    k, v = cuda.tq_paged_decode(*args, dtype=dtype, k_out=outs[0], v_out=outs[1])
    at = 0
    for s, (n_s, m) in enumerate(zip(b.lens, b.new)):
        if m:
            ck, cv = cuda.tq_decode(_contiguous(cuda, b, s), n_s - m, m, dtype=dtype)
            assert torch.equal(k[at:at + m], ck[0].transpose(0, 1)) and torch.equal(v[at:at + m], cv[0].transpose(0, 1))
        at += m
    assert bool((k[b.total:] == 7).all()) and bool((v[b.total:] == 7).all())  # behind the last sequence
    only_k, none = cuda.tq_paged_decode(pool, b.pages(cuda), b.dev(b.starts), b.total, dtype=dtype, want_v=False)
    none2, only_v = cuda.tq_paged_decode(pool, b.pages(cuda), b.dev(b.starts), b.total, dtype=dtype, want_k=False)
    assert none is None and none2 is None
    assert torch.equal(only_k, k[:b.total]) and torch.equal(only_v, v[:b.total])
    assert cuda.tq_device_error() == 0


def _attend(tq, b, QH, seed=1, scale=None, **kw):
    pool = b.pool(tq)
    b.fill(tq, pool)
    q = b.queries(QH, seed)
    out = tq.tq_paged_attention(pool, b.pages(tq), b.dev(b.starts), q.cuda(), max(max(b.new), 1), softmax_scale=scale, **kw)
    check_attention(b, pool, q, out, scale=scale)
    assert tq.tq_device_error() == 0
    return pool, q, out


# decode: lengths around the stages and pages of every kernel, empty slots among them
@pytest.mark.parametrize("d,kb,vb,G,page", [
    (128, 8, 3, 8, 64), (128, 4, 3, 8, 16), (128, 4, 2, 4, 48), (128, 8, 4, 1, 32), (128, 8, 2, 16, 128),
    (128, 4, 4, 12, 96), (128, 5, 3, 8, 32), (128, 2, 8, 3, 16), (64, 8, 3, 8, 64), (64, 4, 4, 5, 16), (64, 8, 2, 16, 80),
    (64, 2, 5, 2, 48), (256, 8, 4, 4, 128), (256, 4, 3, 8, 16), (256, 5, 2, 12, 32), (512, 8, 3, 8, 64), (512, 4, 5, 2, 16),
])
def test_decode_shapes(cuda, d, kb, vb, G, page):
    lens = [1, 0, 15, 16, 17, 63, 64, 65, 96, 97, 128, 129, 300, 1000]
    b = Batch(lens, [min(n, 1) for n in lens], H=2, d=d, kb=kb, vb=vb, page=page, seed=d + G)
    _attend(cuda, b, 2 * G)


@pytest.mark.parametrize("d,kb,vb,G,page,new", [
    (128, 8, 3, 8, 64, 4), (128, 4, 3, 8, 32, 3), (128, 8, 4, 5, 16, 7), (128, 4, 2, 16, 128, 2), (64, 8, 4, 4, 16, 5),
    (64, 4, 3, 8, 48, 9), (256, 8, 3, 4, 32, 4), (256, 4, 4, 16, 64, 3), (512, 8, 3, 2, 16, 6), (128, 5, 5, 3, 80, 8),
])
def test_verification_shapes(cuda, d, kb, vb, G, page, new):
    """Up to `new` new tokens a sequence: fewer in some, as many as rows in others."""
    lens = [1, 2, new, new + 1, 64, 65, 0, 200, 777]
    b = Batch(lens, [min(n, 1 + (i * 3 + new) % new) for i, n in enumerate(lens)], H=2, d=d, kb=kb, vb=vb, page=page, seed=new)
    _attend(cuda, b, 2 * G)


CHUNKS = [
    (128, 8, 3, 8, 64, [300], [300]), (128, 4, 3, 8, 16, [1000, 5, 200], [130, 1, 200]),
    (128, 8, 4, 4, 32, [129, 700, 1, 0, 513], [129, 1, 1, 0, 257]), (64, 8, 4, 4, 32, [640, 90, 1000], [512, 1, 77]),
    (64, 4, 2, 1, 48, [515], [388]), (64, 8, 3, 16, 64, [100, 129], [40, 129]), (128, 5, 2, 3, 16, [444, 100], [150, 99]),
    (128, 2, 5, 8, 256, [300], [100]), (256, 8, 3, 4, 64, [400, 33], [140, 33]), (512, 4, 4, 2, 32, [200], [90]),
    (128, 8, 3, 7, 64, [391], [255]), (128, 8, 8, 8, 64, [257], [256]),
]


@pytest.mark.parametrize("d,kb,vb,G,page,lens,new", CHUNKS)
def test_chunk_shapes(cuda, d, kb, vb, G, page, lens, new):
    b = Batch(lens, new, H=2, d=d, kb=kb, vb=vb, page=page, seed=sum(lens))
    _attend(cuda, b, 2 * G)


@pytest.mark.parametrize("d,kb,vb,G,page,lens,new", CHUNKS)
def test_short_chunks(cuda, d, kb, vb, G, page, lens, new):
    """The same under close bounds: little work in all, which the split kernels take however many columns there are."""
    b = Batch(lens, new, H=2, d=d, kb=kb, vb=vb, page=page, seed=sum(lens))
    b.bound = max(lens)
    _attend(cuda, b, 2 * G)


@pytest.mark.parametrize("d,kb,vb", [(128, 8, 3), (128, 4, 3), (64, 8, 4), (256, 8, 3)])
def test_long_contexts(cuda, d, kb, vb):
    """Many segments a unit, beside sequences far shorter than a segment."""
    lens = [9000, 3, 64, 4097, 1, 2000]
    b = Batch(lens, [1, 1, 2, 1, 1, 4], H=2, d=d, kb=kb, vb=vb, page=64, seed=5)
    _attend(cuda, b, 16)
    b = Batch([5000], [90], H=1, d=d, kb=kb, vb=vb, page=32, seed=6)
    _attend(cuda, b, 8)


def test_many_short_sequences(cuda):
    """More sequences than a warp scans at once, most of a page or less."""
    lens = [(i * 7) % 40 for i in range(200)]
    b = Batch(lens, [min(n, 1 + i % 2) for i, n in enumerate(lens)], H=2, d=128, kb=8, vb=3, page=16, seed=9)
    _attend(cuda, b, 8)


def test_one_step_matches_the_contiguous_attention(cuda):
    """Same rows, same kernels' arithmetic: within one bf16 rounding of tq_decode_attention."""
    b = Batch([777], [1], H=2, d=128, kb=8, vb=3, page=64)
    _, q, out = _attend(cuda, b, 16)
    c = _contiguous(cuda, b, 0)
    want = cuda.tq_decode_attention(c, q.cuda(), 777)
    assert ((out.float() - want).abs() <= 2.0 ** -8 * want.abs() + 2e-3).all()


def test_strided_queries_padding_and_scale(cuda):
    """q as a slice of a fused projection; outputs behind the last sequence stay as they were."""
    b = Batch([100, 30, 200], [5, 1, 130], H=2, d=128, kb=8, vb=3, page=32, pad_rows=6)
    pool = b.pool(cuda)
    b.fill(cuda, pool)
    q = b.queries(8)
    q[b.total:] = float("nan")
    fused = torch.zeros(len(q), 12, 128, dtype=torch.bfloat16)
    fused[:, 2:10] = q
    out = torch.full((len(q), 8, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    cuda.tq_paged_attention(pool, b.pages(cuda), b.dev(b.starts), fused.cuda()[:, 2:10], 130, softmax_scale=0.031, out=out)
    assert bool((out[b.total:] == 3).all())
    check_attention(b, pool, q[:b.total], out[:b.total], scale=0.031)


@pytest.mark.parametrize("d,kb,new", [(128, 8, 4), (64, 4, 3), (128, 8, 150), (64, 8, 300), (256, 8, 20)])
def test_hidden_rows_may_hold_anything(cuda, d, kb, new):
    """NaN and infinities in later rows of the chunk reach only the tokens that see them; rows of a page behind
    the sequence's end reach nobody."""
    b = Batch([new + 50, 77], [new, 1], H=2, d=d, kb=kb, vb=3, page=64, seed=3)
    # one NaN in a key is quantised to the lowest code and leaves its group finite (the codec's clip);
    # the scale written below is what makes a key of kv-head 0 NaN
    b.k[0][50 + new * 3 // 4, 0, 3] = float("nan")
    b.v[0][50 + new // 2, 1, 5] = float("inf")      # a value of kv-head 1
    pool = b.pool(cuda)
    for t in pool.planes():  # what no sequence holds: codes of any kind, scales NaN
        t.fill_(0x7F if t.dtype == torch.uint8 else 0x7FFF)
    b.fill(cuda, pool)
    t = 50 + new * 3 // 4
    pool.k_scale[int(b.table[0, t // 64]), 0, t % 64, 1] = 0x7E00
    q = b.queries(8)
    out = cuda.tq_paged_attention(pool, b.pages(cuda), b.dev(b.starts), q.cuda(), new)
    check_attention(b, pool, q, out)
    nan = (~out.float().isfinite()).any(-1).cpu()  # [token][head]
    assert bool(nan[new * 3 // 4:new, :4].all()) and not bool(nan[:new * 3 // 4, :4].any())
    assert bool(nan[new // 2:new, 4:].all()) and not bool(nan[:new // 2, 4:].any())
    assert not bool(nan[new:].any())


def test_more_new_tokens_than_rows(cuda):
    """Tokens before their sequence's first row: not appended, zeros back, zeros out."""
    b = Batch([3, 0, 40], [3, 0, 4], H=2, d=128, kb=8, vb=3, page=16)
    pool = b.pool(cuda)
    b.fill(cuda, pool)
    before = [t.clone() for t in pool.planes()]
    starts = b.dev(np.array([0, 5, 7, 11], np.int32))  # 5 new tokens of 3 rows, 2 of none
    k = torch.cat([torch.ones(2, 2, 128), b.k[0], torch.ones(2, 2, 128), b.k[2][36:]]).to(torch.bfloat16).cuda()
    v = torch.cat([torch.ones(2, 2, 128), b.v[0], torch.ones(2, 2, 128), b.v[2][36:]]).to(torch.bfloat16).cuda()
    cuda.tq_paged_append(pool, b.pages(cuda), starts, k, v)
    for x, y in zip(before, pool.planes()):
        assert torch.equal(x, y)
    rk, rv = cuda.tq_paged_decode(pool, b.pages(cuda), starts, 11)
    q = b.queries(4, total=11)
    out = cuda.tq_paged_attention(pool, b.pages(cuda), starts, q.cuda(), 5)
    for x in (rk, rv, out):
        assert not bool(x[:2].any()) and not bool(x[5:7].any()) and bool(x[2:5].any())
    check_attention(b, pool, torch.cat([q[2:5], q[7:]]), torch.cat([out[2:5], out[7:]]))


def test_a_long_chunk_with_more_tokens_than_rows(cuda):
    """The same on the wide kernel: 200 new tokens of 150 rows, beside a sequence of its own."""
    b = Batch([150, 90], [150, 1], H=2, d=128, kb=8, vb=3, page=32)
    pool = b.pool(cuda)
    b.fill(cuda, pool)
    q = b.queries(8, total=201)
    out = cuda.tq_paged_attention(pool, b.pages(cuda), b.dev(np.array([0, 200, 201], np.int32)), q.cuda(), 200)
    assert not bool(out[:50].any())
    check_attention(b, pool, q[50:], out[50:])


def test_broadcast_and_reversed_inputs(cuda):
    """One K, V head expanded over all kv-heads (stride 0), as multi-query models have them."""
    b = Batch([40, 70], [40, 70], H=4, d=128, kb=4, vb=4, page=16)
    for x in (b.k, b.v):
        for s in range(2):
            x[s] = x[s][:, :1].expand(-1, 4, -1).contiguous()
    pool, other = b.pool(cuda), b.pool(cuda)
    k, v = b.tokens(b.k, b.new).cuda(), b.tokens(b.v, b.new).cuda()
    cuda.tq_paged_append(pool, b.pages(cuda), b.dev(b.starts), k, v)
    cuda.tq_paged_append(other, b.pages(cuda), b.dev(b.starts), k[:, :1].expand(-1, 4, -1), v[:, :1].expand(-1, 4, -1))
    for x, y in zip(pool.planes(), other.planes()):
        assert torch.equal(x, y)
    # a query head expanded over a group
    q = b.queries(1)
    out = cuda.tq_paged_attention(pool, b.pages(cuda), b.dev(b.starts), q.cuda().expand(-1, 8, -1), 70)
    check_attention(b, pool, q.expand(-1, 8, -1), out)


@pytest.mark.parametrize("scale", [0.0, -0.09, 1e-6, 0.7])
@pytest.mark.parametrize("new", [1, 3, 140])
def test_softmax_scales(cuda, scale, new):
    """Zero (equal weights), negative, tiny and large ones; the last concentrates the weights on a few rows."""
    b = Batch([260, 140], [new, min(new, 140)], H=2, d=128, kb=8, vb=3, page=64, seed=31)
    pool = b.pool(cuda)
    b.fill(cuda, pool)
    q = (b.queries(8).float() * 0.2).to(torch.bfloat16)
    out = cuda.tq_paged_attention(pool, b.pages(cuda), b.dev(b.starts), q.cuda(), new, softmax_scale=scale)
    check_attention(b, pool, q, out, scale=scale)


@pytest.mark.parametrize("new", [2, 130])
def test_sizes_far_from_one(cuda, new):
    """Values of 2^-10 and of 2^12, one sequence each, a row of zeros among them, keys of 2^9 against queries of
    2^-9: powers of two, so that outputs are those of ordinary sizes scaled."""
    ref = Batch([200, 300], [new, new], H=2, d=128, kb=8, vb=3, page=64, seed=41)
    b = Batch([200, 300], [new, new], H=2, d=128, kb=8, vb=3, page=64, seed=41)
    size = (2.0 ** -10, 2.0 ** 12)
    for s in range(2):
        ref.v[s][7], b.v[s][7] = 0, 0
        b.k[s] = b.k[s] * 2.0 ** 9
        b.v[s] = b.v[s] * size[s]
    outs = []
    for x, f in ((ref, 1.0), (b, 2.0 ** -9)):
        pool = x.pool(cuda)
        x.fill(cuda, pool)
        q = x.queries(8) * f
        outs.append(cuda.tq_paged_attention(pool, x.pages(cuda), x.dev(x.starts), q.cuda(), new).float().cpu())
        if f == 1.0:
            check_attention(x, pool, q, outs[0].to(torch.bfloat16))
    # the values' group scales of 2^-10 sizes stay normal fp16 numbers, so their codes are the same; the rms + 1e-8
    # of the index and the fp16 rounding of scales change nothing at powers of two but a code next to a border
    for s in range(2):
        a, c = outs[0][s * new:(s + 1) * new], outs[1][s * new:(s + 1) * new] / size[s]
        assert ((a - c).abs() <= 2 * 2.0 ** -8 * a.abs() + 2 * 2e-3).all()


def test_a_total_that_the_lengths_pass(cuda):
    """Lengths of more than total_len in all, where the workspace is sized by it (4 Mi rows x kv-heads x columns and
    more): recorded, and nothing outside the workspace is touched."""
    b = Batch([700, 800], [200, 300], H=8, d=128, kb=8, vb=3, page=64)
    pool = b.pool(cuda)
    b.fill(cuda, pool)
    q = b.queries(32).cuda()
    exact = cuda.PageTable(b.dev(b.table), b.dev(np.array(b.lens, np.int32)), 800, total_len=1500)
    out = cuda.tq_paged_attention(pool, exact, b.dev(b.starts), q, 300)
    check_attention(b, pool, q.cpu(), out)
    assert cuda.tq_device_error() == 0
    small = cuda.PageTable(b.dev(b.table), b.dev(np.array(b.lens, np.int32)), 800, total_len=600)
    cuda.tq_paged_attention(pool, small, b.dev(b.starts), q, 300)
    assert cuda.tq_device_error() == cuda.TQ_DEVICE_ERR_LENGTH


def test_results_repeat(cuda):
    """No order of arrival enters a result: the same call gives the same bits."""
    b = Batch([3000, 17, 900, 2000], [1, 1, 3, 400], H=2, d=128, kb=4, vb=3, page=32, seed=51)
    pool = b.pool(cuda)
    b.fill(cuda, pool)
    q = b.queries(16).cuda()
    outs = [cuda.tq_paged_attention(pool, b.pages(cuda), b.dev(b.starts), q, 400) for _ in range(5)]
    assert all(torch.equal(outs[0], x) for x in outs[1:])


def test_calls_on_two_streams_at_once(cuda):
    """Two batches over one pool, each on a stream of its own, its workspace of its own."""
    b = Batch([900, 500], [1, 200], H=2, d=128, kb=8, vb=3, page=64, seed=61)
    pool = b.pool(cuda)
    b.fill(cuda, pool)
    q = b.queries(8).cuda()
    want = cuda.tq_paged_attention(pool, b.pages(cuda), b.dev(b.starts), q, 200)
    pages, starts = b.pages(cuda), b.dev(b.starts)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for s, g in zip(streams, got):
            g.append(cuda.tq_paged_attention(pool, pages, starts, q, 200, stream=s))
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(x, want) for x in g)


def test_shared_pages(cuda):
    """Two sequences over one prefix: the same page numbers in both rows of the table."""
    b = Batch([160, 130], [1, 1], H=2, d=128, kb=8, vb=3, page=64)
    b.table[1, :2] = b.table[0, :2]
    for x in (b.k, b.v):
        x[1][:128] = x[0][:128]
    _attend(cuda, b, 8)


def test_a_run_as_a_server_makes_it(cuda):
    """Prompts, then decode steps, a sequence that ends, one that takes over its pages, a verification step:
    every output against the plain implementation, every append read back."""
    H, QH, d, page = 2, 8, 128, 16
    b = Batch([400, 300, 120], [0, 0, 0], H=H, d=d, kb=8, vb=3, page=page, seed=11, spare=4)
    pool = b.pool(cuda)
    lens = [0, 0, 0]

    def step(new):
        nonlocal lens
        lens = [n + m for n, m in zip(lens, new)]
        part = lambda rows: torch.cat([x[n - m:n] for x, n, m in zip(rows, lens, new)]).cuda()  # noqa: E731
        starts, pages = b.dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)), b.pages(cuda, lens)
        cuda.tq_paged_append(pool, pages, starts, part(b.k), part(b.v))
        q = b.queries(QH, seed=sum(lens), total=sum(new))
        out = cuda.tq_paged_attention(pool, pages, starts, q.cuda(), max(new))
        rk, rv = cuda.tq_paged_decode(pool, pages, starts, sum(new), dtype=torch.float32)
        check_attention(b, pool, q, out, lens=lens, new=new)
        at = 0
        for s, m in enumerate(new):
            if m:
                ck, cv = cuda.tq_decode(_contiguous(cuda, b, s, lens[s]), lens[s] - m, m, dtype=torch.float32)
                assert torch.equal(rk[at:at + m], ck[0].transpose(0, 1)) and torch.equal(rv[at:at + m], cv[0].transpose(0, 1))
            at += m

    step([150, 37, 120])
    step([1, 1, 0])
    step([1, 1, 0])
    b.table[2, :4] = b.table[2, :4][::-1].copy()  # sequence 2 ended: another takes its pages, in another order
    b.k[2], b.v[2] = (x[torch.randperm(len(x))] for x in (b.k[2], b.v[2]))
    lens[2] = 0
    step([1, 1, 60])
    step([4, 3, 2])
    assert cuda.tq_device_error() == 0


def test_streams_and_graph_replay(cuda):
    """The same batch through a side stream, and captured once and replayed after the lengths, the table and
    the tokens changed under it."""
    b = Batch([90, 33, 0, 200], [1, 1, 0, 1], H=2, d=128, kb=8, vb=3, page=32, seed=21)
    pool = b.pool(cuda)
    b.fill(cuda, pool)
    q = b.queries(8).cuda()
    pages, starts = b.pages(cuda, max_len=224), b.dev(b.starts)
    want = cuda.tq_paged_attention(pool, pages, starts, q, 1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = cuda.tq_paged_attention(pool, pages, starts, q, 1, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    ws = torch.empty(cuda.tq_paged_attention_workspace_bytes(pool, pages, 8, 3, 1), dtype=torch.uint8, device="cuda")
    knew = torch.zeros(3, 2, 128, dtype=torch.bfloat16, device="cuda")
    vnew, out = knew.clone(), torch.empty_like(want)
    back = [torch.empty(3, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    def step():
        cuda.tq_paged_append(pool, pages, starts, knew, vnew)
        cuda.tq_paged_attention(pool, pages, starts, q, 1, out=out, workspace=ws)
        cuda.tq_paged_decode(pool, pages, starts, 3, k_out=back[0], v_out=back[1])

    take = lambda rows, lens: torch.stack([x[n - 1] for x, n in zip(rows, lens) if n]).cuda()  # noqa: E731
    lens = [90, 33, 0, 200]
    knew.copy_(take(b.k, lens)), vnew.copy_(take(b.v, lens))
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for lens in ([90, 33, 0, 200], [50, 20, 0, 131], [64, 1, 0, 17]):
        pages.seq_lens.copy_(b.dev(np.array(lens, np.int32)))
        knew.copy_(take(b.k, lens)), vnew.copy_(take(b.v, lens))
        g.replay()
        torch.cuda.synchronize()
        check_attention(b, pool, q, out, lens=lens, new=b.new)
    assert cuda.tq_device_error() == 0


def test_bad_pages_and_lengths_are_reported(cuda):
    """A page number outside the pool and a length above the bound: recorded, nothing outside touched, and the
    other sequences' results stand."""
    b = Batch([70, 40], [1, 1], H=2, d=128, kb=8, vb=3, page=32)
    pool = b.pool(cuda)
    b.fill(cuda, pool)
    q = b.queries(8)
    good = b.table.copy()
    for bad in (b.num_pages, -1, 2 ** 31 - 1):
        b.table = good.copy()
        b.table[0, 2] = bad  # holds the new token's row
        pages, starts = b.pages(cuda), b.dev(b.starts)
        before = [t.clone() for t in pool.planes()]
        assert cuda.tq_device_error() == 0
        out = cuda.tq_paged_attention(pool, pages, starts, q.cuda(), 1)
        assert cuda.tq_device_error() == cuda.TQ_DEVICE_ERR_PAGE
        rk, _ = cuda.tq_paged_decode(pool, pages, starts, 2)
        assert cuda.tq_device_error() == cuda.TQ_DEVICE_ERR_PAGE
        new = [torch.stack([x[0][69], x[1][39]]).cuda() for x in (b.k, b.v)]
        cuda.tq_paged_append(pool, pages, starts, *new)
        assert cuda.tq_device_error() == cuda.TQ_DEVICE_ERR_PAGE
        assert not bool(rk[0].any()) and bool(rk[1].any())
        for x, y in zip(before, pool.planes()):
            assert torch.equal(x, y)
        b.table = good
        k1, v1 = b.lens, b.new
        assert k1 == [70, 40] and v1 == [1, 1]
        from pagedtest import ATOL, RTOL, attention64, dequantised
        k, v = dequantised(pool, good[1], 40)
        want = attention64(q[1:2], k, v, 39)
        assert ((out[1:2].cpu().double() - want).abs() <= RTOL * want.abs() + ATOL).all()
    pages = b.pages(cuda, lens=[200, 40], max_len=96)
    cuda.tq_paged_attention(pool, pages, b.dev(b.starts), q.cuda(), 1)
    assert cuda.tq_device_error() & cuda.TQ_DEVICE_ERR_LENGTH
    # starts out of order: more segments than there can be, none of them written outside the workspace
    cuda.tq_paged_attention(pool, b.pages(cuda), b.dev(np.array([0, 2, 0], np.int32)), q.cuda(), 2)
    assert cuda.tq_device_error() & cuda.TQ_DEVICE_ERR_LENGTH


def test_bad_pages_and_lengths_of_long_chunks(cuda):
    """The same for chunks of more than 128 columns, on the kernels that expand their rows first."""
    b = Batch([300, 150], [200, 130], H=2, d=128, kb=8, vb=3, page=32, seed=8)
    pool = b.pool(cuda)
    b.fill(cuda, pool)
    q = b.queries(8)
    good, starts = b.table.copy(), b.dev(b.starts)
    check = lambda out: check_attention(b, pool, q[200:], out[200:], lens=[0, 150], new=[0, 130])  # noqa: E731
    assert cuda.tq_device_error() == 0
    for bad in (b.num_pages, -1, 2 ** 31 - 1):
        b.table = good.copy()
        b.table[0, 3] = bad
        out = cuda.tq_paged_attention(pool, b.pages(cuda), starts, q.cuda(), 200)
        assert cuda.tq_device_error() == cuda.TQ_DEVICE_ERR_PAGE
        b.table = good
        check(out)
    out = cuda.tq_paged_attention(pool, b.pages(cuda, lens=[b.bound + 1, 150]), starts, q.cuda(), 200)
    assert cuda.tq_device_error() == cuda.TQ_DEVICE_ERR_LENGTH
    check(out)
    # starts out of order: the second sequence has no tokens, the first one's results stand
    out = cuda.tq_paged_attention(pool, b.pages(cuda), b.dev(np.array([0, 200, 100], np.int32)), q.cuda(), 200)
    assert cuda.tq_device_error() == cuda.TQ_DEVICE_ERR_LENGTH
    check_attention(b, pool, q[:200], out[:200], new=[200, 0])


def test_long_chunks_strided_padded_and_replayed(cuda):
    """Chunks beside single tokens in one captured graph, q cut out of a wider tensor, rows behind the last sequence
    left as they were; replayed after lengths and starts changed (a chunk for the other sequence, then none)."""
    b = Batch([500, 333, 0, 260], [150, 1, 0, 60], H=2, d=128, kb=4, vb=3, page=48, seed=31)
    pool = b.pool(cuda)
    b.fill(cuda, pool)
    rows, QH = 230, 8
    whole = torch.zeros(rows, QH + 3, 128, dtype=torch.bfloat16, device="cuda")
    q = whole[:, 2:2 + QH]
    pages, starts = b.pages(cuda), b.dev(b.starts)
    ws = torch.empty(cuda.tq_paged_attention_workspace_bytes(pool, pages, QH, rows, 200), dtype=torch.uint8, device="cuda")
    out = torch.empty(rows, QH, 128, dtype=torch.bfloat16, device="cuda")
    step = lambda: cuda.tq_paged_attention(pool, pages, starts, q, 200, out=out, workspace=ws)  # noqa: E731
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i, (lens, new) in enumerate((([500, 333, 0, 260], [150, 1, 0, 60]), ([40, 333, 0, 200], [3, 200, 0, 1]),
                                     ([500, 1, 0, 129], [2, 1, 0, 31]), ([129, 40, 0, 33], [129, 33, 0, 32]))):
        total = sum(new)
        pages.seq_lens.copy_(b.dev(np.array(lens, np.int32)))
        starts.copy_(b.dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)))
        fresh = b.queries(QH, seed=40 + i, total=rows)
        whole.fill_(float("nan"))
        q[:total].copy_(fresh[:total].cuda())
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert bool((out[total:] == 7.0).all())
        check_attention(b, pool, fresh[:total], out[:total], lens=lens, new=new)
    assert cuda.tq_device_error() == 0


def test_many_sequences_some_of_them_long(cuda):
    """More sequences than a warp holds, chunks of every size among them."""
    lens = [(i * 37) % 290 for i in range(70)]
    new = [min(n, (1, 0, 5, 140, 32, 31)[i % 6]) for i, n in enumerate(lens)]
    for d, kb, vb, page in ((128, 8, 3, 32), (64, 4, 4, 16)):
        b = Batch(lens, new, H=2, d=d, kb=kb, vb=vb, page=page, seed=d)
        _attend(cuda, b, 8)


@pytest.mark.parametrize("G", [128, 160])
def test_a_group_of_more_q_heads_than_a_column_group(cuda, G):
    """A single token is a chunk of its own then."""
    b = Batch([300, 1, 0, 140], [1, 1, 0, 2], H=1, d=128, kb=8, vb=3, page=64, seed=G)
    _attend(cuda, b, G)
    b.bound = 300
    _attend(cuda, b, G)


@pytest.mark.parametrize("most,new", [(1, 3), (4, 6), (140, 200), (200, 201)])
def test_more_new_tokens_than_the_bound(cuda, most, new):
    """Starts that pass max_new when a captured call is replayed (one token a sequence, a few, long chunks): recorded,
    the other sequences' results stand, and within the bound nothing is recorded."""
    b = Batch([300, 150, 260], [most, 1, most], H=2, d=128, kb=8, vb=3, page=32, seed=most)
    pool = b.pool(cuda)
    b.fill(cuda, pool)
    rows = new + most + 1
    q = b.queries(8, total=rows)
    pages, starts = b.pages(cuda), b.dev(b.starts)
    ws = torch.empty(cuda.tq_paged_attention_workspace_bytes(pool, pages, 8, rows, most), dtype=torch.uint8, device="cuda")
    ws.fill_(0x11)
    out = torch.zeros(rows, 8, 128, dtype=torch.bfloat16, device="cuda")
    qd = q.cuda()
    step = lambda: cuda.tq_paged_attention(pool, pages, starts, qd, most, out=out, workspace=ws)  # noqa: E731
    step()
    torch.cuda.synchronize()
    assert cuda.tq_device_error() == 0
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    g.replay()
    check_attention(b, pool, q[:b.total], out[:b.total])
    assert cuda.tq_device_error() == 0
    starts.copy_(b.dev(np.array([0, new, new + 1, rows], np.int32)))
    g.replay()
    assert cuda.tq_device_error() == cuda.TQ_DEVICE_ERR_LENGTH
    check_attention(b, pool, q[new:], out[new:], lens=[0, 150, 260], new=[0, 1, most])


def _synth_batch(tq_synth, lens, new, H, d, kb, vb, page, workload="decode"):
    """A batch whose K and V are a workload's: heavy-tailed key channels (log-sigma 1.5), values of Student's t."""
    b = Batch(lens, new, H=H, d=d, kb=kb, vb=vb, page=page)
    bits = lambda x: torch.from_numpy(x.view(np.int16)).view(torch.bfloat16)  # noqa: E731
    for s, n in enumerate(lens):
        k, v = tq_synth.host_kv(tq_synth.WORKLOADS[workload], B=1, H=H, d=d, n=max(n, 1), b_offset=s)
        b.k[s], b.v[s] = (bits(x)[0].transpose(0, 1).contiguous()[:n] for x in (k, v))
    return b


def _synth_queries(tq_synth, total, QH, d):
    w = tq_synth.WORKLOADS["decode"]
    return torch.from_numpy(np.stack([tq_synth.host_q(w, i, B=1, QH=QH, d=d)[0] for i in range(total)]).view(np.int16)) \
        .view(torch.bfloat16)


# Scores of these workloads deviate by 12 and reach 60, so a relative error of the keys is an error of the output 60
# times its size and more: 11 bits of a key (2^-12 of it) would cost 9 times the tolerance.  With keys of two f16 terms
# (2^-23) or exact codes only fp32 sums remain: 16 products of 16 terms into one accumulator, each rounding 2^-23 of
# sums below 2^6 / 0.088, less than 2^-9 / 8 of a score; probabilities and values are rounded as in pagedtest.
@pytest.mark.parametrize("d,kb,vb,page,lens,new", [
    (128, 8, 3, 64, [4096], [128]), (128, 4, 3, 32, [4096], [128]), (128, 5, 2, 48, [1500, 700], [60, 700]),
    (64, 8, 4, 64, [4096], [128]), (64, 4, 3, 16, [3000, 300, 1], [200, 17, 1]), (128, 8, 3, 64, [3000, 900], [1, 4]),
])
def test_heavy_tailed_keys(cuda, d, kb, vb, page, lens, new):
    """The codec's own workload: long chunks keep the keys' precision, as the calls for contiguous caches do."""
    import tq_synth

    b = _synth_batch(tq_synth, lens, new, 2, d, kb, vb, page)
    pool = b.pool(cuda)
    b.fill(cuda, pool)
    q = _synth_queries(tq_synth, b.total, 16, d)
    out = cuda.tq_paged_attention(pool, b.pages(cuda), b.dev(b.starts), q.cuda(), max(new))
    check_attention(b, pool, q, out)
    assert cuda.tq_device_error() == 0


@pytest.mark.parametrize("offset", [64.0, 200.0])
@pytest.mark.parametrize("d,kb,new", [(128, 8, 130), (64, 8, 140), (128, 4, 150), (128, 8, 3)])
def test_keys_with_an_offset(cuda, d, kb, new, offset):
    """One group of 32 key channels far from zero, as keys of trained models have them, against queries of deviation
    3.  The scores' common part, up to 3 * 200 * 32^.5 / 2^3.5, is exact to fp32 sums' 2^-20 of it: below 2^-11."""
    b = Batch([900, 333], [new, min(new, 333)], H=2, d=d, kb=kb, vb=3, page=64, seed=71)
    for s in range(2):
        b.k[s][:, :, 32:64] = (b.k[s][:, :, 32:64].float() + offset).to(torch.bfloat16)
    pool = b.pool(cuda)
    b.fill(cuda, pool)
    q = (b.queries(8).float() * (3 / 1.3)).to(torch.bfloat16)
    out = cuda.tq_paged_attention(pool, b.pages(cuda), b.dev(b.starts), q.cuda(), new)
    check_attention(b, pool, q, out)


@pytest.mark.parametrize("d,kb,new", [(128, 8, 150), (64, 4, 300), (128, 8, 4), (256, 8, 20)])
def test_hidden_rows_may_be_huge(cuda, d, kb, new):
    """Finite keys of 2^32 and values of 2^16 in a later row of the chunk change nothing for the tokens before it,
    rows of ordinary and of tiny keys (2^-20) in the same 128 among them."""
    b = Batch([new + 50, 77], [new, 1], H=2, d=d, kb=kb, vb=3, page=64, seed=3)
    for t in range(50, 50 + new, 7):
        b.k[0][t] = b.k[0][t] * 2.0 ** -20
    pool = b.pool(cuda)
    b.fill(cuda, pool)
    at = 50 + new * 3 // 4
    row = (int(b.table[0, at // 64]), slice(None), at % 64)
    q = b.queries(8)
    args = (pool, b.pages(cuda), b.dev(b.starts), q.cuda(), new)
    plain = cuda.tq_paged_attention(*args)
    check_attention(b, pool, q, plain)
    pool.k_scale[row], pool.k_zero[row], pool.v_scale[row] = 0x7BFF, 0x7BFF, 0x7BFF  # 65504
    out = cuda.tq_paged_attention(*args)
    seen = new * 3 // 4
    keep = torch.ones(len(q), dtype=torch.bool)
    keep[seen:new] = False
    # the tokens before the row: as without it, to the tolerance against the plain implementation
    check_attention(b, pool, q[:seen], out[:seen], lens=[50 + seen, 0], new=[seen, 0])
    assert torch.equal(out[new:], plain[new:])
    assert bool(out[seen:new].float().isfinite().all())
    assert cuda.tq_device_error() == 0


@pytest.mark.parametrize("d,kb,vb,new", [(128, 8, 3, 150), (64, 8, 4, 300), (128, 4, 3, 140), (128, 8, 3, 3)])
def test_far_outliers_that_every_token_sees(cuda, d, kb, vb, new):
    """Rows with keys of up to 2^20 that all queries point away from: no weight of theirs is left, and the other rows
    of their 128 keep their precision; rows with values of 2^-14 beside them."""
    b = Batch([new + 400, 200], [new, min(new, 200)], H=2, d=d, kb=kb, vb=vb, page=64, seed=9)
    way = np.where(np.arange(d) % 2, 1.0, -1.0).astype(np.float32)
    q = b.queries(8).float()
    q = q + torch.from_numpy(way) * (4.0 - (q * torch.from_numpy(way)).mean(-1, keepdim=True))  # mean along `way`: 4
    q = q.to(torch.bfloat16)
    for s in range(2):
        for t, size in ((3, 2.0 ** 20), (64, 2.0 ** 14), (150, 2.0 ** 18)):
            b.k[s][t] = (torch.from_numpy(-size * way) * (1 + 0.25 * torch.rand(2, 1))).to(torch.bfloat16)
        b.v[s][8:16] = b.v[s][8:16] * 2.0 ** -14
    pool = b.pool(cuda)
    b.fill(cuda, pool)
    out = cuda.tq_paged_attention(pool, b.pages(cuda), b.dev(b.starts), q.cuda(), new)
    check_attention(b, pool, q, out)
    assert cuda.tq_device_error() == 0


def test_values_of_very_unlike_sizes(cuda):
    """Values of 2^-14 (group rms the smallest normal fp16 numbers) in the rows that tokens of a chunk see, 65504 in a
    row of the same 128 that they do not: f16 weights and values of exponents of their own keep 2^-12 of each."""
    new = 150
    b = Batch([new + 20], [new], H=2, d=128, kb=8, vb=3, page=64, seed=12)
    size = 2.0 ** -13
    b.v[0] = (b.v[0].float() * size).to(torch.bfloat16)
    pool = b.pool(cuda)
    b.fill(cuda, pool)
    at, seen = 20 + 120, 120
    pool.v_scale[int(b.table[0, at // 64]), :, at % 64] = 0x7BFF
    q = b.queries(8)
    out = cuda.tq_paged_attention(pool, b.pages(cuda), b.dev(b.starts), q.cuda(), new)
    from pagedtest import ATOL, RTOL, attention64, dequantised
    k, v = dequantised(pool, b.table[0], 20 + new)
    want = attention64(q[:seen], k[:, :20 + seen], v[:, :20 + seen], 20)
    err = (out[:seen].cpu().double() - want).abs() - RTOL * want.abs()
    assert float(err.max()) <= ATOL * size, float(err.max()) / size


def test_more_long_chunks_than_the_workspace_expands(cuda):
    """14 chunks over 131072 rows of 8 kv-heads each (one prefix of 512 rows, repeated, so that no memory is needed for
    them): 11 GiB expanded, of which the workspace holds 8.  All against the plain implementation, whose softmax counts
    every row of the prefix as often as it is seen."""
    S, H, d, P, n, new, QH = 14, 8, 128, 128, 131072, 20, 64
    b = Batch([512], [0], H=H, d=d, kb=4, vb=2, page=P, spare=0, seed=77)
    pool = b.pool(cuda)
    b.fill(cuda, pool)
    order = b.table[0, :4]
    table = b.dev(np.tile(order, (S, n // 512)).astype(np.int32))
    lens = [n - 37 * s for s in range(S)]
    pages = cuda.PageTable(table, b.dev(np.array(lens, np.int32)), n)
    new_of = [new - (s % 3) for s in range(S)]
    starts = np.concatenate([[0], np.cumsum(new_of)]).astype(np.int32)
    q = b.queries(QH, total=int(starts[-1]))
    need = cuda.tq_paged_attention_workspace_bytes(pool, pages, QH, len(q), new)
    assert 8 << 30 <= need < 9 << 30
    out = cuda.tq_paged_attention(pool, pages, b.dev(starts), q.cuda(), new).cpu().double()
    assert cuda.tq_device_error() == 0
    from pagedtest import ATOL, RTOL, dequantised
    k, v = (torch.from_numpy(x).double() for x in dequantised(pool, order, 512))
    worst = 0.0
    for s in range(S):
        for i in (0, new_of[s] // 2, new_of[s] - 1):
            seen = lens[s] - new_of[s] + i + 1
            times = torch.tensor([(seen - r + 511) // 512 for r in range(512)], dtype=torch.float64)
            x = q[starts[s] + i].double().view(H, QH // H, d)
            p = torch.softmax(torch.einsum("hgd,hnd->hgn", x, k) * d ** -0.5 + times.log(), -1)
            want = torch.einsum("hgn,hnd->hgd", p, v).reshape(QH, d)
            worst = max(worst, float(((out[starts[s] + i] - want).abs() - RTOL * want.abs()).max()))
    assert worst <= ATOL, worst


@pytest.mark.parametrize("power", [26, 118])
@pytest.mark.parametrize("d,kb,new", [(128, 8, 1), (128, 4, 3), (128, 8, 140), (64, 8, 300), (256, 5, 4), (512, 8, 2)])
def test_scores_of_any_size(cuda, power, d, kb, new):
    """Queries of 2^26 and 2^118: scores whose last bits are 8 and 2^100, and weights of ones and zeros; finite as long
    as the scores are."""
    b = Batch([260, 200], [new, min(new, 200)], H=2, d=d, kb=kb, vb=3, page=64, seed=91)
    pool = b.pool(cuda)
    b.fill(cuda, pool)
    q = (b.queries(8).float() * 2.0 ** power).to(torch.bfloat16)
    for scale in (None, -0.05):
        out = cuda.tq_paged_attention(pool, b.pages(cuda), b.dev(b.starts), q.cuda(), new, softmax_scale=scale)
        check_attention(b, pool, q, out, scale=scale)
    c = _contiguous(cuda, b, 0)
    for s in (None, 0.125):  # and the calls on a contiguous cache
        one = cuda.tq_decode_attention(c, q[new - 1:new].cuda(), 260, softmax_scale=s)
        same = cuda.tq_paged_attention(pool, b.pages(cuda), b.dev(b.starts), q.cuda(), new, softmax_scale=s)
        assert ((same[new - 1].float() - one[0]).abs() <= 2.0 ** -8 * one[0].abs() + 2e-3).all()


@pytest.mark.parametrize("power", [-12, -14, -16])
@pytest.mark.parametrize("d,kb,vb,new", [(128, 8, 3, 1), (128, 4, 3, 3), (64, 8, 4, 1), (256, 8, 3, 2), (512, 8, 3, 1), (128, 5, 5, 4)])
def test_small_values(cuda, power, d, kb, vb, new):
    """Values of 2^power: a weight times a group's rms is one f16 number, within 2^-12 of it or 2^-25, whichever is
    more.  Over n rows the second is an independent error of at most 2^-25 |centroid|, |centroid| < 3.3 and 1 in the
    mean square, uniform: rms 2^-25 / 3^.5 n^.5 of a sum of weights that is 1 at least, and the un-rotation keeps the
    rms; six deviations are 2^-25 * 3.5 n^.5."""
    n = 700
    b = Batch([n, 40], [new, new], H=2, d=d, kb=kb, vb=vb, page=64, seed=55)
    for s in range(2):
        b.v[s] = (b.v[s].float() * 2.0 ** power).to(torch.bfloat16)
    pool = b.pool(cuda)
    b.fill(cuda, pool)
    q = b.queries(8)
    out = cuda.tq_paged_attention(pool, b.pages(cuda), b.dev(b.starts), q.cuda(), new).cpu().double()
    from pagedtest import ATOL, RTOL, attention64, dequantised
    for s in range(2):
        k, v = dequantised(pool, b.table[s], b.lens[s])
        want = attention64(q[s * new:(s + 1) * new], k, v, b.lens[s] - new)
        err = (out[s * new:(s + 1) * new] - want).abs() - RTOL * want.abs()
        assert float(err.max()) <= ATOL * 2.0 ** power + 3.5 * b.lens[s] ** 0.5 * 2.0 ** -25


@pytest.mark.parametrize("d,kb,vb,H,page,rows", [(128, 8, 3, 2, 64, 1 << 26), (64, 4, 2, 1, 16, (1 << 31) + 4096)])
def test_pages_far_into_a_large_pool(cuda, d, kb, vb, H, page, rows):
    """Planes of more than 2^32 bytes, and a pool of more than 2^31 rows: append, fetch and attention of every kind at
    its last pages, the same as in a small pool."""
    per_row = d * kb // 8 + d * vb // 8 + 3 * (d // 32) * 2
    if torch.cuda.mem_get_info()[0] < rows * per_row + (8 << 30):
        torch.cuda.empty_cache()
        if torch.cuda.mem_get_info()[0] < rows * per_row + (8 << 30):
            pytest.skip("not enough device memory")
    lens = [300, 17, 0, 200, 64]
    small = Batch(lens, [1, 1, 0, 1, 1], H=H, d=d, kb=kb, vb=vb, page=page, seed=13, spare=0)
    pool = small.pool(cuda)
    small.fill(cuda, pool)
    big = Batch(lens, [1, 1, 0, 1, 1], H=H, d=d, kb=kb, vb=vb, page=page, seed=13, spare=0)
    pages = rows // (H * page)
    big.table = big.table + (pages - big.num_pages)
    far = cuda.Cache(pages, H, d, page, k_bits=kb, v_bits=vb)
    big.fill(cuda, far)
    for new in ([1, 1, 0, 1, 1], [4, 3, 0, 1, 2], [140, 1, 0, 150, 64]):
        starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        q = small.queries(8 * H, total=int(starts[-1]))
        outs = [cuda.tq_paged_attention(p, b.pages(cuda), b.dev(starts), q.cuda(), max(new)) for b, p in ((small, pool), (big, far))]
        backs = [cuda.tq_paged_decode(p, b.pages(cuda), b.dev(starts), len(q)) for b, p in ((small, pool), (big, far))]
        check_attention(small, pool, q, outs[0], new=new)
        check_attention(small, pool, q, outs[1], new=new)
        for x, y in zip(*backs):
            assert torch.equal(x, y)
    assert cuda.tq_device_error() == 0
    del far
    torch.cuda.empty_cache()
