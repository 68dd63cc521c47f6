"""Queries of any finite size on the calls for contiguous caches: scores beyond 2^24 (whose last bit is more than 1) and
near the end of single precision give weights of ones and zeros, not NaN."""
import numpy as np
import pytest
import torch

import oracle
import tq_synth
from tqtest import planes_from_device, to_device_bf16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("power", [0, 26, 116])
@pytest.mark.parametrize("d,kb,M", [(128, 8, 16), (128, 4, 40), (64, 8, 16), (64, 5, 20), (128, 8, 3), (256, 8, 4)])
def test_queries_of_any_size(cuda, power, d, kb, M):
    """The two largest scores of a row are further apart than fp32 sums can err (2^-20 of them; the inputs were looked
    at on the host: no gap below 2^-17), so the weights are those of binary64."""
    H, G, T = 2, 8, 333
    k, v = tq_synth.host_kv(tq_synth.WORKLOADS["sweep"], B=1, H=H, d=d, n=T)
    cache = cuda.Cache(1, H, d, T, k_bits=kb, v_bits=3)
    cuda.tq_encode_append(cache, to_device_bf16(k), to_device_bf16(v), 0)
    w = tq_synth.WORKLOADS["decode"]
    q = np.stack([tq_synth.host_q(w, i, B=1, QH=H * G, d=d) for i in range(M)], axis=1)
    q = (torch.from_numpy(q.view(np.int16)).view(torch.bfloat16).float() * 2.0 ** power).to(torch.bfloat16)
    out = cuda.tq_multi_token_attention(cache, q.cuda(), T)
    want = oracle.attention_multi(planes_from_device(cache), q.view(torch.int16).numpy().view(np.uint16), T)
    assert np.isfinite(want).all()
    assert np.abs(out.cpu().numpy().astype(np.float64) - want).max() < 2e-3
    assert cuda.tq_device_error() == 0
