"""A step of drafted tokens at sizes and in shapes that the small tests do not reach."""
import numpy as np
import pytest
import torch

from test_drafts_gpu import check_verify

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("wide", [1, 3, 7, 40])
def test_verify_rejects_and_accepts_in_turn(cuda, wide, draft, dtype):
    """Level after level `wide` children are rejected and the next one is accepted: what is crossed out at a node counts for
    it alone, whether its children stand among 32 nodes with others' or behind them; some rejected tokens come twice."""
    levels = 200 // (wide + 1)

    def edit(p, r, tokens, parents, u, last, starts):
        rng = np.random.default_rng(wide)
        for s, t in enumerate(parents):
            cur, j = 0, 1
            while j < len(t):
                kids = range(j, min(j + wide + 1, len(t)))
                for c in kids:
                    row, back = starts[s] + cur, c < j + wide
                    x = rng.integers(0, 40) if back else rng.integers(40, 500)
                    t[c], tokens[starts[s] + c] = cur, x
                    u[starts[s] + c] = np.float32(1) - np.float32(2.0 ** -24) if back else 0.0
                    if draft:  # (without draft probabilities the number alone rejects: no token has all of the probability)
                        r[row, x] = r[row, x] if back else 0.0
                        p[row, x] = r[row, x] / 2 if back else p[row, x]
                cur, j = kids[-1], j + wide + 1

    kept = check_verify(cuda, [1 + levels * (wide + 1), 33, 65, 2], 500, draft, dtype, seed=wide, edit=edit)
    assert int(kept[0]) == 1 + levels
    assert cuda.tq_device_error() == 0
