"""Sampling from the largest vocabularies where rows are many (they share one row's memory): one entry
on top, all others equal, so the mass up to v is 1 + v w and the token has a closed form.  The drawn
position times 1 / w is off by the weights' 2^-34 of itself over w V, far below the 0.01 that every
border here is away; log probabilities as in test_sample_gpu."""
import math

import numpy as np
import pytest

from tests import serving as H

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [2 ** 21 + 1, 2 ** 22 + 1, 2 ** 23 + 5, 2 ** 24 - 1])
@pytest.mark.parametrize("rows", [1, 310])
def test_equal_entries(V, dtype, rows):
    torch = pytest.importorskip("torch")
    L = H.lib()
    rng = np.random.default_rng([V, rows])
    for value in (-0.3125, -1.0, -1.6875, -2.5, -3.25, -7.0):
        w = math.exp(value)
        row = torch.full((1, 1, V), value, dtype=H.storage(torch, dtype), device="cuda")
        row[0, 0, 0] = 0.0
        # the smallest v with 1 + v w > u (1 + (V - 1) w)
        u = rng.uniform(0.01, 0.99, (4 * rows, 1)).astype(np.float32)
        at = (u.astype(np.float64) * (1 + (V - 1) * w) - 1) / w
        far = np.abs(at - np.rint(at)) > 0.01
        u, at = u[far][:rows, None], at[far][:rows]
        assert len(u) == rows
        tokens, kept = (torch.full((rows, 1), 77, dtype=torch.int32, device="cuda") for _ in range(2))
        lp, st = torch.zeros((rows, 1), device="cuda"), H.new_status()
        L.spec_sample(row.expand(rows, 1, V), H.dev(u), tokens, st, logprob=lp, kept=kept)
        torch.cuda.synchronize()
        assert H.status(st) == 0 and (kept == V).all()
        assert np.array_equal(tokens.cpu().numpy()[:, 0], np.floor(at).astype(np.int64) + 1), value
        want = value - math.log(1 + (V - 1) * w)
        assert np.abs(lp.double().cpu().numpy() - want).max() <= 2.0 ** -23 * abs(want) + 2.0 ** -31
