"""Draws whose borders follow from whole numbers alone: equal logits weigh the same, so tokens, counts and log-probabilities
are computed here without an exponential."""
import math

import numpy as np
import pytest
import torch

from test_gpu_rows import DEV, held, run_sample

pytestmark = pytest.mark.gpu
INF = math.inf


@pytest.mark.parametrize("rows,V", [(300, 4000), (700, 40000), (200, 40000), (20, 40000)])    # 1, 2, 4 and 8 CTAs search a row
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_equal_logits_under_min_p_alone(dtype, rows, V):
    """More equal tokens than a list holds, all of which min-p keeps: with n of them, token floor(u n) of the order.

    Log-probability: -ln n, from a log2 and a product, 2^-24 (4 |lp| + 24).
    """
    rng = np.random.default_rng(rows)
    x = np.full((rows, V), 0.25)
    x[::3, 1::4] = -INF                    # a mask leaves three of four
    x[1::3] = -7.0
    x = held(x, dtype)
    live = [np.nonzero(row)[0] for row in np.isfinite(x.float().cpu().numpy())]
    for _ in range(30):
        u = rng.random(rows).astype(np.float32)
        token, lp, kept, status = run_sample(x, u, [(1.7, 0, 1.0, 0.3)], rows)
        assert status == 0
        for r, ids in enumerate(live):
            n = ids.size
            assert (token[r], kept[r]) == (ids[int(float(u[r]) * n)], n), r
            assert abs(lp[r] + math.log(n)) <= 2.0 ** -24 * (4 * math.log(n) + 24), r
