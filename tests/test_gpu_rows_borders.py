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


@pytest.mark.parametrize("rows", [1, 40, 700])
def test_tokens_of_about_one_unit(rows):
    """A mass is a whole number of 2^-42 of the first token's.  Tokens of 1.63 of these count 2 each, so together they reach
    farther than the sum of their probabilities, whether a row's borders are found with that sum or by a search.

    2^42 units for the first token, 9065 for each of 600 (9065.05), 2 for each of the others.
    """
    V, n_mid, mid = 1 << 20, 600, 9065
    x = torch.full((1, V), -28.625, dtype=torch.bfloat16, device=DEV)
    at = 1000 + 1700 * np.arange(n_mid)
    x[0, at] = -20.0
    x[0, V // 3] = 0.0
    rest = np.setdiff1d(np.arange(V), np.append(at, V // 3))
    order = np.concatenate(([V // 3], at, rest))
    mass = np.concatenate(([0], np.cumsum(np.repeat([1 << 42, mid, 2], [1, n_mid, rest.size]).astype(object)))).tolist()
    x = x.expand(rows, V).contiguous()
    cut = np.asarray(mass, np.float64)                 # exact: below 2^53
    ks = np.arange(rows) % 30 + 1
    u = 1 - 2.0 ** -24 * ks
    for k_p in (0, 9, 20):
        p, n = 1 - 2.0 ** -24 * k_p, V
        if k_p:                                        # tokens before which less than p of all lies
            share = -(-((1 << 24) - k_p) * mass[V] >> 24)
            n = int(np.searchsorted(cut[:-1], share, "left"))
        token, lp, kept, status = run_sample(x, u, [(1.0, 0, p, 0.0)], rows)
        assert status == 0
        for r in range(rows):
            above = ((1 << 24) - int(ks[r])) * mass[n] >> 24          # the first running mass above it
            t = int(np.searchsorted(cut[1:], above, "right"))
            assert (token[r], kept[r]) == (order[t], n), (r, k_p)
