"""The drafter's loss and gradient far out: weights that are no numbers."""
import math

import numpy as np
import pytest
import torch

from test_gpu_rows import f32, f64, held, lists, logits, run_backward, run_distill

pytestmark = pytest.mark.gpu
INF, NAN = math.inf, math.nan


# ------------------------------------------------------------------------------ weights that are no numbers
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V", [130, 40000])
@pytest.mark.parametrize("w", [NAN, INF, -INF])
def test_a_weight_that_is_no_number_reaches_the_whole_row(dtype, V, w):
    n, K = 5, 8
    ids, vals, lses = lists(logits(41, n, V).astype(np.float32), K, 1.0, V)
    ids[3] = -1                            # a list without entries: others only
    z = logits(42, n, V)
    z[1, ::2] = -INF
    z = held(z, dtype)
    plain = run_distill(z, ids, vals, lses, 1.0)
    weight = f32([1.0, w, w, w, 1.0])
    loss, stats, grad, status = run_distill(z, ids, vals, lses, 1.0, weight=weight)
    back, status2 = run_backward(z, ids, vals, lses, 1.0, plain[1], weight=weight)
    up, status3 = run_backward(z, ids, vals, lses, 1.0, plain[1], grad_loss=weight)
    assert status == status2 == status3 == 0
    hl = f64(loss)
    assert not np.isfinite(hl[1:4]).any() and hl[0] == f64(plain[0])[0] and hl[4] == f64(plain[0])[4]
    for g in (grad, back, up):
        assert not torch.isfinite(g[1:4]).any() and torch.isfinite(g[[0, 4]]).all()
    assert torch.equal(grad[[0, 4]], plain[2][[0, 4]])
