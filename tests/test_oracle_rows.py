"""Pins of the float64 restatement of the operators on rows of logits (CPU)."""
import math

import numpy as np
import pytest
import torch

from oracle import rows


def test_order_breaks_ties_by_id_and_leaves_masked_tokens_out():
    assert rows.order([1.0, 3.0, -np.inf, 3.0, -0.0, 0.0]).tolist() == [1, 3, 0, 4, 5]
    assert rows.order([-np.inf] * 3).size == 0


@pytest.mark.parametrize("seed", range(4))
def test_filters_are_the_definitions(seed):
    rng = np.random.default_rng(seed)
    x = np.round(rng.normal(0, 2, 40) * 4) / 4            # many equal logits
    T, k, p, low = 0.7, 12, 0.8, 0.05
    w = np.exp((x - x.max()) / T)
    ids = sorted(range(40), key=lambda i: (-x[i], i))
    first = ids[:k]
    keep = [i for r, i in enumerate(first) if sum(w[j] for j in first[:r]) < p * sum(w[j] for j in first) and w[i] >= low]
    got, prob = rows.kept(x, T, k, p, low)
    assert got.tolist() == keep
    np.testing.assert_allclose(prob, w[keep] / w[keep].sum(), rtol=1e-12)


def test_draw_frequencies_are_the_kept_probabilities():
    rng = np.random.default_rng(5)
    x = rng.normal(0, 2, 30)
    ids, p = rows.kept(x, 1.0, 10, 0.9, 0.0)
    us = (np.arange(20000) + 0.5) / 20000
    drawn = np.array([rows.draw(x, u, top_k=10, top_p=0.9)[0] for u in us])
    for i, pi in zip(ids, p):
        assert abs((drawn == i).mean() - pi) <= 1 / 20000 + 1e-12
    assert rows.draw(x, 0.0)[0] == int(x.argmax())
    assert rows.draw(x, 0.7, temperature=0)[0] == int(x.argmax())
    assert rows.draw([-np.inf, -np.inf], 0.3) == (-1, -math.inf, 0)


def test_top_against_torch():
    x = np.random.default_rng(6).normal(0, 3, 200)
    i, v, lse = rows.top(x, 7, 0.5)
    tv, ti = torch.from_numpy(x).topk(7)
    assert i.tolist() == ti.tolist() and np.array_equal(v, tv.numpy())
    assert abs(lse - float(torch.logsumexp(torch.from_numpy(x) / 0.5, 0))) < 1e-12
    i, v, _ = rows.top([2.0, -np.inf], 3)
    assert i.tolist() == [0, -1, -1] and v[0] == 2.0 and np.isneginf(v[1:]).all()


@pytest.mark.parametrize("full", [False, True])
def test_distill_gradient_by_differences_and_autograd(full):
    rng = np.random.default_rng(7)
    V, K, T = 50, 6, 1.5
    z, y = torch.from_numpy(rng.normal(0, 2, V)), rng.normal(0, 2, V)
    ids, vals, lse = rows.top(y, K, T)
    lse = lse if full else None
    loss, grad, stats = rows.distill(z.numpy(), ids, vals, lse, T, 0.3)
    zt = z.clone().requires_grad_()
    lq = torch.log_softmax(zt / T, -1)
    t = torch.from_numpy(np.exp(vals / T - lse) if full else np.exp(vals / T) / np.exp(vals / T).sum())
    kl = (t * (t.log() - lq[torch.from_numpy(ids).long()])).sum()
    if full:
        other = torch.ones(V, dtype=torch.bool)
        other[torch.from_numpy(ids).long()] = False
        rho = 1 - t.sum()
        kl = kl + rho * (rho.log() - lq[other].logsumexp(0))
    (0.3 * kl).backward()
    assert abs(loss - 0.3 * float(kl)) < 1e-12
    np.testing.assert_allclose(grad, zt.grad.numpy(), atol=1e-12)
    for j in (0, int(ids[0]), V - 1):
        d = np.zeros(V)
        d[j] = 1e-5
        num = (rows.distill(z.numpy() + d, ids, vals, lse, T, 0.3)[0] - rows.distill(z.numpy() - d, ids, vals, lse, T, 0.3)[0]) / 2e-5
        assert abs(num - grad[j]) < 1e-8
    assert stats[0] == z.numpy().max() and abs(grad.sum()) < 1e-12


def test_distill_of_the_teacher_itself_is_zero():
    x = np.random.default_rng(8).normal(0, 2, 64)
    i, v, lse = rows.top(x, 10)
    loss, grad, _ = rows.distill(x, i, v, lse, 1.0)
    assert abs(loss) < 1e-12 and np.abs(grad).max() < 1e-12
