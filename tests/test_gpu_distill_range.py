"""The drafter's loss and gradient far out: students that are sure, small temperatures, weights that are no numbers, lists whose
log-sum is not theirs.  The reference works with logarithms in float64, so that no sum in it falls to 0.

Tolerances, with s = 2^-24 (V / 512 + 48) the bound of an fp32 sum's relative error:
  t, rho     t_i = exp(v_i / T - lse) is off by 2^-22 (2 + |ln t_i|) of itself, rho by the sum of these (d); a sum of t
             that is above 1 by no more than lse's rounding is taken as 1, which the gradient's q carries
  loss       t_i (ln t_i - ln q_i): t_i's error times |ln t_i - ln q_i|, and t_i (2^-22 (2 + |ln t_i| + |ln q_i|) + s);
             rho (ln rho - ln sigma): d (2 + |ln rho| + |ln sigma|) + rho (2 s + 2^-22 |ln R|); 2^-23 of it for its rounding
  gradient   a token's share e^(y - ln R) of those outside the list: off by 2^-21 + 2^-22 (|y - ln R| + min(|ln R|, 64)) + 2 s
             of itself, y - ln R of kept statistics by 2^-47 |ln R| more (ln R in two floats); times rho, and d on top; the
             terms q and t as in the loss; then the type's rounding.  What lies below 2^-126 may be 0
"""
import math

import numpy as np
import pytest
import torch

from block_diffusion_draft_dflash_gb300 import _lib
from test_gpu_rows import DEV, LOWEST, f32, f64, held, i32, lists, logits, run_backward, run_distill

pytestmark = pytest.mark.gpu
INF, NAN = math.inf, math.nan
EPS = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8}


def lse(x):
    m = x.max(initial=-INF)
    return m + math.log(np.exp(x - m).sum()) if m > -INF else -INF


def check(z, ids, vals, list_lse, T, loss, stats, grads, dtype, w=1.0):
    """One row against the definition; grads: (gradient, whether it comes from kept statistics) pairs."""
    z, vals, on = np.asarray(z, np.float64), np.asarray(vals, np.float64), np.asarray(ids) >= 0
    T = float(np.float32(T))
    ids = np.asarray(ids)[on]
    ln_t = vals[on] / T - (lse(vals[on] / T) if list_lse is None else list_lse)
    t = np.exp(ln_t)
    rho, total, over = 0.0, 1.0, 0.0
    if list_lse is not None:
        rho, over = max(0.0, 1.0 - t.sum()), max(0.0, t.sum() - 1)
        if over > 2.0 ** -20 + 2.0 ** -23 * abs(list_lse):
            total, over = t.sum(), 0.0
    m = z.max()
    y = (z - m) / T
    other = np.ones(z.size, bool)
    other[ids] = False
    lns, lnr = lse(y), lse(y[other])
    if lnr < -2.0 ** 30:
        lnr = -INF                       # counts as masked
    ln_q = y - lns
    s = 2.0 ** -24 * (z.size / 512 + 48)
    d = 0.0 if list_lse is None else 2.0 ** -22 * (t[t > 0] * (2 + np.abs(ln_t[t > 0]))).sum()
    a = t > 0
    ln_qi, ln_ti, ti = ln_q[ids][a], ln_t[a], t[a]
    want = (ti * (ln_ti - ln_qi)).sum()
    slack = (ti * (2.0 ** -22 * (2 + np.abs(ln_ti)) * (1 + np.abs(ln_ti - ln_qi)) + 2.0 ** -22 * (2 + np.abs(ln_qi)) + s)).sum()
    if rho > 0:
        want += rho * (math.log(rho) - (lnr - lns))
    if lnr > -INF:
        slack += d * (2 + abs(math.log(max(rho, d, 1e-30))) + abs(lnr - lns)) + rho * (2 * s + 2.0 ** -22 * abs(lnr))
    want *= w
    if not abs(want) < float(np.finfo(np.float32).max):
        assert loss == want or loss == math.copysign(INF, want), (loss, want)
    elif lnr == -INF and rho <= d:
        assert abs(loss - want) <= abs(w) * slack + 2.0 ** -23 * abs(want) or loss == INF, (loss, want)     # rho may be 0 or not
    else:
        assert abs(loss - want) <= abs(w) * slack + 2.0 ** -23 * abs(want), (loss, want, abs(w) * slack)
    assert stats[0] == m and abs(stats[1] - lns) <= s + 2.0 ** -23 * abs(lns)
    if lnr == -INF:
        assert stats[2] == -INF and stats[3] == 0
    else:
        assert abs(stats[2] + stats[3] - lnr) <= s + 2.0 ** -22 * min(abs(lnr), 64) + 2.0 ** -23 * 14 + 2.0 ** -47 * abs(lnr)
        assert stats[3] == 0 or lnr < -63
    q = np.exp(ln_q)
    tol = q * (2.0 ** -21 + 2.0 ** -22 * np.abs(np.where(q > 0, ln_q, 0.0)) + s + over) * total
    grad = q * total
    kept = np.zeros(z.size)
    if lnr > -INF:
        share = np.zeros(z.size)
        share[other] = np.exp(y[other] - lnr)
        grad[other] -= (rho * share)[other]
        far = np.where(share > 0, np.abs(y - lnr), 0.0)
        rel = 2.0 ** -21 + 2.0 ** -22 * (far + min(abs(lnr), 64)) + 2 * s
        tol[other] += (share * (rho * rel + d))[other]
        kept[other] = (share * rho * 2.0 ** -47 * abs(lnr))[other]
    grad[ids] -= t
    tol[ids] = tol[ids] + t * 2.0 ** -22 * (3 + np.abs(np.where(t > 0, ln_t, 0.0)))
    for got, from_stats in grads:
        g = grad * (w / T)
        bound = abs(w) / T * (tol + from_stats * kept + 2.0 ** -125) + np.abs(g) * EPS[dtype] * 1.01 + 1e-38
        bad = np.abs(got - g) / bound
        assert (bad <= 1).all(), (bad.max(), got[bad.argmax()], g[bad.argmax()], from_stats)


def teach(z, ids, vals, lses, T, dtype, status=0):
    """Both calls on the rows, every one checked; z float64 [rows][V]."""
    x = held(z, dtype)
    loss, stats, grad, s1 = run_distill(x, ids, vals, lses, T)
    alone = run_distill(x, ids, vals, lses, T, grad=False)[0]
    back, s2 = run_backward(x, ids, vals, lses, T, stats)
    assert s1 == s2 == status and torch.equal(loss, alone)
    hz, hi, hv, hl, hs, hg, hb = f64(x), ids.cpu().numpy(), f64(vals), f64(loss), f64(stats), f64(grad), f64(back)
    for r in range(x.shape[0]):
        check(hz[r], hi[r], hv[r], None if lses is None else float(lses[r]), T, hl[r], hs[r], ((hg[r], False), (hb[r], True)), dtype)
    return hl, hs, hg, hb


# ------------------------------------------------------------------------------ what a list leaves, far below it
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V,K", [(300, 4), (3000, 33), (40000, 4), (40000, 1000)])
@pytest.mark.parametrize("margin,T", [(60.0, 1.0), (90.0, 1.0), (100.0, 1.0), (200.0, 1.0), (1000.0, 1.0), (65536.0, 1.0),
                                      (float(1 << 29), 1.0), (20.0, 0.1), (48.0, 0.3), (2.0 ** 20, 2.0 ** -8), (3.0, 0.001)])
def test_a_margin_between_the_list_and_the_others(dtype, V, K, margin, T):
    """The teacher leaves mass to the others, of which the student has next to none."""
    rng = np.random.default_rng(V + K)
    n = 6
    y = np.zeros((n, V), np.float32)
    at = np.stack([rng.permutation(V)[:K] for _ in range(n)])
    np.put_along_axis(y, at, T * rng.uniform(3.0, 6.0, (n, K)).astype(np.float32), 1)
    z = T * rng.normal(0, 2, (n, V))
    np.put_along_axis(z, at, margin * (1 + 0.01 * rng.random((n, K))), 1)
    for r, upto in ((1, V // 2), (2, 7)):  # the others masked from there on: whole parts of the row have none
        z[r, upto:] = np.where(np.isin(np.arange(upto, V), at[r]), z[r, upto:], -INF)
    ids, vals, lses = lists(y, K, float(np.float32(T)), V)
    teach(z, ids, vals, lses, T, dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T", [0.1, 0.05, 0.01])
def test_a_student_like_its_teacher_at_a_small_temperature(dtype, T):
    V, K, n = 20000, 20, 200
    y = logits(40, n, V)
    x = held(y, dtype)
    ids, vals, lses = lists(f64(x).astype(np.float32), K, float(np.float32(T)), V)
    hl, _, _, _ = teach(f64(x), ids, vals, lses, T, dtype)
    assert np.isfinite(hl).all()


def test_what_lies_beyond_all_statistics_counts_as_masked():
    V, K = 5000, 3
    y = np.zeros((2, V), np.float32)
    y[:, :K] = [6.0, 5.0, 4.0]
    z = np.zeros((2, V))
    z[:, :K] = float(1 << 32)
    z[1, 100:] = -INF
    ids, vals, lses = lists(y, K, 1.0, V)
    hl, hs, hg, hb = teach(z, ids, vals, lses, 1.0, "fp32")
    assert (hl == INF).all() and (hg[:, K:] == 0).all() and (hb[:, K:] == 0).all()


@pytest.mark.parametrize("margin", [30.0, 90.0, 200.0])
def test_gradient_by_differences_far_out(margin):
    V, K, h = 64, 4, 0.0625
    rng = np.random.default_rng(3)
    y, z = (rng.normal(0, 2, (1, V)).astype(np.float32) for _ in range(2))
    ids, vals, lses = lists(y, K, 1.0, V)
    z[0, ids[0].long().cpu().numpy()] = margin + rng.normal(0, 1, K).astype(np.float32)
    grad = f64(run_distill(f32(z), ids, vals, lses, 1.0)[2])[0]
    for j in (0, 5, V - 1, int(ids[0, 0])):
        d = np.zeros((1, V), np.float32)
        d[0, j] = h
        up, down = (f64(run_distill(f32(z + k * d), ids, vals, lses, 1.0, grad=False)[0])[0] for k in (1, -1))
        # the third derivative of a log-sum is at most 1/4: h^2 / 24; losses below 2^8 and their terms are off by 2^-15
        assert abs((up - down) / (2 * h) - grad[j]) <= h * h / 24 + 2.0 ** -15 / h


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


# ------------------------------------------------------------------------------ the lowest number over a small temperature
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("full", [True, False])
@pytest.mark.parametrize("V", [500, 40000])
@pytest.mark.parametrize("T", [1e-9, 1.1e-9, 1.3e-9, 1.7e-12, 2.3e-20, 2.0 ** -100, 1.9e-30])
def test_the_lowest_number_over_a_small_temperature(dtype, full, V, T):
    """v / T is far outside of fp32 for what is masked by the type's lowest number, in lists and in students."""
    n, K = 6, 12
    rng = np.random.default_rng(V)
    y = np.full((n, V), float(np.finfo(np.float32).min), np.float32)
    at = np.stack([rng.permutation(V)[:K] for _ in range(n)])
    np.put_along_axis(y, at[:, :5], np.float32(T) * rng.normal(0, 2, (n, 5)).astype(np.float32), 1)   # five that may come
    z = np.float32(T) * rng.normal(0, 2, (n, V))
    z[1, V // 2:] = LOWEST[dtype]
    z[2, at[2, 5:]] = LOWEST[dtype]        # listed, without mass
    z[3, at[3, 0]] = LOWEST[dtype]         # listed, with mass: an infinite loss
    T = float(np.float32(T))
    ids, vals, lses = lists(y, K, T, V)
    # (fp32 subnormals count as 0 or not: none is among them)
    teach(z, ids, vals, lses if full else None, T, dtype)


# ------------------------------------------------------------------------------ a log-sum that is not the list's
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V", [200, 40000])
@pytest.mark.parametrize("shift", [-0.5, -3.0, 0.25])
def test_a_log_sum_of_another_list(dtype, V, shift):
    """Listed probabilities that sum to more than 1 leave nothing to the others, and the gradient is still the loss's own."""
    K, n = 9, 4
    ids, vals, lses = lists(logits(43, n, V).astype(np.float32), K, 1.0, V)
    teach(logits(44, n, V), ids, vals, lses + shift, 1.0, dtype)


def test_gradient_by_differences_of_a_log_sum_of_another_list():
    V, K, h = 50, 6, 0.0625
    ids, vals, lses = lists(logits(45, 1, V).astype(np.float32), K, 1.0, V)
    lses = lses - 1.0
    z = logits(46, 1, V).astype(np.float32)
    loss, stats, grad, _ = run_distill(f32(z), ids, vals, lses, 1.0)
    back, _ = run_backward(f32(z), ids, vals, lses, 1.0, stats)
    for j in (0, V - 1, int(ids[0, 0]), int(ids[0, 5])):
        d = np.zeros((1, V), np.float32)
        d[0, j] = h
        up, down = (f64(run_distill(f32(z + k * d), ids, vals, lses, 1.0, grad=False)[0])[0] for k in (1, -1))
        for g in (f64(grad)[0], f64(back)[0]):
            # up to e in all: e h^2 / 24; losses below 2^5 are off by 2^-18
            assert abs((up - down) / (2 * h) - g[j]) <= 3 * h * h / 24 + 2.0 ** -18 / h


def test_a_log_sum_that_no_list_has():
    """Probabilities out of fp32's range: the row is left out, with an error."""
    V, K = 300, 5
    ids, vals, lses = lists(logits(47, 2, V).astype(np.float32), K, 1.0, V)
    lses[1] -= 200.0
    z = held(logits(48, 2, V), "fp32")
    loss, stats, grad, status = run_distill(z, ids, vals, lses, 1.0)
    back, _ = run_backward(z, ids, vals, lses, 1.0, stats)
    assert status == -6 and np.isnan(f64(loss)[1]) and np.isnan(f64(stats)[1]).all() and not grad[1].any() and not back[1].any()
    check(f64(z)[0], ids[0].cpu().numpy(), f64(vals)[0], float(lses[0]), 1.0, f64(loss)[0], f64(stats)[0],
          ((f64(grad)[0], False), (f64(back)[0], True)), "fp32")
