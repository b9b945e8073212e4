"""Operators on rows of logits (draws, largest logits, distillation) against their float64 oracle.

Whole numbers (tokens, counts, ids) have to be the oracle's: a border is missed where two masses that it compares lie
within 2^-34 of each other, about once in 10^7 rows here.  Tolerances of the rest:
  logprob   log1p(x) with x off by 3 * 2^-24 of itself, or a difference of log2's: 2^-24 (4 |lp| + 24) + 2^-23; where
            nothing is cut the mass of the tokens behind the list is an fp32 sum: the lse's bound on top of it
  lse       a term is off by 2^-22 (ex2.approx) and by its exponent's rounding, 2^-23 |y| at a weight of 2^-y (|y| 2^-y <
            0.54); a thread adds up to V / 512 terms one after the other, then 2^5 sums: 2^-24 (V / 512 + 48) in all,
            and the result is rounded (2^-23 of it)
  loss      sum_i t_i (ln t_i - ln q_i): ln t_i and ln q_i are off by 2^-22 (1 + |ln|) and the lse's bound, t_i by 2^-22 (1 + |ln t_i|)
  gradient  scale (q - t): q off by 2^-21 + 2^-22 |ln q| and the sum's bound of itself, t as above, then the type's rounding
"""
import math

import numpy as np
import pytest
import torch

from block_diffusion_draft_dflash_gb300 import _lib
from oracle import rows as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
INF = math.inf


def held(x, dtype, pad=0, fill=123.0):
    """x [rows][V] in the type, with `pad` values behind each row."""
    x = torch.as_tensor(np.asarray(x, np.float32))
    whole = torch.full((x.shape[0], x.shape[1] + pad), fill, dtype=TYPES[dtype], device=DEV)
    whole[:, :x.shape[1]] = x.to(DEV)
    return whole[:, :x.shape[1]]


def f64(t):
    return t.double().cpu().numpy()


def f32(v):
    return torch.tensor(np.asarray(v, np.float32), device=DEV)


def i32(v):
    return torch.tensor(np.asarray(v, np.int32), device=DEV)


def logits(seed, rows, V, spread=2.0, heads=24, shift=0.0):
    rng = np.random.default_rng(seed)
    x = rng.normal(shift, spread, (rows, V))
    for r in range(rows):
        at = rng.integers(0, V, min(heads, V))
        x[r, at] = shift + 4 + rng.exponential(1 + 4 * rng.random(), at.size)
    return x


# ------------------------------------------------------------------------------ sample
def run_sample(x, u, settings=None, group=1, ws=None):
    """settings: list of (temperature, top_k, top_p, min_p) for each group, or None."""
    n = x.shape[0]
    ws = ws or _lib.Workspace(_lib.sample_workspace_size(n, x.shape[1]))
    token, lp, kept = (torch.full((n,), 77, dtype=t, device=DEV) for t in (torch.int32, torch.float32, torch.int32))
    named = {}
    if settings is not None:
        T, k, p, low = zip(*settings)
        named = dict(temperature=f32(T), top_k=i32(k), top_p=f32(p), min_p=f32(low))
    _lib.sample(x, f32(u), token, ws, group=group, logprob=lp, n_kept=kept, **named)
    torch.cuda.synchronize()
    return token.tolist(), lp.tolist(), kept.tolist(), ws.status()


def check_sample(x, u, settings=None, group=1):
    got = run_sample(x, u, settings, group)
    rows, u = f64(x), np.asarray(u, np.float32).astype(np.float64)
    for r in range(rows.shape[0]):
        s = (1.0, 0, 1.0, 0.0) if settings is None else settings[r // group]
        T, p, low = (float(np.float32(v)) for v in (s[0], s[2], s[3]))
        token, lp, n = ref.draw(rows[r], u[r], temperature=T, top_k=s[1], top_p=p, min_p=low)
        assert (got[0][r], got[2][r]) == (token, n), (r, s, u[r])
        if token < 0:
            assert got[1][r] == -INF
        else:
            open_ = s[1] <= 0 and p == 1 and low == 0
            assert abs(got[1][r] - lp) <= 2.0 ** -24 * (4 * abs(lp) + 24) + 2.0 ** -23 + open_ * lse_tol(0, rows.shape[1]), \
                (r, s, got[1][r], lp)
    assert got[3] == 0
    return got


SETTINGS = [(0.6, 20, 0.95, 0.0), (0.0, 0, 1.0, 0.0), (1.0, 0, 0.9, 0.0), (0.8, 200, 0.98, 0.02), (1.3, 0, 1.0, 0.1),
            (1.0, 50, 1.0, 0.0), (0.7, 0, 0.8, 0.0), (1.0, 0, 1.0, 0.0), (1.0, 1500, 0.7, 0.0), (2.0, 3000, 1.0, 0.001),
            (1.5, 1024, 0.999, 0.0), (1.0, 1, 1.0, 0.0), (5.0, 0, 0.3, 0.0), (1.0, 0, 1e-6, 0.0), (0.6, 1 << 20, 0.5, 1.0)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,V,pad", [(15, 1, 0), (15, 7, 3), (30, 129, 0), (30, 1000, 1), (15, 4001, 0), (15, 32003, 5),
                                        (15, 151936, 0), (15, 262147, 0)])
def test_sample_every_setting(dtype, rows, V, pad):
    x = held(logits(V + rows, rows, V), dtype, pad)
    u = np.random.default_rng(V).random(rows).astype(np.float32)
    check_sample(x, u, SETTINGS, rows // 15)


@pytest.mark.parametrize("rows", [1, 40, 700])
def test_sample_does_not_depend_on_how_many_ctas_share_a_row(rows):
    base = logits(11, 20, 20011)
    x = held(np.concatenate([base] * (rows // 20 + 1))[:rows], "fp32")
    u = np.tile(np.random.default_rng(3).random(20).astype(np.float32), rows // 20 + 1)[:rows]
    s = [SETTINGS[2], SETTINGS[3], SETTINGS[7], SETTINGS[8]] * 5
    got = check_sample(x, u, (s * (rows // 20 + 1))[:rows], 1)
    for r in range(20, rows):
        assert all(got[i][r] == got[i][r % 20] for i in (0, 2))


@pytest.mark.parametrize("kind", ["constant", "two", "whole", "flat", "steps"])
@pytest.mark.parametrize("V", [5000, 40000])
def test_sample_among_equal_logits(kind, V):
    rng = np.random.default_rng(V)
    x = {"constant": np.zeros((15, V)), "two": rng.integers(0, 2, (15, V)) * 3.0, "whole": np.round(rng.normal(0, 3, (15, V))),
         "flat": rng.normal(0, 1e-6, (15, V)), "steps": np.round(rng.normal(0, 1, (15, V)) * 512) / 512}[kind]
    for dtype in ("fp32", "bf16"):
        check_sample(held(x, dtype), rng.random(15), SETTINGS, 1)
    check_sample(held(np.sort(x, -1), "fp32"), rng.random(15), SETTINGS, 1)     # ordered rows
    check_sample(held(-np.sort(x, -1), "fp32"), rng.random(15), SETTINGS, 1)


def test_sample_u_walks_through_the_order():
    x = logits(5, 1, 3000)
    x[0, :8] = [9.0, 8.5, 8.5, 8.0, -0.0, 0.0, 7.0, 9.0]
    n = 200
    u = np.concatenate((np.linspace(0, 1, n - 2, endpoint=False), [np.nextafter(np.float32(1), np.float32(0)), 1e-30])).astype(np.float32)
    for s in ((1.0, 0, 1.0, 0.0), (1.0, 10, 1.0, 0.0), (1.0, 0, 0.95, 0.0)):
        check_sample(held(np.repeat(x, n, 0), "fp32"), u, [s], n)


def test_sample_masked_rows():
    V = 9000
    x = np.full((8, V), -INF)
    x[1, 17] = -3.0
    x[2, [5, 8999]] = [1.0, 1.0]
    x[3] = logits(1, 1, V)[0]
    x[3, ::2] = -INF
    x[4] = -1e30
    x[5, :100] = np.linspace(-1e4, -1e4 + 3, 100)
    x[6, 4:2500] = 1.0
    for s in ((1.0, 0, 1.0, 0.0), (0.6, 20, 0.95, 0.0), (0.0, 0, 1.0, 0.0), (1.0, 0, 0.9, 0.1), (1.0, 3000, 0.9, 0.0)):
        for dtype in ("fp32", "bf16"):
            check_sample(held(x, dtype), np.linspace(0.1, 0.99, 8), [s], 8)


@pytest.mark.parametrize("shift,T", [(0.0, 1e-3), (1e4, 1.0), (-3e4, 0.05), (1e-3, 1e-6), (300.0, 0.01), (0.0, 1e5), (0.0, 1e30),
                                     (5.0, 1e-30), (0.0, 2.0 ** -126), (0.0, 1e-45)])
def test_sample_far_exponents(shift, T):
    x = held(logits(9, 6, 5000, shift=shift), "fp32")
    if T < 2.0 ** -126:
        got = run_sample(x, [0.5] * 6, [(T, 0, 1.0, 0.0)], 6)
        assert got[0] == f64(x).argmax(-1).tolist() and got[2] == [1] * 6
        return
    for s in ((T, 0, 1.0, 0.0), (T, 40, 0.9, 0.0), (T, 0, 0.8, 0.01)):
        check_sample(x, np.linspace(0.05, 0.95, 6), [s], 6)


def test_sample_leaves_out_what_is_not_a_number():
    x = logits(3, 6, 7000)
    x[1, 6999] = np.nan
    x[3, 0] = INF
    x[4, 5] = -np.nan
    for s in ((1.0, 0, 1.0, 0.0), (1.0, 20, 0.9, 0.0)):
        t, lp, n, status = run_sample(held(x, "fp32"), [0.5] * 6, [s], 6)
        assert status == -6
        for r in (1, 3, 4):
            assert (t[r], lp[r], n[r]) == (-1, -INF, 0)
        for r in (0, 2, 5):
            assert (t[r], n[r]) == ref.draw(x[r].astype(np.float32), 0.5, temperature=1.0, top_k=s[1], top_p=float(np.float32(s[2])))[::2]


@pytest.mark.parametrize("bad", [(-1.0, 0, 1.0, 0.0), (math.nan, 0, 1.0, 0.0), (INF, 0, 1.0, 0.0), (1.0, 0, 0.0, 0.0), (1.0, 0, 1.5, 0.0),
                                 (1.0, 0, math.nan, 0.0), (1.0, 0, 1.0, -0.1), (1.0, 0, 1.0, 1.1), (1.0, 0, 1.0, math.nan)])
def test_sample_bad_settings_are_recorded(bad):
    x = held(logits(4, 4, 3000), "fp32")
    t, lp, n, status = run_sample(x, [0.25] * 4, [(1.0, 5, 1.0, 0.0), bad], 2)
    assert status == -1 and t[2:] == [-1, -1] and n[2:] == [0, 0] and lp[2:] == [-INF, -INF]
    assert t[:2] == [ref.draw(f64(x)[r], 0.25, top_k=5)[0] for r in (0, 1)]


def test_sample_bad_numbers_are_recorded():
    x = held(logits(4, 5, 3000), "fp32")
    t, _, n, status = run_sample(x, [0.25, 1.0, -0.1, math.nan, -0.0])
    assert status == -1 and t[1:4] == [-1] * 3 and t[0] == ref.draw(f64(x)[0], 0.25)[0] and t[4] == int(f64(x)[4].argmax())


def test_sample_optional_outputs_and_empty_call():
    x = held(logits(4, 3, 300), "bf16")
    ws = _lib.Workspace(_lib.sample_workspace_size(3, 300))
    token = i32([9, 9, 9])
    _lib.sample(x, f32([0.1, 0.5, 0.9]), token, ws)
    assert token.tolist() == [ref.draw(f64(x)[r], float(np.float32(v)))[0] for r, v in enumerate((0.1, 0.5, 0.9))]
    _lib.sample(x[:0], f32([]), i32([]), ws)
    assert ws.status() == 0


def test_sample_captured_and_on_another_stream():
    x, u = held(logits(6, 32, 50000), "bf16"), f32(np.random.default_rng(1).random(32))
    ws, token = _lib.Workspace(_lib.sample_workspace_size(32, 50000)), i32([0] * 32)
    T, p = f32([0.9]), f32([0.9])
    call = lambda: _lib.sample(x, u, token, ws, temperature=T, top_p=p, group=32)  # noqa: E731
    call()
    g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st), torch.cuda.graph(g, stream=st):
        call()
    for seed in (2, 3):
        u.copy_(f32(np.random.default_rng(seed).random(32)))
        g.replay()
        torch.cuda.synchronize()
        want = [ref.draw(f64(x)[r], float(u[r]), temperature=float(T[0]), top_p=float(p[0]))[0] for r in range(32)]
        assert token.tolist() == want
        token.zero_()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            call()
        st.synchronize()
        assert token.tolist() == want


# ------------------------------------------------------------------------------ top logits
def lse_tol(lse, V):
    return 2.0 ** -24 * (V / 512 + 48) + 2.0 ** -23 * abs(lse)


def run_top(x, K, T=1.0):
    n = x.shape[0]
    ws = _lib.Workspace(_lib.top_logits_workspace_size(n, x.shape[1]))
    i, v = torch.full((n, K), 7, dtype=torch.int32, device=DEV), torch.full((n, K), 7.0, device=DEV)
    lse = torch.full((n,), 7.0, device=DEV)
    _lib.top_logits(x, T, i, v, lse, ws)
    torch.cuda.synchronize()
    return i.cpu().numpy(), f64(v), f64(lse), ws.status()


def check_top(x, K, T=1.0):
    i, v, lse, status = run_top(x, K, T)
    assert status == 0
    for r, row in enumerate(f64(x)):
        ri, rv, rl = ref.top(row, K, T)
        np.testing.assert_array_equal(i[r], ri)
        np.testing.assert_array_equal(v[r], rv)
        assert lse[r] == rl or abs(lse[r] - rl) <= lse_tol(rl, row.size), (lse[r], rl)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,V,pad", [(3, 1, 0), (5, 9, 2), (400, 77, 0), (9, 1000, 1), (700, 2050, 0), (4, 33333, 3),
                                        (2, 151936, 0), (2, 1048576, 0)])
def test_top_logits(dtype, rows, V, pad):
    x = held(logits(V, rows, V), dtype, pad)
    for K in (1, 5, 64, 500, 1024):
        check_top(x, K, 0.5 if K == 5 else 1.0)


@pytest.mark.parametrize("V", [3000, 70000])
def test_top_logits_among_equal_ones(V):
    rng = np.random.default_rng(V)
    x = np.stack([np.zeros(V), np.round(rng.normal(0, 2, V)), np.where(np.arange(V) % 3, 1.0, 2.0), np.sort(rng.normal(0, 1, V)),
                  np.where(np.arange(V) < 2500, 5.0, -1.0), np.where(rng.random(V) < 0.99, -INF, 1.5), np.where(np.arange(V) == 9, -2.0, -INF),
                  np.where(rng.random(V) < 0.5, 0.0, -0.0)])
    for dtype in ("fp32", "bf16"):
        for K in (1, 20, 1000):
            check_top(held(x, dtype), K)


def test_top_logits_leaves_rows_out():
    x = logits(2, 4, 6000)
    x[1] = -INF
    x[2, 3] = np.nan
    i, v, lse, status = run_top(held(x, "fp32"), 4)
    assert status == -6 and (i[1:3] == -1).all() and np.isneginf(v[1:3]).all() and lse[1] == -INF and np.isnan(lse[2])
    assert i[3].tolist() == ref.top(x[3].astype(np.float32), 4)[0].tolist()


# ------------------------------------------------------------------------------ distillation
def lists(x, K, T, V):
    i, v, l = zip(*(ref.top(r, K, T) for r in x))
    return i32(np.stack(i)), f32(np.stack(v)), f32(l)


def run_distill(z, ids, vals, lse, T, teacher_row=None, weight=None, grad=True, in_place=False):
    n, V = z.shape
    ws = _lib.Workspace(_lib.distill_workspace_size(n, V))
    loss, stats = torch.full((n,), 7.0, device=DEV), torch.full((n, 4), 7.0, device=DEV)
    g = None if not grad else z if in_place else torch.full((n, V + 3), 7.0, dtype=z.dtype, device=DEV)[:, :V]
    _lib.distill(z, ids, vals, lse, T, loss, stats, ws, teacher_row=teacher_row, weight=weight, grad=g)
    torch.cuda.synchronize()
    return loss, stats, g, ws.status()


def run_backward(z, ids, vals, lse, T, stats, grad_loss=None, teacher_row=None, weight=None, in_place=False):
    n, V = z.shape
    ws = _lib.Workspace(_lib.distill_workspace_size(n, V))
    g = z if in_place else torch.full((n, V), 7.0, dtype=z.dtype, device=DEV)
    _lib.distill_backward(z, ids, vals, lse, T, stats, g, ws, grad_loss=grad_loss, teacher_row=teacher_row, weight=weight)
    torch.cuda.synchronize()
    return g, ws.status()


def check_row(got_loss, got_stats, grads, z, ids, vals, lse, T, w, scales, dtype):
    loss, grad, stats = ref.distill(z, ids, vals, lse, T, w)
    m, lns, lnr, _ = stats
    V = z.size
    s_tol = 2.0 ** -24 * (V / 512 + 48)
    _, t, rho = ref.teacher(ids, vals, lse, T)
    on = np.asarray(ids)[np.asarray(ids) >= 0]
    with np.errstate(divide="ignore", invalid="ignore"):
        ln_q = (z - m) / T - lns
        ln_t = np.log(t)
    part = t * (2.0 ** -22 * (2 + np.abs(ln_t) + np.abs(ln_q[on]) + np.abs(lse if lse is not None else 0.0) / 4) + s_tol) * (1 + np.abs(ln_t - ln_q[on]))
    slack = part[t > 0].sum()
    r_tol = 2.0 ** -22 * (t * (2 + np.abs(ln_t))).sum() if t.size else 0.0      # of rho
    if rho > 0 and np.isfinite(lnr):
        slack += (r_tol + rho * 2 * s_tol) * (2 + abs(math.log(rho)) + abs(lnr - lns))
    elif lse is not None:
        slack += r_tol * 40
    if np.isfinite(loss):
        assert abs(got_loss - loss) <= abs(w) * slack + 2.0 ** -23 * abs(loss), (got_loss, loss, slack)
    else:
        assert got_loss == loss
    assert got_stats[0] == m and got_stats[3] == 0
    assert abs(got_stats[1] - lns) <= lse_tol(lns, V) and (got_stats[2] == lnr or abs(got_stats[2] - lnr) <= lse_tol(lnr, V))
    eps = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8}[dtype]
    with np.errstate(invalid="ignore"):
        q = np.exp(ln_q)
        rel = np.where(q > 0, 2.0 ** -21 + 2.0 ** -22 * np.abs(ln_q) + s_tol + 2.0 ** -23 * abs(lns), 0.0)
    tol = q * rel
    if rho > 0 or lse is not None:
        if np.isfinite(lnr):
            tol = tol + q * np.exp(lns - lnr) * (rho * (rel + 2 * s_tol + 2.0 ** -22 * abs(lnr)) + r_tol)
    tol[on] = q[on] * rel[on] + t * 2.0 ** -22 * (3 + np.abs(np.where(t > 0, ln_t, 0.0)) + abs(lse or 0.0) / 4)
    for g, scale in zip(grads, scales):
        want = grad * scale
        bound = abs(w) / T * abs(scale) * tol + np.abs(want) * eps * 1.01 + 1e-38
        assert (np.abs(g - want) <= bound).all(), (np.abs(g - want) / bound).max()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,V,K,T,full,pad", [
    (3, 1, 1, 1.0, True, 0), (5, 13, 4, 2.0, True, 1), (40, 300, 33, 1.0, True, 0), (40, 300, 33, 0.5, False, 3),
    (700, 501, 20, 1.0, True, 0), (6, 5000, 1, 1.0, True, 0), (6, 5000, 1024, 1.0, False, 5), (4, 33333, 64, 2.0, True, 0),
    (3, 151936, 128, 1.0, True, 0), (2, 600001, 512, 1.0, True, 0), (9, 20, 20, 1.0, True, 0)])
def test_distill(dtype, rows, V, K, T, full, pad):
    rng = np.random.default_rng(V)
    y = logits(V, rows, V).astype(np.float32)
    z = held(0.8 * y + rng.normal(0, 1, y.shape), dtype, pad)
    row = rng.permutation(rows)
    row[rows // 2] = -1
    weight = rng.random(rows) + 0.1
    weight[0] = 0.0
    ids, vals, lse = lists(y, K, T, V)
    lse = lse if full else None
    loss, stats, grad, status = run_distill(z, ids, vals, lse, T, i32(row), f32(weight))
    alone, _, _, status2 = run_distill(z, ids, vals, lse, T, i32(row), f32(weight), grad=False)
    up = rng.random(rows) + 0.5
    back, status3 = run_backward(z, ids, vals, lse, T, stats, f32(up), i32(row), f32(weight))
    assert status == status2 == status3 == 0 and torch.equal(loss, alone)
    hz, hid, hval = f64(z), ids.cpu().numpy(), f64(vals)
    hl, hs, hg, hb, w, up = f64(loss), f64(stats), f64(grad), f64(back), f64(f32(weight)), f64(f32(up))
    for r in range(rows):
        a = row[r]
        if a < 0 or w[r] == 0:
            assert hl[r] == 0 and (hs[r] == 0).all() and (hg[r] == 0).all() and (hb[r] == 0).all()
            continue
        check_row(hl[r], hs[r], (hg[r], hb[r]), hz[r], hid[a], hval[a], float(lse[a]) if full else None, T, w[r], (1.0, up[r]), dtype)
    assert (f64(grad._base)[:, V:] == 7).all()       # what lies behind a gradient's rows
    for call in (lambda c: run_distill(c, ids, vals, lse, T, i32(row), f32(weight), in_place=True)[2],
                 lambda c: run_backward(c, ids, vals, lse, T, stats, None, i32(row), f32(weight), in_place=True)[0]):
        whole = z._base.clone()
        mine = call(whole[:, :V])
        assert torch.equal(whole[:, V:], z._base[:, V:])
        np.testing.assert_allclose(f64(mine), hg, rtol=2.0 ** -7 if dtype == "bf16" else 1e-4, atol=1e-6)


def test_distill_gradient_by_differences():
    V, K, T = 200, 8, 1.0
    y = logits(1, 1, V).astype(np.float32)
    z = logits(2, 1, V).astype(np.float32)
    ids, vals, lse = lists(y, K, T, V)
    _, _, grad, _ = run_distill(f32(z), ids, vals, lse, T)
    grad = f64(grad)[0]
    h = 0.0625
    for j in (0, 5, int(ids[0, 0]), int(ids[0, 7]), V - 1):
        d = np.zeros((1, V), np.float32)
        d[0, j] = h
        up, down = (f64(run_distill(f32(z + s * d), ids, vals, lse, T, grad=False)[0])[0] for s in (1, -1))
        # the third derivative of a log-sum is at most 1/4 q: h^2 / 24; losses near 10 are off by 2^-20
        assert abs((up - down) / (2 * h) - grad[j]) <= h * h / 24 + 2.0 ** -19 / h


def test_distill_masked_student():
    V, K = 4000, 16
    y = logits(3, 5, V).astype(np.float32)
    z = logits(4, 5, V)
    z[1, 100:] = -INF                  # most of it, listed tokens among them
    z[2, :] = -INF
    z[3, ::2] = -INF
    ids, vals, lse = lists(y, K, 1.0, V)
    z[4] = -INF
    z[4, ids[4].long().cpu().numpy()] = 1.0   # only listed tokens: sigma 0
    x = held(z, "fp32")
    loss, stats, grad, status = run_distill(x, ids, vals, lse, 1.0)
    assert status == -6 and np.isnan(f64(loss)[2]) and np.isnan(f64(stats)[2]).all() and (f64(grad)[2] == 0).all()
    back, _ = run_backward(x, ids, vals, lse, 1.0, stats)
    assert (f64(back)[2] == 0).all()
    for r in (0, 1, 3, 4):
        check_row(f64(loss)[r], f64(stats)[r], (f64(grad)[r], f64(back)[r]), f64(x)[r], ids[r].cpu().numpy(), f64(vals)[r],
                  float(lse[r]), 1.0, 1.0, (1.0, 1.0), "fp32")
    assert f64(loss)[4] == INF


def test_distill_a_sure_student_keeps_its_digits():
    # the mass outside the list is 1e-12 of the row's: as a difference it would have no digit left
    V, K = 3000, 4
    z = np.zeros((1, V))
    z[0, :K] = 35.0
    y = np.zeros((1, V), np.float32)
    y[0, :K] = [6.0, 5.0, 4.0, 3.0]
    ids, vals, lse = lists(y, K, 1.0, V)
    loss, stats, grad, status = run_distill(held(z, "fp32"), ids, vals, lse, 1.0)
    assert status == 0
    check_row(f64(loss)[0], f64(stats)[0], (f64(grad)[0],), z[0], ids[0].cpu().numpy(), f64(vals)[0], float(lse[0]), 1.0, 1.0, (1.0,), "fp32")


def test_distill_bad_lists_are_left_out():
    V, K, n = 5000, 6, 8
    y = logits(5, n, V).astype(np.float32)
    ids, vals, lse = lists(y, K, 1.0, V)
    ids[1, 3] = V
    ids[2, 0] = -2
    ids[3, 5] = ids[3, 1]
    vals[4, 2] = math.nan
    lse[5] = math.nan
    row = i32([0, 1, 2, 3, 4, 5, n, 7])
    z = held(logits(6, n, V), "bf16")
    z[7, 11] = math.nan
    loss, stats, grad, status = run_distill(z, ids, vals, lse, 1.0, row)
    assert status in (-1, -6)
    hl = f64(loss)
    assert np.isfinite(hl[0]) and np.isnan(hl[1:]).all() and np.isnan(f64(stats)[1:]).all() and (f64(grad)[1:] == 0).all()
    back, _ = run_backward(z, ids, vals, lse, 1.0, stats, None, row)
    assert (f64(back)[1:] == 0).all() and (f64(back)[0] != 0).any()
    for r in range(1, 8):      # each by itself says what it is
        status = run_distill(z[r:r + 1], ids, vals, lse, 1.0, row[r:r + 1].clone())[3]
        assert status == (-1 if r in (1, 2, 3, 6) else -6), r


def test_distill_short_and_empty_lists():
    V = 700
    y, z = logits(7, 3, V).astype(np.float32), held(logits(8, 3, V), "fp32")
    ids, vals, lse = lists(y, 8, 1.0, V)
    ids[1, 5:] = -1
    ids[2, :] = -1
    vals[1, 5:] = math.nan             # of entries that are not there
    loss, stats, grad, status = run_distill(z, ids, vals, lse, 1.0)
    assert status == 0
    for r in range(3):
        check_row(f64(loss)[r], f64(stats)[r], (f64(grad)[r],), f64(z)[r], ids[r].cpu().numpy(), f64(vals)[r], float(lse[r]), 1.0,
                  1.0, (1.0,), "fp32")
    _, _, _, status = run_distill(z, ids, vals, None, 1.0)
    assert status == -6


def test_distill_captured_with_its_gradient():
    V, K, n = 20000, 32, 24
    y = logits(9, n, V).astype(np.float32)
    ids, vals, lse = lists(y, K, 1.0, V)
    z = held(logits(10, n, V), "bf16")
    ws = _lib.Workspace(_lib.distill_workspace_size(n, V))
    loss, stats = torch.zeros(n, device=DEV), torch.zeros(n, 4, device=DEV)
    grad, back = torch.zeros_like(z), torch.zeros_like(z)

    def call():
        _lib.distill(z, ids, vals, lse, 1.0, loss, stats, ws, grad=grad)
        _lib.distill_backward(z, ids, vals, lse, 1.0, stats, back, ws)

    call()
    g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st), torch.cuda.graph(g, stream=st):
        call()
    z.copy_(held(logits(11, n, V), "bf16"))
    g.replay()
    torch.cuda.synchronize()
    want = [t.clone() for t in (loss, stats, grad, back)]
    call()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (loss, stats, grad, back)))
    assert abs(f64(loss)[0] - ref.distill(f64(z)[0], ids[0].cpu().numpy(), f64(vals)[0], float(lse[0]), 1.0)[0]) < 1e-4


# ------------------------------------------------------------------------------ sizes and orders
LOWEST = {"fp32": float(torch.finfo(torch.float32).min), "bf16": float(torch.finfo(torch.bfloat16).min)}


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V", [1, 500, 40000])
def test_rows_masked_by_the_lowest_number(dtype, V):
    x = logits(21, 15, V)
    keep = np.random.default_rng(V).random(x.shape) < 0.01
    x[~keep] = LOWEST[dtype]
    x[3] = LOWEST[dtype]                 # nothing but masked tokens: all alike
    x[7, :] = LOWEST[dtype]
    x[7, V // 2] = -LOWEST[dtype]        # and one as far above
    check_sample(held(x, dtype), np.random.default_rng(1).random(15), SETTINGS, 1)
    for T in (1.0, 0.3, 2.0 ** 60):
        i, v, lse, status = run_top(held(x, dtype), 30, T)
        assert status == 0
        for r, row in enumerate(f64(held(x, dtype))):
            ri, rv, rl = ref.top(row, 30, T)
            np.testing.assert_array_equal(i[r], ri)
            np.testing.assert_array_equal(v[r], rv)
            if abs(rl) < 2.0 ** 127:
                assert abs(lse[r] - rl) <= lse_tol(rl, V)
    y = logits(22, 15, V).astype(np.float32)
    ids, vals, lse = lists(y, 20, 1.0, V)
    if V > 40:                           # masked tokens outside the lists
        np.put_along_axis(x, ids.cpu().numpy().astype(np.int64), np.random.default_rng(2).normal(0, 2, (15, 20)), 1)
        z = held(x, dtype)
        z[7, V // 2] = 1.0
        loss, stats, grad, status = run_distill(z, ids, vals, lse, 1.0)
        assert status == 0
        for r in range(15):
            check_row(f64(loss)[r], f64(stats)[r], (f64(grad)[r],), f64(z)[r], ids[r].cpu().numpy(), f64(vals)[r], float(lse[r]),
                      1.0, 1.0, (1.0,), dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_distill_a_part_of_the_row_masked_by_the_lowest_number(dtype):
    """What one CTA of a row reads is masked as a whole, and its largest logit over T is out of range."""
    V, T = 40000, 0.5
    x, y = logits(30, 15, V), logits(31, 15, V).astype(np.float32)
    x[:, V // 2:], y[:, V // 2:] = LOWEST[dtype], -20.0
    ids, vals, lse = lists(y, 20, T, V)
    z = held(x, dtype)
    loss, stats, grad, status = run_distill(z, ids, vals, lse, T)
    back, status2 = run_backward(z, ids, vals, lse, T, stats)
    assert status == status2 == 0 and torch.isfinite(loss).all()
    for r in range(15):
        check_row(f64(loss)[r], f64(stats)[r], (f64(grad)[r], f64(back)[r]), f64(z)[r], ids[r].cpu().numpy(), f64(vals)[r],
                  float(lse[r]), T, 1.0, (1.0, 1.0), dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_largest_vocabulary(dtype):
    V = 1 << 20
    x = held(logits(23, 15, V), dtype)
    check_sample(x, np.random.default_rng(4).random(15), SETTINGS, 1)
    check_top(x, 1024)
    ids, vals, lse = lists(f64(x)[::-1].copy(), 1024, 1.0, V)
    loss, stats, grad, status = run_distill(x, ids, vals, lse, 1.0)
    assert status == 0
    for r in range(15):
        check_row(f64(loss)[r], f64(stats)[r], (f64(grad)[r],), f64(x)[r], ids[r].cpu().numpy(), f64(vals)[r], float(lse[r]),
                  1.0, 1.0, (1.0,), dtype)


@pytest.mark.parametrize("rows,V", [(1500, 9001), (700, 40000), (80000, 300)])
def test_many_rows_whose_borders_lie_far_behind(rows, V):
    """Flat rows cut by mass: more of them to search than there are places at once, in all three more than a list holds."""
    base, u = logits(29, 16, V, spread=0.5, heads=0), np.random.default_rng(7).random(16).astype(np.float32)
    settings = [(1.0, 0, 0.9, 0.0), (1.0, 0, 1.0, 0.0), (0.8, 0, 0.99, 0.0), (1.0, 2000, 0.95, 0.0)] * 4
    small, n = held(base, "bf16"), rows // 16 + 1
    one = check_sample(small, u, settings, 1)
    got = run_sample(small.repeat(n, 1)[:rows], np.tile(u, n)[:rows], (settings * n)[:rows], 1)
    assert got[3] == 0
    for i in (0, 2):
        assert got[i] == (one[i] * n)[:rows]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V", [9001, 150001])
def test_borders_among_tokens_of_next_to_no_probability(dtype, V):
    """All but one token lie below 2^-32 of the first; together they still hold the last numbers' draws.

    A mass is a whole number of 2^-42 of the first token's: off by at most 2^-43 (its rounding) and 2^-35 of itself, so a
    sum of up to V of them by V 2^-43 + 2^-35 M.  A border compares two such sums: it is right within twice that.
    """
    rng = np.random.default_rng(V)
    x = rng.normal(-23.6, 0.3, (15, V))
    x[np.arange(15), rng.integers(0, V, 15)] = 0.0
    u = 1 - 2.0 ** -24 * np.arange(1, 16) ** 2
    p = 1 - 2.0 ** -24
    x = held(x, dtype)
    for settings, group in (([(1.0, 0, 1.0, 0.0)], 15), ([(1.0, 0, p, 0.0)], 15),
                            ([(1.0, V // 2, p, 0.0), (0.95, V - 5, 1.0, 0.0), (1.0, 3, 1.0, 0.0)], 5)):
        token, _, kept, status = run_sample(x, u, settings, group)
        assert status == 0
        for r, row in enumerate(f64(x)):
            T, k, top_p, _ = settings[r // group]
            T, top_p = float(np.float32(T)), float(np.float32(top_p))
            order = np.lexsort((np.arange(V), -row))
            cum = np.cumsum(np.exp(row[order] / T))
            if k:
                cum = cum[:k]
            tol = 2 * (V * 2.0 ** -43 + 2.0 ** -35 * cum[-1])
            n = kept[r]
            if top_p < 1:
                assert cum[n - 1] >= top_p * cum[-1] - tol and (n == 1 or cum[n - 2] < top_p * cum[-1] + tol)
            else:
                assert n == cum.size
            at = int(np.nonzero(order == token[r])[0][0])
            want = float(np.float32(u[r])) * cum[n - 1]
            assert at < n and cum[at] > want - tol and (at == 0 or cum[at - 1] <= want + tol)


def test_rows_farther_apart_than_32_bits():
    """Element offsets beyond 2^31 and byte offsets beyond 2^32, of the rows and of the gradient."""
    V, ld = 5001, (1 << 30) + 13
    far, out = (torch.empty(3 * ld + V, dtype=torch.bfloat16, device=DEV).as_strided((4, V), (ld, 1)) for _ in range(2))
    x = held(logits(24, 4, V), "bf16")
    far.copy_(x)
    u = np.random.default_rng(5).random(4)
    for s in ([SETTINGS[0]], [SETTINGS[2]], [SETTINGS[7]]):
        check_sample(far, u, s, 4)
    check_top(far, 64)
    ids, vals, lse = lists(f64(x)[::-1].copy(), 64, 1.0, V)
    ws = _lib.Workspace(_lib.distill_workspace_size(4, V))
    loss, stats = torch.zeros(4, device=DEV), torch.zeros(4, 4, device=DEV)
    _lib.distill(far, ids, vals, lse, 1.0, loss, stats, ws, grad=out)
    grad = f64(out)
    out.zero_()
    _lib.distill_backward(far, ids, vals, lse, 1.0, stats, out, ws)
    for r in range(4):      # not bit for bit those of rows that lie close: pieces, and so the order of sums, go by a row's address
        check_row(f64(loss)[r], f64(stats)[r], (grad[r], f64(out)[r]), f64(x)[r], ids[r].cpu().numpy(), f64(vals)[r],
                  float(lse[r]), 1.0, 1.0, (1.0, 1.0), "bf16")
    assert ws.status() == 0


def test_calls_at_once_on_two_streams():
    """Each with its own workspace; results are those of the calls one after the other, to the bit."""
    V, n = 50021, 96
    x, y = (held(logits(s, n, V), "bf16") for s in (25, 26))
    u, settings = np.random.default_rng(6).random(n), [SETTINGS[2], SETTINGS[7], SETTINGS[3]]
    streams = [torch.cuda.Stream() for _ in range(2)]
    T, k, p, low = (f(v) for f, v in zip((f32, i32, f32, f32), zip(*settings)))
    uu = f32(u)
    named = dict(temperature=T, top_k=k, top_p=p, min_p=low, group=n // 3)
    alone = [run_sample(t, u, settings, n // 3) for t in (x, y)]
    tops = [run_top(t, 100) for t in (x, y)]
    ids, vals, lse = i32(tops[0][0]), f32(tops[0][1]), f32(tops[0][2])
    taught = run_distill(y, ids, vals, lse, 1.0)
    held_out = []
    torch.cuda.synchronize()
    for _ in range(5):
        for t, st in zip((x, y), streams):
            with torch.cuda.stream(st):
                token, lp, kept = (torch.empty(n, dtype=d, device=DEV) for d in (torch.int32, torch.float32, torch.int32))
                ws = _lib.Workspace(_lib.sample_workspace_size(n, V))
                _lib.sample(t, uu, token, ws, logprob=lp, n_kept=kept, **named)
                i, v, l = (torch.empty(*s, dtype=d, device=DEV) for s, d in (((n, 100), torch.int32), ((n, 100), torch.float32), ((n,), torch.float32)))
                _lib.top_logits(t, 1.0, i, v, l, ws)
                loss, stats, grad = torch.empty(n, device=DEV), torch.empty(n, 4, device=DEV), torch.empty_like(y)
                _lib.distill(y, ids, vals, lse, 1.0, loss, stats, ws, grad=grad)
                held_out.append((t is y, ws, token, lp, kept, i, v, l, loss, stats, grad))
    torch.cuda.synchronize()
    for j, ws, token, lp, kept, i, v, l, loss, stats, grad in held_out:
        assert (token.tolist(), lp.tolist(), kept.tolist()) == alone[j][:3] and ws.status() == 0
        assert (i.cpu().numpy() == tops[j][0]).all() and (f64(v) == tops[j][1]).all() and (f64(l) == tops[j][2]).all()
        assert torch.equal(loss, taught[0]) and torch.equal(stats, taught[1]) and torch.equal(grad, taught[2])


def test_distill_one_list_for_many_rows():
    V, n = 2003, 37
    z = held(logits(27, n, V), "fp32")
    ids, vals, lse = lists(logits(28, 2, V).astype(np.float32), 50, 1.0, V)
    row = np.arange(n) % 2
    loss, stats, grad, status = run_distill(z, ids, vals, lse, 1.0, i32(row))
    each = run_distill(z, ids[i32(row).long()], vals[i32(row).long()], lse[i32(row).long()], 1.0)
    assert status == 0 and all(torch.equal(a, b) for a, b in zip((loss, stats, grad), each))


# ------------------------------------------------------------------------------ together
def test_draw_then_teach():
    """What a target's logits of an accepted path are used for: tokens drawn, lists handed out, the drafter's rows taught."""
    V, T, D, K = 30011, 33, 15, 24
    x = held(logits(12, T, V), "fp32")
    token, _, _, _ = run_sample(x, np.random.default_rng(2).random(T), [(0.6, 20, 0.95, 0.0)], T)
    ids = torch.zeros(T, K, dtype=torch.int32, device=DEV)
    vals, lse = torch.zeros(T, K, device=DEV), torch.zeros(T, device=DEV)
    ws = _lib.Workspace(_lib.distill_workspace_size(T, V))
    _lib.top_logits(x, 1.0, ids, vals, lse, ws)
    assert all(token[r] in ids[r].tolist() for r in range(T))
    path = [0, 4, 9, 30]
    row = i32(path + [-1] * (D - len(path)))
    z = held(logits(13, D, V), "fp32")
    loss, stats = torch.zeros(D, device=DEV), torch.zeros(D, 4, device=DEV)
    grad = torch.zeros_like(z)
    weight = f32(np.exp(-np.arange(D) / 7))
    for _ in range(3):
        _lib.distill(z, ids, vals, lse, 1.0, loss, stats, ws, teacher_row=row, weight=weight, grad=grad)
        for r, a in enumerate(path):
            want = ref.distill(f64(z)[r], ids[a].cpu().numpy(), f64(vals)[a], float(lse[a]), 1.0, float(weight[r]))
            assert abs(float(loss[r]) - want[0]) <= 1e-5 * max(1.0, want[0])
            np.testing.assert_allclose(f64(grad)[r], want[1], atol=2e-6)
        assert (f64(grad)[len(path):] == 0).all() and (f64(loss)[len(path):] == 0).all()
        z -= 0.5 * grad
    assert ws.status() == 0
