"""Pins of the 4-bit KV cache's oracle (CPU), and the library's refusals, which are host code."""
import ctypes as C
import itertools

import numpy as np
import pytest
import torch

from block_diffusion_draft_dflash_gb300 import _lib
from oracle import kv4


def test_e4m3_grid_is_torchs():
    ref = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(kv4.E4M3, ref)


def test_nearest_against_every_candidate():
    rng = np.random.default_rng(0)
    for grid in (kv4.E2M1, kv4.E4M3):
        mids = (grid[1:] + grid[:-1]) / 2                      # the ties
        x = np.concatenate([grid, mids, -mids, rng.uniform(0, 1.2 * grid[-1], 500), [np.inf]])
        got = kv4.nearest(x, grid)
        for v, i in zip(np.minimum(np.abs(x), grid[-1]), got):
            d = np.abs(grid - v)
            best = np.flatnonzero(d == d.min())
            assert i == (best[0] if len(best) == 1 else best[best % 2 == 0][0])
        np.testing.assert_array_equal(kv4.nearest(grid, grid), np.arange(len(grid)))
        np.testing.assert_array_equal(kv4.nearest(mids, grid) % 2, 0)


def test_scale_rounding_is_torchs():
    x = np.random.default_rng(1).lognormal(0, 3, (400, 128)).astype(np.float32)
    x = torch.from_numpy(x).bfloat16()
    _, s = kv4.round_rows(x.double().numpy(), 0)
    amax = x.float().view(400, 8, 16).amax(-1) / 6
    ref = amax.clamp(max=448.0).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(s, ref)


def test_error_bound_of_a_block():
    # half the widest gap of the codes is 1 of a scale, a scale at most (1 + 2^-4) amax / 6; where the
    # scale was rounded down the largest value is cut at 6 (1 - 2^-4) amax / 6
    x = np.random.default_rng(2).normal(0, 1, (64, 128))
    v = kv4.values(*kv4.round_rows(x, -3), -3)
    err = np.abs(v - x).reshape(64, 8, 16).max(-1)
    assert (err <= np.abs(x).reshape(64, 8, 16).max(-1) / 6 * (1 + 2.0 ** -4)).all()
    z, zs = kv4.round_rows(np.zeros((1, 128)), 0)
    assert not z.any() and not zs.any()


def test_attend_is_torchs():
    rng = np.random.default_rng(3)
    q, k, v = rng.normal(size=(5, 6, 128)), rng.normal(size=(20, 3, 128)), rng.normal(size=(20, 3, 128))
    sets = [list(range(15 + i + 1)) for i in range(5)]
    out, lse, _ = kv4.attend(q, k, v, 0.1, sets)
    mask = torch.ones(5, 20, dtype=torch.bool).tril(15)
    ref = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(q).transpose(0, 1), torch.from_numpy(k).transpose(0, 1).repeat_interleave(2, 0),
        torch.from_numpy(v).transpose(0, 1).repeat_interleave(2, 0), attn_mask=mask, scale=0.1).transpose(0, 1)
    np.testing.assert_allclose(out, ref.numpy(), atol=1e-12)
    x = np.einsum("thd,nhd->htn", q, np.repeat(k, 2, 1)) * 0.1
    x[:, ~mask.numpy()] = -np.inf
    np.testing.assert_allclose(lse, np.log(np.exp(x).sum(-1)).T, atol=1e-12)


def test_weights_sum_to_the_heads():
    # every (row, head) distributes weight 1 over the slots it sees
    rng = np.random.default_rng(4)
    q, k = rng.normal(size=(7, 4, 128)), rng.normal(size=(30, 2, 128))
    rows = [0, 2, 5]
    lse = np.full((7, 4), np.nan)
    for j, node in enumerate(rows):
        _, l, _ = kv4.attend(q[node:node + 1], k, k, 0.1, [range(27 + j + 1)])
        lse[node] = l[0]
    got = kv4.weights(q, lse, k, 0.1, np.zeros((2, 30)), 30, rows)
    np.testing.assert_allclose(got.sum(1), [6.0, 6.0])       # 3 rows x 2 heads a kv head
    again = kv4.weights(q, lse, k, 0.1, np.full((2, 30), 8.0), 30, rows, decay=0.5)
    np.testing.assert_allclose(again[:, :27], got[:, :27] + 4.0)
    np.testing.assert_allclose(again[:, 27:], got[:, 27:])   # slots of the rows start from 0


def test_evict_against_every_subset():
    for n, budget, sink, recent in ((6, 3, 1, 1), (7, 4, 0, 2), (5, 5, 1, 1), (6, 2, 0, 0)):
        score = np.array([3.0, 1.0, 1.0, np.nan, 1.0, 0.5, 2.0][:n])
        got = kv4.evict(score, n, budget, sink, recent)
        fixed = set(range(min(sink, n))) | set(range(max(0, n - recent), n))
        val = np.where(np.isnan(score), -1.0, score)
        best = max((c for c in itertools.combinations(range(n), budget) if fixed <= set(c)),
                   key=lambda c: (sum(val[i] for i in c), [-i for i in c]))
        assert tuple(got) == best


# ---------------------------------------------------------------------------- refusals (host)
def _cache(n_layers=2, b=1, Hkv=2, hd=128, cap=64, k_exp=0, v_exp=0, ptrs=(4096, 8192, 12288, 16384)):
    return _lib.Kv4CacheStruct(*ptrs, n_layers, b, Hkv, hd, cap, k_exp, v_exp)


BAD = [(dict(n_layers=0), -1), (dict(b=-1), -1), (dict(Hkv=0), -1), (dict(cap=0), -1), (dict(cap=60), -2),
       (dict(hd=64), -2), (dict(k_exp=33), -1), (dict(v_exp=-33), -1), (dict(ptrs=(None, 8192, 12288, 16384)), -1),
       (dict(ptrs=(4096, 8200, 12288, 16384)), -3)]


def _append(c, layer=0, k=16, v=16, n=3, n_new=None, clen=16, kh=None, vh=None, ws=None, nb=0):
    return _lib.load().dflash_kv4_append(C.byref(c), layer, k, v, n, n_new, clen, kh, vh, ws, nb, None)


def _attention(c, layer=0, n_tree=3, Hq=4, q=16, clen=16, anc=None, scale=0.1, out=16, lse=None, ws=None, nb=0):
    return _lib.load().dflash_kv4_attention(C.byref(c), layer, n_tree, Hq, q, clen, anc, scale, out, lse, ws, nb, None)


def _weights(c, layer=0, n_tree=3, Hq=4, q=16, lse=16, clen=16, n_rows=None, src=None, max_src=0, scale=0.1, decay=1.0,
             score=16, out=16, ws=None, nb=0):
    return _lib.load().dflash_kv4_attention_weights(C.byref(c), layer, n_tree, Hq, q, lse, clen, n_rows, src, max_src,
                                                    scale, decay, score, out, ws, nb, None)


def _compact(c, src=16, max_src=3, n_acc=16, clen=16, ws=None, nb=0):
    return _lib.load().dflash_kv4_compact(C.byref(c), src, max_src, n_acc, clen, ws, nb, None)


def _evict(c, score=1 << 30, clen=16, budget=16, sink=2, recent=4, to=None, score_out=None, new_len=16, kept=16, ws=None,
           nb=0):
    to = _cache(ptrs=(1 << 24, 2 << 24, 3 << 24, 4 << 24)) if to is None else to
    return _lib.load().dflash_kv4_evict(C.byref(c), score, clen, budget, sink, recent, C.byref(to), score_out, new_len,
                                        kept, ws, nb, None)


@pytest.mark.parametrize("call", [_append, _attention, _weights, _compact, _evict])
def test_refusals_of_caches(call):
    for kw, code in BAD:
        assert call(_cache(**kw)) == code, kw
    assert call(_cache()) == -9                                # nothing else is wrong: no workspace
    assert call(_cache(), ws=4096, nb=255) == -9               # too small
    if call is not _evict:                                     # no sequences: nothing to do
        assert call(_cache(b=0, ptrs=(None,) * 4)) == 0


@pytest.mark.parametrize("call,kw,code", [
    (_append, dict(layer=2), -1), (_append, dict(layer=-1), -1), (_append, dict(n=-1), -1), (_append, dict(k=None), -1),
    (_append, dict(clen=None), -1), (_append, dict(kh=16), -1), (_append, dict(k=24), -3), (_append, dict(kh=8, vh=16), -3),
    (_append, dict(n=0), 0),
    (_attention, dict(layer=2), -1), (_attention, dict(n_tree=0), -1), (_attention, dict(Hq=3), -1),
    (_attention, dict(scale=0.0), -1), (_attention, dict(scale=-1.0), -1), (_attention, dict(scale=float("nan")), -1),
    (_attention, dict(scale=float("inf")), -1), (_attention, dict(q=None), -1), (_attention, dict(out=None), -1),
    (_attention, dict(q=8), -3), (_attention, dict(anc=4), -3), (_attention, dict(Hq=1 << 30), -2),
    (_weights, dict(layer=-1), -1), (_weights, dict(Hq=5), -1), (_weights, dict(decay=-0.1), -1),
    (_weights, dict(decay=1.1), -1), (_weights, dict(decay=float("nan")), -1), (_weights, dict(scale=0.0), -1),
    (_weights, dict(max_src=-1), -1), (_weights, dict(lse=None), -1), (_weights, dict(score=8), -3),
    (_compact, dict(max_src=-1), -1), (_compact, dict(src=None), -1), (_compact, dict(n_acc=None), -1),
    (_compact, dict(max_src=0), 0),
    (_evict, dict(budget=0), -1), (_evict, dict(budget=65), -4), (_evict, dict(sink=-1), -1), (_evict, dict(recent=-1), -1),
    (_evict, dict(sink=10, recent=7), -1), (_evict, dict(to=_cache()), -1), (_evict, dict(to=_cache(b=2)), -1),
    (_evict, dict(to=_cache(n_layers=1)), -1), (_evict, dict(to=_cache(Hkv=1)), -1), (_evict, dict(to=_cache(k_exp=1)), -1),
    (_evict, dict(score=None), -1), (_evict, dict(kept=None), -1), (_evict, dict(new_len=None), -1),
    (_evict, dict(kept=8), -3), (_evict, dict(score=1 << 30, score_out=(1 << 30) + 64), -1),
])
def test_refusals_of_arguments(call, kw, code):
    assert call(_cache(), **kw) == code


def test_binding_refuses_wrong_tensors():
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    with pytest.raises(ValueError):          # host memory
        _lib.Kv4Cache(u8(1, 1, 1, 8, 64), u8(1, 1, 1, 8, 8), u8(1, 1, 1, 8, 64), u8(1, 1, 1, 8, 8))
    with pytest.raises(ValueError):
        _lib.Kv4Cache(u8(1, 1, 8, 64), u8(1, 1, 1, 8, 8), u8(1, 1, 1, 8, 64), u8(1, 1, 1, 8, 8))
