"""The 4-bit KV cache against its float64 oracle.

Tolerances.  The cache's values are fp16 numbers, so a score is an fp32 sum of 128 exact products: its
error is at most 130 * 2^-24 * sum |scale q k| (E below; in the exponent it is a relative error of a
probability).  ex2.approx adds 2^-22, the exponent's own rounding 2^-23 of its size (scores here stay
below 2^6 in log2 units: 2^-17).  A probability is then rounded to fp16 (2^-11, half a step) and the
output to bf16 (2^-8 of its value); summing n of them in fp32 adds at most 2^-24 n <= 2^-11.
"""
import numpy as np
import pytest
import torch

import synth
from block_diffusion_draft_dflash_gb300 import _lib
from oracle import ddtree, kv4

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = 128 ** -0.5


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(DEV, torch.bfloat16)


def np64(t):
    return t.double().cpu().numpy()


def new_cache(n_layers, b, Hkv, cap, k_exp=0, v_exp=0, fill=0):
    c = _lib.Kv4Cache.empty(n_layers, b, Hkv, cap, k_exp, v_exp, DEV)
    for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales):
        t.fill_(fill)
    return c


def filled(seed, n_layers, b, Hkv, cap, lens, k_exp=0, v_exp=-2):
    """A cache whose slots below lens[s] hold rounded rows and whose other bytes are all ones (NaN as e4m3),
    with the float64 values of every row."""
    c = new_cache(n_layers, b, Hkv, cap, k_exp, v_exp, fill=255)
    k = synth.normal(seed, "k", (n_layers, b, Hkv, cap, 128))
    v = synth.normal(seed, "v", (n_layers, b, Hkv, cap, 128)) * 0.2
    kc, ks = kv4.round_rows(k, k_exp)
    vc, vs = kv4.round_rows(v, v_exp)
    for s, n in enumerate(lens):
        for t, x in ((c.k_codes, kc), (c.k_scales, ks), (c.v_codes, vc), (c.v_scales, vs)):
            t[:, s, :, :n] = torch.from_numpy(x[:, s, :, :n]).to(DEV)
    return c, kv4.values(kc, ks, k_exp), kv4.values(vc, vs, v_exp)


def ws_of(n):
    return _lib.Workspace(n, DEV)


# ------------------------------------------------------------------------------ append
def run_append(c, layer, k, v, lens, n_new=None, held=True):
    ws = ws_of(_lib.kv4_append_workspace_size())
    kh, vh = (torch.full_like(k, 7.0), torch.full_like(v, 7.0)) if held else (None, None)
    _lib.kv4_append(c, layer, k, v, i32(lens), ws, n_new=None if n_new is None else i32(n_new), k_held=kh, v_held=vh)
    torch.cuda.synchronize()
    return kh, vh, ws.status()


def awkward(shape, seed, exp):
    """Rows with every kind of block: normal, zeros, ties, one large value, beyond the scales' range on either side."""
    rng = np.random.default_rng(seed)
    x = rng.normal(0, 1, (*shape[:-1], 8, 16))
    kind = rng.integers(0, 8, shape[:-1] + (8,))
    x[kind == 0] = 0.0
    x[kind == 1] = rng.choice([0.25, 0.5, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -5.0, -3.5], x[kind == 1].shape)
    x[kind == 2] *= np.where(rng.random(x[kind == 2].shape) < 0.1, 100.0, 1.0)
    x[kind == 3] *= 2.0 ** -12
    x[kind == 4] *= 2.0 ** 14
    x[kind == 5] = np.where(rng.random(x[kind == 5].shape) < 0.5, -0.0, x[kind == 5] * 0.01)
    return torch.from_numpy((x * 2.0 ** exp).reshape(shape).astype(np.float32)).bfloat16()


@pytest.mark.parametrize("b,n,Hkv,cap,lens,n_new,k_exp,v_exp", [
    (1, 1, 1, 8, [0], None, 0, 0),
    (1, 1, 8, 16, [15], None, 0, -3),
    (3, 16, 8, 64, [0, 7, 48], [16, 5, 0], 0, -3),
    (2, 65, 3, 200, [100, 0], [64, 65], 3, -7),
    (1, 257, 4, 264, [7], None, -20, 20),
    (5, 130, 2, 136, [0, 1, 2, 3, 6], [130, 129, 128, 1, 130], 32, -32),
])
def test_append_bits(b, n, Hkv, cap, lens, n_new, k_exp, v_exp):
    c = new_cache(3, b, Hkv, cap, k_exp, v_exp, fill=0xA5)
    k, v = awkward((b, n, Hkv, 128), 1, k_exp), awkward((b, n, Hkv, 128), 2, v_exp)
    kh, vh, st = run_append(c, 1, k.to(DEV), v.to(DEV), lens, n_new)
    assert st == 0
    for x, codes, scales, held, exp in ((k, c.k_codes, c.k_scales, kh, k_exp), (v, c.v_codes, c.v_scales, vh, v_exp)):
        rc, rs = kv4.round_rows(x.double().numpy(), exp)
        val = kv4.values(rc, rs, exp)
        want_c, want_s = np.full(codes.shape, 0xA5, np.uint8), np.full(scales.shape, 0xA5, np.uint8)
        want_h = np.full(held.shape, 7.0)
        for s in range(b):
            m = n if n_new is None else n_new[s]
            want_c[1, s, :, lens[s]:lens[s] + m] = rc[s, :m].transpose(1, 0, 2)
            want_s[1, s, :, lens[s]:lens[s] + m] = rs[s, :m].transpose(1, 0, 2)
            want_h[s, :m] = val[s, :m]
        got_c = codes.cpu().numpy()
        # a code 8 (minus zero) and 0 stand for the same value
        plain = lambda z: np.where((z & 0x77) == 0, 0, np.where((z & 0x70) == 0, z & 0x0F, np.where((z & 7) == 0, z & 0xF0, z)))  # noqa: E731
        np.testing.assert_array_equal(plain(got_c), plain(want_c))
        np.testing.assert_array_equal(scales.cpu().numpy(), want_s)
        np.testing.assert_array_equal(np64(held), want_h)


def test_append_infinities_and_nan():
    c = new_cache(1, 1, 1, 8)
    x = torch.ones(1, 2, 1, 128)
    x[0, 0, 0, 3], x[0, 0, 0, 20], x[0, 1, 0, 5] = float("inf"), float("-inf"), float("nan")
    kh, vh, st = run_append(c, 0, x.bfloat16().to(DEV), torch.ones_like(x).bfloat16().to(DEV), [0])
    assert st == -6
    want = torch.ones(2, 128, dtype=torch.float64)
    want[0, :32] = 0.0                       # beside an infinity the scale is 448: 1 / 448 rounds to 0
    want[0, 3], want[0, 20], want[1, 5] = 2688.0, -2688.0, 0.0
    rc, rs = kv4.round_rows(x[0, :, 0].numpy(), 0)
    np.testing.assert_array_equal(kv4.values(rc, rs, 0)[0, :32], want[0, :32].numpy())
    np.testing.assert_array_equal(np64(kh)[0, :, 0], kv4.values(rc, rs, 0))
    assert np64(kh)[0, 1, 0, 5] == 0.0


def test_append_records_what_does_not_fit():
    c = new_cache(1, 3, 2, 16, fill=3)
    k = torch.ones(3, 4, 2, 128, device=DEV, dtype=torch.bfloat16)
    _, _, st = run_append(c, 0, k, k, [13, -1, 12])
    assert st == -4
    assert (c.k_codes[0, :2] == 3).all() and (c.v_scales[0, :2] == 3).all() and not (c.k_codes[0, 2, :, 12:] == 3).any()
    c2 = new_cache(1, 3, 2, 16, fill=3)
    _, _, st = run_append(c2, 0, k, k, [0, 0, 0], n_new=[5, -1, 0])
    assert st == -1 and (c2.k_codes == 3).all()


# --------------------------------------------------------------------------- attention
def random_tree(T, seed):
    rng = np.random.default_rng(seed)
    return np.array([-1] + [int(rng.integers(max(0, i - 40), i)) for i in range(1, T)])


def run_attention(c, layer, q, lens, anc, ws=None):
    b, T, Hq, _ = q.shape
    out = torch.full(q.shape, 9.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((b, T, Hq), 9.0, device=DEV)
    ws = ws or ws_of(_lib.kv4_attention_workspace_size(c, T, Hq))
    _lib.kv4_attention(c, layer, q, i32(lens), anc, SCALE, out, ws, lse=lse)
    torch.cuda.synchronize()
    return out, lse, ws.status()


def check_attention(got, got_lse, q, k, v, sets, rows, scale=SCALE):
    out, lse, size = kv4.attend(q[rows], k, v, scale, [sets[i] for i in rows])
    E = 130 * 2.0 ** -24 * np.abs(scale) * np.abs(q[rows]).sum(-1) * np.abs(k).max()
    rel = 2.0 ** -11 + 2.0 ** -11 + 2 * E + 2.0 ** -16
    # A probability is an fp16 number that carries 2^7 at least: where it is subnormal its rounding is off by 2^-25
    # at most, while the sum of all is 2^7 at least, the largest one's: 2^-32 of the value for each key that a row sees.
    low = 2.0 ** -32 * np.array([len(sets[i]) for i in rows])[:, None, None] * np.abs(v).max()
    assert (np.abs(got[rows] - out) <= 2.0 ** -8 * np.abs(out) + rel[..., None] * size + low).all()
    fin = np.isfinite(lse)
    np.testing.assert_array_equal(fin, np.isfinite(got_lse[rows]))
    tol = E + 2.0 ** -16 + 2.0 ** -22 * np.abs(np.where(fin, lse, 0))
    assert (np.abs(np.where(fin, got_lse[rows] - lse, 0)) <= tol).all()


CASES = [
    # b, T, Hq, Hkv, lens, cap, tree
    (1, 1, 1, 1, [0], 8, False),                       # one key
    (1, 1, 8, 2, [7], 8, False),                       # a full cache
    (3, 1, 8, 2, [0, 31, 32], 40, False),              # a stage's edges
    (2, 1, 32, 8, [1000, 33], 1008, False),
    (1, 1, 16, 1, [300], 304, False),                  # 16 heads on one kv head
    (2, 1, 40, 8, [257, 64], 264, False),              # 5 heads a kv head
    (1, 3, 5, 5, [97], 104, False),
    (5, 2, 6, 2, [0, 5, 63, 200, 513], 520, True),     # 3 heads a kv head, ragged
    (1, 16, 8, 2, [500], 520, False),                  # a chain of a draft block
    (2, 16, 32, 8, [90, 700], 720, True),
    (1, 17, 8, 8, [40], 64, True),
    (1, 33, 16, 2, [255], 288, True),                  # rows past two tiles
    (2, 65, 12, 4, [128, 3], 200, True),
    (1, 257, 8, 2, [300], 560, True),
    (1, 130, 16, 16, [0], 136, False),                 # a prompt into an empty cache
    (1, 300, 4, 2, [0], 304, False),
    (1, 129, 24, 2, [129], 264, True),                 # 12 heads a kv head: tiles cut nodes
    (1, 2, 512, 2, [50], 56, True),                    # 256 heads a kv head
]


@pytest.mark.parametrize("b,T,Hq,Hkv,lens,cap,tree", CASES)
def test_attention(b, T, Hq, Hkv, lens, cap, tree):
    c, k, v = filled(5, 2, b, Hkv, cap, [n + T for n in lens])
    q = bf16(synth.normal(6, "q", (b, T, Hq, 128)) * 1.5)
    parents = [random_tree(T, s) for s in range(b)] if tree else [None] * b
    anc = torch.from_numpy(np.stack([ddtree.ancestor_mask(p) for p in parents]).view(np.int32)).to(DEV) if tree else None
    out, lse, st = run_attention(c, 1, q, lens, anc)
    assert st == 0
    qn, o, l = np64(q), np64(out), np64(lse)
    rng = np.random.default_rng(0)
    for s in range(b):
        rows = sorted({0, T - 1, *rng.integers(0, T, 12).tolist()})
        sets = {i: list(range(lens[s])) + [lens[s] + j for j in kv4.visible(parents[s], T, i)] for i in rows}
        check_attention(o[s], l[s], qn[s], k[1, s].transpose(1, 0, 2), v[1, s].transpose(1, 0, 2), sets, rows)


def test_attention_long_cache_with_a_far_peak():
    # 20000 slots; one key agrees with the query, so that its weight is nearly all; another row sees a flat cache
    b, T, Hq, Hkv, N = 1, 1, 8, 2, 20000
    c, k, v = filled(7, 1, b, Hkv, N + 8, [N + T])
    q = synth.normal(8, "q", (b, T, Hq, 128))
    q[0, 0, 0] = k[0, 0, 0, 17777] * 4
    q[0, 0, 7] = 0
    q = bf16(q)
    out, lse, st = run_attention(c, 0, q, [N], None)
    assert st == 0
    check_attention(np64(out)[0], np64(lse)[0], np64(q)[0], k[0, 0].transpose(1, 0, 2), v[0, 0].transpose(1, 0, 2),
                    [list(range(N + T))], [0])


@pytest.mark.parametrize("T", [3, 70])
def test_attention_rows_that_see_nothing(T):
    c, k, v = filled(9, 1, 2, 2, 160, [T, 80 + T])
    anc = np.stack([ddtree.ancestor_mask(random_tree(T, 0))] * 2)
    anc[:, 1] = 0                                       # no ancestor, not even itself
    q = bf16(synth.normal(9, "q", (2, T, 4, 128)))
    out, lse, st = run_attention(c, 0, q, [0, 80], torch.from_numpy(anc.view(np.int32)).to(DEV))
    assert st == 0
    assert (out[0, 1] == 0).all() and (lse[0, 1] == -torch.inf).all()      # an empty cache: nothing at all
    check_attention(np64(out)[1], np64(lse)[1], np64(q)[1], k[0, 1].transpose(1, 0, 2), v[0, 1].transpose(1, 0, 2),
                    {1: list(range(80))}, [1])


@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -20, 2.0 ** 20])
def test_attention_queries_far_from_one(size):
    c, k, v = filled(10, 1, 1, 2, 64, [50])
    q = bf16(synth.normal(10, "q", (1, 2, 4, 128)) * size)
    out = torch.zeros_like(q)
    lse = torch.zeros(1, 2, 4, device=DEV)
    _lib.kv4_attention(c, 0, q, i32([48]), None, SCALE / size, out, ws_of(_lib.kv4_attention_workspace_size(c, 2, 4)), lse=lse)
    check_attention(np64(out)[0], np64(lse)[0], np64(q)[0], k[0, 0].transpose(1, 0, 2), v[0, 0].transpose(1, 0, 2),
                    [list(range(49)), list(range(50))], [0, 1], SCALE / size)


@pytest.mark.parametrize("T", [1, 4, 40])
@pytest.mark.parametrize("k_exp", [-32, 32])
def test_attention_queries_of_zeros(T, k_exp):
    # a padded row's weights are equal over what it sees, whatever the keys' exponent
    c, k, v = filled(27, 1, 1, 2, 200, [130 + T], k_exp=k_exp)
    q = synth.normal(27, "q", (1, T, 8, 128)) * 2.0 ** -k_exp
    q[0, T - 1, :] = 0
    q[0, 0, 3] = 0
    q = bf16(q)
    out, lse, st = run_attention(c, 0, q, [130], None)
    assert st == 0
    sets = {i: list(range(130 + i + 1)) for i in {0, T // 2, T - 1}}
    check_attention(np64(out)[0], np64(lse)[0], np64(q)[0], k[0, 0].transpose(1, 0, 2), v[0, 0].transpose(1, 0, 2), sets, sorted(sets))


@pytest.mark.parametrize("T", [1, 40])
def test_attention_records_lengths_that_do_not_fit(T):
    c, k, v = filled(11, 1, 3, 2, 80, [80, 80, 30 + T])
    q = bf16(synth.normal(11, "q", (3, T, 4, 128)))
    out, lse, st = run_attention(c, 0, q, [81 - T, -3, 30], None)
    assert st == -4
    assert (out[:2] == 0).all() and (lse[:2] == -torch.inf).all()
    sets = {i: list(range(30 + i + 1)) for i in (0, T - 1)}
    check_attention(np64(out)[2], np64(lse)[2], np64(q)[2], k[0, 2].transpose(1, 0, 2), v[0, 2].transpose(1, 0, 2), sets, list(sets))


@pytest.mark.parametrize("T,Hq", [(1, 8), (48, 8)])
def test_attention_repeats_and_replays(T, Hq):
    # the same bits every time; a captured call reads the lengths of its replay, on another stream
    c, k, v = filled(12, 1, 2, 2, 400, [400, 400])
    q = bf16(synth.normal(12, "q", (2, T, Hq, 128)))
    ws = ws_of(_lib.kv4_attention_workspace_size(c, T, Hq))
    a = run_attention(c, 0, q, [300, 111], None, ws)
    b = run_attention(c, 0, q, [300, 111], None, ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    lens, out, lse = i32([300, 111]), torch.zeros_like(q), torch.zeros(2, T, Hq, device=DEV)
    g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st), torch.cuda.graph(g, stream=st):
        _lib.kv4_attention(c, 0, q, lens, None, SCALE, out, ws, lse=lse)
    for new in ([300, 111], [0, 400 - T], [17, 32]):
        lens.copy_(i32(new))
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            g.replay()
        torch.cuda.synchronize()
        w = run_attention(c, 0, q, new, None)
        assert torch.equal(out, w[0]) and torch.equal(lse, w[1])


# --------------------------------------------------------------------------- weights
def run_weights(c, layer, q, lse, lens, score, n_rows=None, src=None, decay=1.0, score_out=None):
    ws = ws_of(_lib.kv4_attention_weights_workspace_size(c, q.shape[1], q.shape[2]))
    _lib.kv4_attention_weights(c, layer, q, lse, i32(lens), SCALE, score, ws, n_rows=None if n_rows is None else i32(n_rows),
                               src_slot=None if src is None else i32(src), decay=decay, score_out=score_out)
    torch.cuda.synchronize()
    return ws.status()


@pytest.mark.parametrize("b,T,Hq,Hkv,lens,cap,rows,decay", [
    (1, 1, 2, 2, [1], 8, None, 1.0),                                          # the row's own slot alone
    (2, 1, 8, 2, [128, 129], 136, None, 1.0),
    (1, 16, 32, 8, [600], 600, None, 0.5),                                    # a chain
    (3, 20, 10, 2, [150, 20, 3], 152, [[0, 3, 19], [0], []], 0.25),           # paths of a tree, one without rows
    (1, 70, 12, 1, [300], 304, [[0] + list(range(2, 66))], 0.0),              # 65 rows x 12 heads: several rounds
    (2, 5, 1, 1, [5, 40], 40, [[0, 1, 2, 3, 4], [0, 4]], 1.0),                # every slot is a row's own
    (2, 40, 32, 4, [2999, 130], 3000, None, 0.5),                             # 320 rows over parts of a long cache
    (2, 9, 16, 2, [1500, 3000], 3000, [[], [0, 1, 8]], 0.5),                  # a long sequence that only decays
    (1, 1, 128, 1, [1025], 1032, None, 1.0),                                  # 128 rows just fill a pass
])
def test_weights(b, T, Hq, Hkv, lens, cap, rows, decay):
    c, k, v = filled(13, 2, b, Hkv, cap, lens)
    q = bf16(synth.normal(13, "q", (b, T, Hq, 128)) * 1.5)
    qn = np64(q)
    paths = rows or [list(range(T))] * b
    lse = np.full((b, T, Hq), np.nan, np.float32)
    for s in range(b):
        kk = k[1, s].transpose(1, 0, 2)
        for j, node in enumerate(paths[s]):
            _, l, _ = kv4.attend(qn[s, node:node + 1], kk, kk, SCALE, [range(lens[s] - len(paths[s]) + j + 1)])
            lse[s, node] = l[0]
    score = torch.from_numpy(np.random.default_rng(0).random((2, b, Hkv, cap), np.float32)).to(DEV)
    before = score.clone()
    out = torch.full_like(score, 5.0)
    kw = {}
    if rows:
        m = max(len(r) for r in rows)
        src = np.full((b, m), -1)
        for s in range(b):
            src[s, :max(0, len(rows[s]) - 1)] = [lens[s] - len(rows[s]) + node for node in rows[s][1:]]
        kw = dict(n_rows=[len(r) for r in rows], src=src)
    assert run_weights(c, 1, q, torch.from_numpy(lse).to(DEV), lens, score, decay=decay, score_out=out, **kw) == 0
    assert torch.equal(score, before) and (out[0] == 5).all()
    for s in range(b):
        kk = k[1, s].transpose(1, 0, 2)
        want = kv4.weights(qn[s], lse[s], kk, SCALE, np64(before)[1, s], lens[s], paths[s], decay)
        E = 130 * 2.0 ** -24 * SCALE * np.abs(qn[s]).sum(-1).max() * np.abs(kk).max() + 2.0 ** -16
        got = np64(out)[1, s]
        assert (got[:, lens[s]:] == 5).all()
        assert (np.abs(got - want)[:, :lens[s]] <= (2 * E + 2.0 ** -20) * want[:, :lens[s]] + 1e-30).all()
    # in place gives the same bits
    assert run_weights(c, 1, q, torch.from_numpy(lse).to(DEV), lens, score, decay=decay, **kw) == 0
    for s in range(b):
        assert torch.equal(score[1, s, :, :lens[s]], out[1, s, :, :lens[s]])
        assert torch.equal(score[1, s, :, lens[s]:], before[1, s, :, lens[s]:])


def test_weights_ignore_rows_that_saw_nothing():
    c, k, v = filled(14, 1, 1, 2, 64, [40])
    q = bf16(synth.normal(14, "q", (1, 2, 4, 128)))
    lse = torch.full((1, 2, 4), -torch.inf, device=DEV)
    score = torch.ones(1, 1, 2, 64, device=DEV)
    assert run_weights(c, 0, q, lse, [40], score) == 0
    assert (score[..., :38] == 1).all() and (score[..., 38:40] == 0).all() and (score[..., 40:] == 1).all()


def test_weights_record_bad_lists():
    c, k, v = filled(15, 1, 4, 1, 16, [16] * 4)
    q = bf16(synth.normal(15, "q", (4, 3, 1, 128)))
    lse = torch.zeros(4, 3, 1, device=DEV)
    score = torch.ones(1, 4, 1, 16, device=DEV)
    # more rows than slots; a count below 0; more rows than the tree has; a length beyond the cache
    assert run_weights(c, 0, q, lse, [1, 8, 8, 17], score, n_rows=[2, -1, 4, 1]) in (-1, -4)
    assert (score == 1).all()
    # a node that the tree does not have gets no vote
    assert run_weights(c, 0, q, lse, [8] * 4, score, n_rows=[2] * 4, src=[[6 + 3], [5], [6 + 2], [-1]]) == -1


# ------------------------------------------------------------------- compact and evict
@pytest.mark.parametrize("n_layers,b,Hkv,cap,N,paths", [
    (1, 1, 1, 64, [10], [[1, 2, 5]]),
    (3, 4, 2, 120, [0, 7, 50, 90], [[3, 4, 9, 20], [], [1], [2, 3, 4, 5, 6, 7, 8]]),   # sources that are destinations too
    (2, 2, 3, 200, [3, 11], [list(range(1, 80, 2)), list(range(5, 105))]),               # more rows than one round
])
def test_compact(n_layers, b, Hkv, cap, N, paths):
    c, _, _ = filled(16, n_layers, b, Hkv, cap, [cap] * b)
    before = [t.cpu().numpy().copy() for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales)]
    m = max(len(p) for p in paths) + 1
    src = np.full((b, m), -1)
    for s, p in enumerate(paths):
        src[s, :len(p)] = [N[s] + x for x in p]
        for t in before:
            t[:, s, :, N[s] + 1:N[s] + 1 + len(p)] = t[:, s, :, [N[s] + x for x in p]].transpose(1, 2, 0, 3) if len(p) else t[:, s, :, N[s] + 1:N[s] + 1]
    ws = ws_of(_lib.kv4_compact_workspace_size())
    n_acc = [len(p) for p in paths]
    _lib.kv4_compact(c, i32(src), i32(n_acc), i32([n + 1 + a for n, a in zip(N, n_acc)]), ws)
    torch.cuda.synchronize()
    assert ws.status() == 0
    for t, w in zip((c.k_codes, c.k_scales, c.v_codes, c.v_scales), before):
        np.testing.assert_array_equal(t.cpu().numpy(), w)


def test_compact_records_bad_lists():
    c, _, _ = filled(17, 1, 5, 2, 32, [32] * 5)
    before = c.k_codes.clone()
    src = [[9, 8, 0], [3, 4, 5], [30, 31, 32], [12, 13, 14], [9, 10, 11]]
    ws = ws_of(_lib.kv4_compact_workspace_size())
    # descending; before its destination; beyond the cache; a count beyond the list; a length beyond the cache
    _lib.kv4_compact(c, i32(src), i32([2, 3, 3, 4, 3]), i32([10, 10, 12, 12, 33]), ws)
    torch.cuda.synchronize()
    assert ws.status() == -1 and torch.equal(c.k_codes, before)


def scores(kind, shape, seed):
    rng = np.random.default_rng(seed)
    if kind == "normal":
        x = rng.normal(size=shape)
    elif kind == "ties":
        x = rng.integers(0, 3, shape).astype(float)
    elif kind == "equal":
        x = np.full(shape, 0.25)
    else:
        x = rng.choice([0.0, -0.0, np.nan, np.inf, -np.inf, 1.0, 1 + 2.0 ** -23, -1.0, 1e-42], shape)
    return x.astype(np.float32)


@pytest.mark.parametrize("n_layers,b,Hkv,cap,lens,budget,sink,recent,kind", [
    (1, 1, 1, 8, [8], 1, 0, 0, "normal"),
    (1, 1, 1, 8, [8], 1, 0, 1, "normal"),
    (2, 3, 2, 104, [100, 0, 33], 33, 4, 8, "normal"),
    (1, 2, 3, 2008, [2001, 1024], 1024, 1, 100, "ties"),
    (1, 1, 2, 5000, [4999], 1500, 0, 0, "equal"),
    (1, 2, 2, 3000, [2999, 1030], 1025, 3, 7, "odd"),
    (1, 1, 1, 64, [50], 40, 40, 0, "normal"),              # sinks fill the budget
    (1, 1, 2, 9000, [8999], 8998, 0, 8998, "normal"),      # one slot goes
    (1, 1, 1, 70000, [70000], 3000, 4, 64, "ties"),
    (1, 1, 1, 70000, [69999], 30000, 4, 64, "normal"),     # longer than what one CTA holds
    (1, 1, 1, 20000, [19997], 300, 0, 1, "normal"),
])
def test_evict(n_layers, b, Hkv, cap, lens, budget, sink, recent, kind):
    c, _, _ = filled(18, n_layers, b, Hkv, cap, lens) if cap < 10000 else (new_cache(n_layers, b, Hkv, cap), None, None)
    if cap >= 10000:
        c.k_codes.random_(0, 256), c.v_scales.random_(0, 256)
    score = scores(kind, (n_layers, b, Hkv, cap), 3)
    to = new_cache(n_layers, b, Hkv, (budget + 15) // 8 * 8, 0, c.v_exp, fill=0x5A)
    sc, so = torch.from_numpy(score).to(DEV), torch.full(to.rows, 5.0, device=DEV)
    kept = torch.full((n_layers, b, Hkv, budget), -7, dtype=torch.int32, device=DEV)
    ws = ws_of(_lib.kv4_evict_workspace_size(c, budget))
    length = i32(lens)
    _lib.kv4_evict(c, sc, length, budget, sink, recent, to, so, length, kept, ws)       # the new length in place
    torch.cuda.synchronize()
    assert ws.status() == 0
    assert length.tolist() == [min(n, budget) for n in lens]
    src = [t.cpu().numpy() for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales)]
    dst = [t.cpu().numpy() for t in (to.k_codes, to.k_scales, to.v_codes, to.v_scales)]
    kept, so = kept.cpu().numpy(), so.cpu().numpy()
    for l in range(n_layers):
        for s in range(b):
            for h in range(Hkv):
                want = kv4.evict(score[l, s, h], lens[s], budget, sink, recent)
                n = len(want)
                assert kept[l, s, h].tolist() == want + [-1] * (budget - n)
                np.testing.assert_array_equal(so[l, s, h, :n], score[l, s, h, want])
                assert (so[l, s, h, n:] == 5).all()
                for x, y in zip(src, dst):
                    np.testing.assert_array_equal(y[l, s, h, :n], x[l, s, h, want])
                    assert (y[l, s, h, n:] == 0x5A).all()


def test_evict_records_lengths_that_do_not_fit():
    c, _, _ = filled(19, 1, 2, 1, 64, [64, 64])
    to = new_cache(1, 2, 1, 32, 0, -2, fill=1)
    kept, new_len = torch.zeros(1, 2, 1, 20, dtype=torch.int32, device=DEV), i32([9, 9])
    ws = ws_of(_lib.kv4_evict_workspace_size(c, 20))
    _lib.kv4_evict(c, torch.rand(1, 2, 1, 64, device=DEV), i32([65, -1]), 20, 0, 0, to, None, new_len, kept, ws)
    torch.cuda.synchronize()
    assert ws.status() == -4 and new_len.tolist() == [0, 0] and (kept == -1).all() and (to.k_codes == 1).all()


# ------------------------------------------------------------------------- all of them
def test_a_run_of_steps():
    """Prompt, then steps of tree verification: append, attend, walk, compact, vote; then eviction, and a step on
    the smaller cache.  Two layers, two sequences of uneven prompts, against the oracle on the oracle's own cache."""
    n_layers, b, Hq, Hkv, cap, T, P = 2, 2, 8, 2, 160, 24, [70, 41]
    rng = np.random.default_rng(20)
    c = new_cache(n_layers, b, Hkv, cap, 0, -2, fill=255)
    length, score = i32([0, 0]), torch.zeros(n_layers, b, Hkv, cap, device=DEV)
    held = [[[np.zeros((0, Hkv, 128))] * 2 for _ in range(b)] for _ in range(n_layers)]      # the oracle's rows
    want = np.zeros((n_layers, b, Hkv, cap))
    w1 = ws_of(_lib.kv4_append_workspace_size())
    wa = ws_of(_lib.accept_and_compact_workspace_size(b, T))
    wc = ws_of(_lib.kv4_compact_workspace_size())

    def put(layer, n, n_new):
        k, v = synth.normal(int(rng.integers(1 << 30)), "k", (2, b, n, Hkv, 128))
        k, v = bf16(k), bf16(v * 0.2)
        _lib.kv4_append(c, layer, k, v, length, w1, n_new=i32(n_new))
        rows = [kv4.values(*kv4.round_rows(np64(x), e), e) for x, e in ((k, 0), (v, -2))]
        for s in range(b):
            held[layer][s] = [np.concatenate([held[layer][s][i], rows[i][s, :n_new[s]]]) for i in range(2)]

    for layer in range(n_layers):
        put(layer, 70, P)
    length.copy_(i32(P))
    for step in range(3):
        N = length.tolist()
        parents = [random_tree(T, 100 * step + s) for s in range(b)]
        anc = torch.from_numpy(np.stack([ddtree.ancestor_mask(p) for p in parents]).view(np.int32)).to(DEV)
        qs, lses = [], []
        for layer in range(n_layers):
            put(layer, T, [T] * b)
            q = bf16(synth.normal(int(rng.integers(1 << 30)), "q", (b, T, Hq, 128)))
            out, lse, st = run_attention(c, layer, q, N, anc)
            assert st == 0
            for s in range(b):
                rows = [0, 5, T - 1]
                sets = {i: list(range(N[s])) + [N[s] + j for j in kv4.visible(parents[s], T, i)] for i in rows}
                check_attention(np64(out)[s], np64(lse)[s], np64(q)[s], *held[layer][s], sets, rows)
            qs.append(q), lses.append(lse)
        # a target that follows one branch: the path to a deep node
        tok = np.tile(np.arange(T), (b, 1))
        choice = np.full((b, T), -5)
        paths = []
        for s in range(b):
            path = kv4.visible(parents[s], T, T - 1 - s)
            for x, y in zip(path, path[1:]):
                choice[s, x] = y
            paths.append(path)
        acc = {x: torch.zeros(b, dtype=torch.int32, device=DEV) for x in ("n_new", "n_acc", "new_bonus")}
        acc.update({x: torch.zeros(b, 32, dtype=torch.int32, device=DEV) for x in ("acc_tok", "src_slot")})
        _lib.accept_and_compact(i32(choice), i32(tok), i32(np.stack(parents)), None, None, length, None, None, acc, wa, cap=cap)
        _lib.kv4_compact(c, acc["src_slot"], acc["n_acc"], length, wc)
        assert acc["n_new"].tolist() == [len(p) for p in paths]
        for layer in range(n_layers):
            ww = ws_of(_lib.kv4_attention_weights_workspace_size(c, T, Hq))
            _lib.kv4_attention_weights(c, layer, qs[layer], lses[layer], length, SCALE, score, ww, n_rows=acc["n_new"],
                                       src_slot=acc["src_slot"], decay=0.9)
            torch.cuda.synchronize()
            assert ww.status() == 0
            for s in range(b):
                n = N[s] + len(paths[s])
                held[layer][s] = [np.concatenate([x[:N[s]], x[N[s]:][paths[s]]]) for x in held[layer][s]]
                w = kv4.weights(np64(qs[layer])[s], np64(lses[layer])[s], held[layer][s][0], SCALE,
                                want[layer, s], n, paths[s], 0.9)
                want[layer, s] = w
                np.testing.assert_allclose(np64(score)[layer, s, :, :n], w[:, :n], rtol=2e-3, atol=1e-6)
        assert w1.status() == wa.status() == wc.status() == 0
        assert length.tolist() == [N[s] + len(paths[s]) for s in range(b)]
    # eviction into a cache of 64 slots, by the scores as the device holds them
    N = length.tolist()
    to = new_cache(n_layers, b, Hkv, 64, 0, -2, fill=255)
    kept = torch.zeros(n_layers, b, Hkv, 40, dtype=torch.int32, device=DEV)
    small = torch.zeros(to.rows, device=DEV)
    _lib.kv4_evict(c, score, length, 40, 2, 10, to, small, length, kept, ws_of(_lib.kv4_evict_workspace_size(c, 40)))
    torch.cuda.synchronize()
    assert length.tolist() == [40, 40]
    sc = score.cpu().numpy()
    for layer in range(n_layers):
        for s in range(b):
            for h in range(Hkv):
                assert kept[layer, s, h].tolist() == kv4.evict(sc[layer, s, h], N[s], 40, 2, 10)
            held[layer][s] = [np.stack([x[kept[layer, s, h].cpu().numpy(), h] for h in range(Hkv)], 1) for x in held[layer][s]]
    c = to
    put(0, 1, [1] * b)
    q = bf16(synth.normal(77, "q", (b, 1, Hq, 128)))
    out, lse, st = run_attention(c, 0, q, [40, 40], None)
    assert st == 0
    for s in range(b):
        check_attention(np64(out)[s], np64(lse)[s], np64(q)[s], *held[0][s], [list(range(41))], [0])


# ------------------------------------------------------------ shares, streams, failures
@pytest.mark.parametrize("b,T,Hq,Hkv,cap,tree", [
    (40, 1, 32, 8, 400, False),        # more (sequence, kv head) units than CTAs: shares cut the units of few rows
    (24, 65, 32, 8, 200, True),        # the same for tiles of 256 rows, the last of them with 4
    (70, 2, 8, 4, 96, False),          # more sequences than a warp has lanes
    (33, 20, 8, 2, 136, True),
    (3, 700, 8, 2, 1000, False),       # a chain's tiles differ in length
    (1, 513, 32, 8, 2000, True),
])
def test_attention_over_many_units(b, T, Hq, Hkv, cap, tree):
    rng = np.random.default_rng(b)
    lens = [int(x) for x in rng.integers(0, cap - T + 1, b)]
    lens[0], lens[-1] = 0, cap - T
    c, k, v = filled(21, 1, b, Hkv, cap, [n + T for n in lens])
    q = bf16(synth.normal(22, "q", (b, T, Hq, 128)) * 1.5)
    parents = [random_tree(T, s) for s in range(b)] if tree else [None] * b
    anc = torch.from_numpy(np.stack([ddtree.ancestor_mask(p) for p in parents]).view(np.int32)).to(DEV) if tree else None
    out, lse, st = run_attention(c, 0, q, lens, anc)
    assert st == 0
    qn, o, l = np64(q), np64(out), np64(lse)
    for s in sorted({0, b - 1, *rng.integers(0, b, 6).tolist()}):
        rows = sorted({0, T - 1, *rng.integers(0, T, 5).tolist()})
        sets = {i: list(range(lens[s])) + [lens[s] + j for j in kv4.visible(parents[s], T, i)] for i in rows}
        check_attention(o[s], l[s], qn[s], k[0, s].transpose(1, 0, 2), v[0, s].transpose(1, 0, 2), sets, rows)


def test_weights_of_a_long_chain_over_many_units():
    # 300 rows x 2 heads: ten rounds of rows; 80 units
    b, T, Hq, Hkv, cap = 10, 300, 16, 8, 360
    lens = [300 + 6 * s for s in range(b)]
    c, k, v = filled(23, 1, b, Hkv, cap, lens)
    q = bf16(synth.normal(23, "q", (b, T, Hq, 128)))
    out, lse, st = run_attention(c, 0, q, [n - T for n in lens], None)
    assert st == 0
    score = torch.zeros(1, b, Hkv, cap, device=DEV)
    assert run_weights(c, 0, q, lse, lens, score) == 0
    # every (row, head) distributes weight 1; 2 heads a kv head
    np.testing.assert_allclose(np64(score).sum(-1), np.full((1, b, Hkv), 2.0 * T), rtol=2e-5)
    for s in (0, b - 1):
        kk = k[0, s].transpose(1, 0, 2)
        want = kv4.weights(np64(q)[s], np64(lse)[s], kk, SCALE, np.zeros((Hkv, cap)), lens[s], list(range(T)))
        E = 130 * 2.0 ** -24 * SCALE * np.abs(np64(q)[s]).sum(-1).max() * np.abs(kk).max() + 2.0 ** -16
        assert (np.abs(np64(score)[0, s] - want) <= (2 * E + 300 * 2.0 ** -24) * want + 1e-30).all()


def test_calls_on_two_streams():
    # two attentions at once, each with a workspace of its own, give what they give alone
    cases = []
    for seed, T, N in ((24, 1, 3000), (25, 80, 900)):
        c, _, _ = filled(seed, 1, 2, 2, (N + 87) // 8 * 8, [N + T] * 2)     # cap is a multiple of 8
        q = bf16(synth.normal(seed, "q", (2, T, 8, 128)))
        lens = i32([N, N // 2])
        alone = run_attention(c, 0, q, [N, N // 2], None)
        cases.append((c, q, lens, alone, torch.zeros_like(q), ws_of(_lib.kv4_attention_workspace_size(c, T, 8)), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for c, q, lens, _, out, ws, st in cases:
            with torch.cuda.stream(st):
                _lib.kv4_attention(c, 0, q, lens, None, SCALE, out, ws)
    torch.cuda.synchronize()
    for c, q, lens, alone, out, ws, st in cases:
        assert ws.status() == 0 and torch.equal(out, alone[0])


@pytest.mark.parametrize("T", [1, 4, 60])
def test_attention_gives_up_when_its_waits_run_out(T):
    # a limit of 1 ns on every wait: the call may report DF_ERR_TIMEOUT, and it ends; the next one is right
    c, k, v = filled(26, 1, 2, 2, 2400, [2300, 2300])
    q = bf16(synth.normal(26, "q", (2, T, 8, 128)))
    ws = ws_of(_lib.kv4_attention_workspace_size(c, T, 8))
    good = run_attention(c, 0, q, [2200, 500], None, ws)
    assert good[2] == 0
    ws.configure(wait_limit_ns=1)
    for _ in range(3):
        assert run_attention(c, 0, q, [2200, 500], None, ws)[2] in (0, -7)
    ws.configure()
    again = run_attention(c, 0, q, [2200, 500], None, ws)
    assert again[2] == 0 and torch.equal(again[0], good[0]) and torch.equal(again[1], good[1])


def test_weights_give_up_when_their_waits_run_out():
    c, k, v = filled(28, 1, 2, 2, 2400, [2300, 900])
    q = bf16(synth.normal(28, "q", (2, 40, 8, 128)))
    out, lse, st = run_attention(c, 0, q, [2260, 860], None)
    assert st == 0
    ws = ws_of(_lib.kv4_attention_weights_workspace_size(c, 40, 8))
    score, lens = torch.zeros(1, 2, 2, 2400, device=DEV), i32([2300, 900])

    def call():
        to = torch.zeros_like(score)
        _lib.kv4_attention_weights(c, 0, q, lse, lens, SCALE, score, ws, score_out=to)
        torch.cuda.synchronize()
        return to, ws.status()

    good = call()
    assert good[1] == 0
    ws.configure(wait_limit_ns=1)
    for _ in range(3):
        assert call()[1] in (0, -7)
    ws.configure()
    again = call()
    assert again[1] == 0 and torch.equal(again[0], good[0])


def test_binding_refuses_what_the_kernels_would_misread():
    c = new_cache(1, 2, 2, 64)
    q, out = torch.zeros(2, 3, 4, 128, dtype=torch.bfloat16, device=DEV), torch.zeros(2, 3, 4, 128, dtype=torch.bfloat16, device=DEV)
    ws = ws_of(_lib.kv4_attention_workspace_size(c, 3, 4))
    lens = i32([0, 0])
    for bad in (dict(q=q.float()), dict(q=q.transpose(1, 2)), dict(q=q[:1]), dict(cache_len=lens.long()), dict(cache_len=lens.cpu()),
                dict(anc=torch.zeros(2, 3, 2, dtype=torch.int32, device=DEV)), dict(out=out[:, :2]), dict(lse=torch.zeros(2, 3, 3, device=DEV))):
        kw = dict(q=q, cache_len=lens, anc=None, out=out, lse=None)
        kw.update(bad)
        with pytest.raises(ValueError):
            _lib.kv4_attention(c, 0, kw["q"], kw["cache_len"], kw["anc"], SCALE, kw["out"], ws, lse=kw["lse"])
    with pytest.raises(_lib.StatusError):
        _lib.kv4_attention(c, 0, q, lens, None, SCALE, out, ws_of(256))           # a workspace too small
    with pytest.raises(ValueError):
        _lib.kv4_attention_weights(c, 0, q, torch.zeros(2, 3, 4, device=DEV), lens, SCALE, torch.zeros(1, 2, 2, 63, device=DEV), ws)
    with pytest.raises(ValueError):
        _lib.kv4_append(c, 0, q, q, lens, ws)                                      # 4 heads, the cache has 2


# ------------------------------------------------------- rows and lists at the edge of a call
def vote(c, k, q, lse, lens, paths, scale=SCALE, decay=1.0, layer=0, cap=None):
    """Scores of a call over paths (nodes of each sequence), and what the oracle makes of it."""
    b, m = len(paths), max(2, max(len(p) for p in paths))
    src = np.full((b, m), -1)
    for s, p in enumerate(paths):
        src[s, :len(p) - 1] = [lens[s] - len(p) + node for node in p[1:]]
    score = torch.from_numpy(np.random.default_rng(1).random(c.rows, np.float32)).to(DEV)
    before = np64(score)
    ws = ws_of(_lib.kv4_attention_weights_workspace_size(c, q.shape[1], q.shape[2]))
    _lib.kv4_attention_weights(c, layer, q, lse, i32(lens), scale, score, ws, n_rows=i32([len(p) for p in paths]), src_slot=i32(src),
                               decay=decay)
    torch.cuda.synchronize()
    want = [kv4.weights(np64(q)[s], np64(lse)[s], k[layer, s].transpose(1, 0, 2), scale, before[layer, s], lens[s], p, decay)
            for s, p in enumerate(paths)]
    return np64(score)[layer], want, ws.status()


def path_lse(k, q, lens, paths, scale):
    """The oracle's log-sums of the rows of each path."""
    lse = np.full(q.shape[:3], np.nan, np.float32)
    for s, p in enumerate(paths):
        kk = k[0, s].transpose(1, 0, 2)
        for j, node in enumerate(p):
            lse[s, node] = kv4.attend(np64(q)[s, node:node + 1], kk, kk, scale, [range(lens[s] - len(p) + j + 1)])[1][0]
    return torch.from_numpy(lse).to(DEV)


def check_votes(got, want, q, k, lens, paths, scale=SCALE):
    # as in test_weights: a score is off by E at most, a weight by twice that of its value; a sum of rows x heads terms
    for s, p in enumerate(paths):
        n = lens[s]
        E = 130 * 2.0 ** -24 * scale * np.abs(np64(q)[s]).sum(-1).max() * np.abs(k[0, s, :, :n]).max() + 2.0 ** -16
        assert (np.abs(got[s][:, :n] - want[s][:, :n]) <= (2 * E + 2.0 ** -20) * want[s][:, :n] + 1e-30).all()


@pytest.mark.parametrize("k_exp,scale", [(-32, SCALE), (32, SCALE), (-22, SCALE), (0, 1e-8), (0, 2.0 ** -120)])
@pytest.mark.parametrize("Hq", [2, 16])
def test_weights_of_query_rows_of_zeros(k_exp, scale, Hq):
    # such a row's weights are equal over what it sees, and nothing behind that: the first row, one of the path, one head
    T, lens = 9, [140, 30]
    c, k, v = filled(29, 1, 2, 2, 200, lens, k_exp=k_exp)
    q = synth.normal(29, "q", (2, T, Hq, 128)) * 2.0 ** -k_exp
    q[:, 0] = 0
    q[:, 4] = 0
    q[:, 2, Hq - 1] = 0
    q = bf16(q)
    paths = [[0, 2, 4, 7, 8], [0, 1, 4]]
    got, want, st = vote(c, k, q, path_lse(k, q, lens, paths, scale), lens, paths, scale)
    assert st == 0
    check_votes(got, want, q, k, lens, paths, scale)


# ------------------------------------------------------------------ calls that give up
def random_cache(b, Hkv, cap):
    c = new_cache(1, b, Hkv, cap, 0, -2)
    for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales):
        t.random_(0, 256)
    return c


@pytest.mark.parametrize("b,T,Hq,Hkv,lens", [
    (1, 1, 8, 2, [0]),                     # few rows: one stage
    (2, 1, 8, 2, [2300, 500]),
    (2, 4, 8, 2, [2300, 500]),             # 16 rows
    (40, 1, 32, 8, [300] * 40),            # several units a CTA
    (1, 17, 8, 8, [0]),                    # tcgen05, half a tile: one stage, then the issuer has nothing left
    (2, 60, 8, 2, [2300, 500]),
    (1, 513, 8, 8, [0]),                   # whole tiles
    (2, 300, 8, 2, [6000, 500]),
    (24, 65, 32, 8, [130] * 24),           # several units a CTA
])
def test_attention_that_is_held_gives_up(b, T, Hq, Hkv, lens):
    # held for 20 ms behind its first copies and products: the call reports it and ends, and the next one is right
    c = random_cache(b, Hkv, max(lens) // 8 * 8 + (T + 15) // 8 * 8)
    q = bf16(synth.normal(30, "q", (b, T, Hq, 128)))
    ws = ws_of(_lib.kv4_attention_workspace_size(c, T, Hq))
    good = run_attention(c, 0, q, lens, None, ws)
    assert good[2] == 0
    for _ in range(3):
        ws.configure(wait_limit_ns=20_000_000, hold=True)
        assert run_attention(c, 0, q, lens, None, ws)[2] == -7
        ws.configure()
        again = run_attention(c, 0, q, lens, None, ws)
        assert again[2] == 0 and torch.equal(again[0], good[0]) and torch.equal(again[1], good[1])


@pytest.mark.parametrize("b,T,Hq,Hkv,lens", [
    (1, 1, 2, 2, [8]),                     # one block, then the issuer has nothing left
    (2, 40, 8, 2, [2300, 900]),
    (2, 100, 16, 2, [2300, 900]),          # several passes
    (8, 16, 32, 8, [4096] * 8),            # more blocks a CTA than products in flight
    (40, 16, 32, 8, [300] * 40),           # several units a CTA
])
def test_weights_that_are_held_give_up(b, T, Hq, Hkv, lens):
    c = random_cache(b, Hkv, max(lens) // 8 * 8 + 8)
    q = bf16(synth.normal(31, "q", (b, T, Hq, 128)))
    lse = run_attention(c, 0, q, [n - T for n in lens], None)[1]
    ws = ws_of(_lib.kv4_attention_weights_workspace_size(c, T, Hq))
    score, length = torch.zeros(c.rows, device=DEV), i32(lens)

    def call():
        to = torch.zeros_like(score)
        _lib.kv4_attention_weights(c, 0, q, lse, length, SCALE, score, ws, score_out=to)
        torch.cuda.synchronize()
        return to, ws.status()

    good = call()
    assert good[1] == 0
    for _ in range(3):
        ws.configure(wait_limit_ns=20_000_000, hold=True)
        assert call()[1] == -7
        ws.configure()
        again = call()
        assert again[1] == 0 and torch.equal(again[0], good[0])


@pytest.mark.parametrize("b,T,n,at,bad", [
    (3, 3, 2, 0, 3),                       # a list of one entry: behind the tree, before it, far off on either side
    (3, 3, 2, 0, -1),
    (2, 40, 9, 7, 40),
    (2, 40, 9, 0, 2 ** 31 - 1),
    (2, 40, 9, 4, -2 ** 31),
    (2, 90, 70, 33, -1),                   # beyond the first lanes, rows of several passes
    (2, 90, 70, 68, 90),
])
def test_weights_leave_a_sequence_with_a_bad_list_out(b, T, n, at, bad):
    # its scores stay as they were, decay or not, in place or not; the other sequences' votes are right
    lens = [300 + 7 * s for s in range(b)]
    c, k, v = filled(32, 1, b, 2, 400, lens)
    q = bf16(synth.normal(32, "q", (b, T, 8, 128)))
    paths = [list(range(n))] * b
    lse = path_lse(k, q, lens, paths, SCALE)
    src = np.array([[lens[s] - n + j for j in range(1, n)] for s in range(b)])
    src[0, at] = np.clip(lens[0] - n + bad, -2 ** 31, 2 ** 31 - 1)
    score = torch.rand(c.rows, device=DEV)
    before, out = score.clone(), torch.full_like(score, 5.0)
    kw = dict(n_rows=[n] * b, src=src, decay=0.5)
    assert run_weights(c, 0, q, lse, lens, score, score_out=out, **kw) == -1
    assert torch.equal(score, before) and (out[0, 0] == 5).all()
    assert run_weights(c, 0, q, lse, lens, score, **kw) == -1
    assert torch.equal(score[0, 0], before[0, 0])
    for s in range(1, b):
        assert torch.equal(score[0, s, :, :lens[s]], out[0, s, :, :lens[s]])
    check_votes(np64(score)[0][1:], [kv4.weights(np64(q)[s], np64(lse)[s], k[0, s].transpose(1, 0, 2), SCALE, np64(before)[0, s], lens[s],
                                                 paths[s], 0.5) for s in range(1, b)], q[1:], k[:, 1:], lens[1:], paths[1:])


@pytest.mark.parametrize("size", [2.0 ** 112, 2.0 ** 116, 2.0 ** 119, 2.0 ** 124])
@pytest.mark.parametrize("T", [1, 4, 40])
def test_attention_and_weights_of_the_largest_queries(T, size):
    # a bf16 row up to the type's largest, under a scale that makes ordinary scores of it
    c, k, v = filled(33, 1, 1, 2, 200, [130 + T])
    q = bf16(synth.normal(33, "q", (1, T, 8, 128)).clip(-7.9, 7.9) * size)
    assert torch.isfinite(q).all()
    scale, kk, vv = 0.1 / size, k[0, 0].transpose(1, 0, 2), v[0, 0].transpose(1, 0, 2)
    out, lse = torch.zeros_like(q), torch.zeros(1, T, 8, device=DEV)
    ws = ws_of(_lib.kv4_attention_workspace_size(c, T, 8))
    if scale < 2.0 ** -126:      # not a normal number, and refused: the smallest power of two that is taken with room
        with pytest.raises(_lib.StatusError):
            _lib.kv4_attention(c, 0, q, i32([130]), None, scale, out, ws, lse=lse)
        scale = 2.0 ** -125
    _lib.kv4_attention(c, 0, q, i32([130]), None, scale, out, ws, lse=lse)
    torch.cuda.synchronize()
    assert ws.status() == 0
    sets = {i: list(range(130 + i + 1)) for i in {0, T // 2, T - 1}}
    check_attention(np64(out)[0], np64(lse)[0], np64(q)[0], kk, vv, sets, sorted(sets), scale)
    lens, paths = [130 + T], [list(range(T))]
    got, want, st = vote(c, k, q, path_lse(k, q, lens, paths, scale), lens, paths, scale)
    assert st == 0
    check_votes(got, want, q, k, lens, paths, scale)


@pytest.mark.parametrize("what", ["lse", "q", "both", "low"])
def test_weights_keep_a_nan_to_the_slots_that_its_row_sees(what):
    # row 2 of 5 has a NaN (or a log-sum that no score is as low as): the path's slots behind its own stay numbers
    lens, T = [140, 40], 5
    c, k, v = filled(34, 1, 2, 2, 200, lens)
    q = bf16(synth.normal(34, "q", (2, T, 8, 128)))
    paths = [list(range(T))] * 2
    lse = path_lse(k, q, lens, paths, SCALE)
    if what in ("lse", "both"):
        lse[0, 2, 5] = torch.nan
    if what in ("q", "both"):
        q[0, 2, 5, 77] = torch.nan
    if what == "low":
        lse[0, 2, 5] = -3e38
    with np.errstate(over="ignore", invalid="ignore"):
        got, want, st = vote(c, k, q, lse, lens, paths)
    assert st == 0
    n, bad = lens[0] - T + 3, (np.isinf if what == "low" else np.isnan)      # head 5 belongs to kv head 1
    assert bad(got[0][1, :n]).all() and bad(want[0][1, :n]).all()
    rows = bf16(np.nan_to_num(np64(q)))
    got[0][1, :n], want[0][1, :n] = 0, 0
    check_votes(got, want, rows, k, lens, paths)


@pytest.mark.parametrize("T,N", [(1, 50), (1, 9000), (4, 900), (40, 3000), (200, 700), (300, 0)])
def test_attention_of_a_row_with_a_nan(T, N):
    # its output and log-sum are NaN, not those of a row that sees nothing; the other heads and rows are right
    c, k, v = filled(35, 1, 1, 2, (N + T + 7) // 8 * 8, [N + T])
    q = bf16(synth.normal(35, "q", (1, T, 8, 128)))
    clean = q.clone()
    q[0, T - 1, 3, 100] = torch.nan
    out, lse, st = run_attention(c, 0, q, [N], None)
    assert st == 0
    assert torch.isnan(out[0, T - 1, 3]).all() and torch.isnan(lse[0, T - 1, 3])
    want, want_lse, _ = run_attention(c, 0, clean, [N], None)
    out[0, T - 1, 3], lse[0, T - 1, 3] = want[0, T - 1, 3], want_lse[0, T - 1, 3]
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    sets = {i: list(range(N + i + 1)) for i in {0, T - 1}}
    check_attention(np64(out)[0], np64(lse)[0], np64(clean)[0], k[0, 0].transpose(1, 0, 2), v[0, 0].transpose(1, 0, 2), sets, sorted(sets))


def test_weights_with_lists_without_entries():
    # the root alone may vote: more rows do not fit such a list, and they are not the rows of a chain
    lens = [60, 20]
    c, k, v = filled(36, 1, 2, 2, 64, lens)
    q = bf16(synth.normal(36, "q", (2, 3, 4, 128)))
    lse = path_lse(k, q, lens, [[0, 1], [0]], SCALE)
    score = torch.rand(c.rows, device=DEV)
    before = score.clone()
    empty = torch.zeros(2, 0, dtype=torch.int32, device=DEV)
    ws = ws_of(_lib.kv4_attention_weights_workspace_size(c, 3, 4))
    _lib.kv4_attention_weights(c, 0, q, lse, i32(lens), SCALE, score, ws, n_rows=i32([2, 1]), src_slot=empty)
    torch.cuda.synchronize()
    assert ws.status() == -1 and torch.equal(score[0, 0], before[0, 0])
    want = kv4.weights(np64(q)[1], np64(lse)[1], k[0, 1].transpose(1, 0, 2), SCALE, np64(before)[0, 1], 20, [0])
    check_votes(np64(score)[0][1:], [want], q[1:], k[:, 1:], [20], [[0]])
