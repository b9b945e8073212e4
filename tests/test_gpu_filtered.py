"""The target forward that draws under settings, the lists that it hands out, and a step that teaches: against the oracle.

A node's list holds its first tokens with their fp32 logits as the GPU made them, so draws among at most that many tokens
can be repeated exactly from it (oracle/rows.py), whatever the forward's own rounding; the lists themselves are compared
with the oracle's logits within the bound for bf16 activations (2e-2 of the largest)."""
import numpy as np
import pytest
import torch

import synth
from block_diffusion_draft_dflash_gb300 import _lib, engine
from oracle import ddtree, rows, sample, step

from gpu_util import bf16_dev, cache_to_oracle

pytestmark = pytest.mark.gpu
TS, DS = synth.SMALL_TARGET, synth.SMALL_DRAFTER
DEV = "cuda"


@pytest.fixture(scope="module")
def models():
    tw = synth.target_weights(TS, 2201)
    dw = synth.drafter_weights(DS, tw, TS.n_feat, 2201)
    tm = engine.DeviceModel.from_host(tw)
    return tw, tm, engine.DeviceModel.from_host(dw, embed=tm.embed, n_feat=TS.n_feat)


def f32(v):
    return torch.tensor(v, dtype=torch.float32, device=DEV)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def number(seed, s, n):
    return float(sample.uniforms(seed, s, n, 1)[0])


def check_draws(choice, ids, vals, settings, seed, positions):
    """choice [b][T] from the nodes' lists; settings (T, k, p, min_p) of each sequence, k at most the lists' length."""
    for s, (temp, k, p, low) in enumerate(settings):
        temp, p, low = (float(np.float32(v)) for v in (temp, p, low))
        for i in range(choice.shape[1]):
            at, _, _ = rows.draw(vals[s, i], number(seed, s, int(positions[s, i]) + 1), temperature=temp, top_k=k, top_p=p, min_p=low)
            # the list is in order, so a place in it orders as ids do among equal logits
            assert choice[s, i] == ids[s, i, at], (s, i)


def forward(tm, b, T, tok, depth, anc, k, v, clen, settings, seed, K, temperature=1.0):
    ws = _lib.Workspace(_lib.target_tree_forward_filtered_workspace_size(tm.cfg, b, T))
    choice = torch.full((b, T), -7, dtype=torch.int32, device=DEV)
    top = dict(top_id=torch.zeros(b, T, K, dtype=torch.int32, device=DEV), top_val=torch.zeros(b, T, K, device=DEV),
               top_lse=torch.zeros(b, T, device=DEV), top_temperature=temperature) if K else {}
    Ts, ks, ps, lows = zip(*settings)
    _lib.target_tree_forward_filtered(tm.cfg, tm.weights, tok, depth, anc, k, v, clen, choice, None, ws, f32(Ts), i32(ks),
                                      f32(ps), f32(lows), seed, **top)
    torch.cuda.synchronize()
    return choice.cpu().numpy(), {n: t.cpu().numpy() for n, t in top.items() if torch.is_tensor(t)}, ws.status()


@pytest.mark.parametrize("b,B,K", [(2, 20, 64), (5, 256, 40)])      # one block of logits, and two
def test_filtered_forward(models, b, B, K):
    tw, tm, _ = models
    T, cap, seed = B + 1, 512, 0x1122334455
    Ns = [37, 150, 5, 80, 200][:b]
    settings = [(0.6, 20, 0.95, 0.0), (1.0, 40, 1.0, 0.02), (0.0, 0, 1.0, 0.0), (1.5, 40, 0.7, 0.0), (0.8, 1, 1.0, 0.0)][:b]
    rng = np.random.default_rng(B)
    kc = synth.normal(B, "ftk", (TS.n_layers, b, TS.n_kv_heads, cap, 128))
    vc = synth.normal(B, "ftv", (TS.n_layers, b, TS.n_kv_heads, cap, 128))
    trees = []
    for s in range(b):
        kc[:, s, :, Ns[s]:] = 0
        vc[:, s, :, Ns[s]:] = 0
        t = ddtree.build_tree(ddtree.log_softmax(rng.normal(0, 2, size=(7, TS.vocab))), B)
        t["tok"][0] = int(rng.integers(0, TS.vocab))
        trees.append(t)
    st = lambda key: torch.from_numpy(np.stack([t[key] for t in trees]).astype(np.int32)).cuda()
    anc = torch.from_numpy(np.stack([ddtree.ancestor_mask(t["parent"]) for t in trees]).view(np.int32)).cuda()
    k, v = bf16_dev(kc), bf16_dev(vc).transpose(-1, -2).contiguous()
    choice, top, status = forward(tm, b, T, st("tok"), st("depth"), anc, k, v, i32(Ns), settings, seed, K)
    assert status == 0
    pos = np.stack([Ns[s] + trees[s]["depth"] for s in range(b)])
    check_draws(choice, top["top_id"], top["top_val"], settings, seed, pos)
    for s in range(min(b, 2)):
        cache = cache_to_oracle(torch.from_numpy(kc).to(torch.bfloat16), torch.from_numpy(vc).transpose(-1, -2), s)
        _, _, logits = step.target_tree_forward(tw, trees[s]["tok"], trees[s]["parent"], trees[s]["depth"], cache, Ns[s])
        bound = 2e-2 * np.abs(logits).max()
        got = np.take_along_axis(logits, top["top_id"][s].astype(np.int64), -1)
        assert np.abs(got - top["top_val"][s]).max() <= bound
        assert (top["top_val"][s][:, -1] >= np.sort(logits, -1)[:, -K] - bound).all()
        lse = np.log(np.exp(logits - logits.max(-1, keepdims=True)).sum(-1)) + logits.max(-1)
        assert np.abs(lse - top["top_lse"][s]).max() <= bound
    # without lists: the same choices
    again, _, _ = forward(tm, b, T, st("tok"), st("depth"), anc, bf16_dev(kc), bf16_dev(vc).transpose(-1, -2).contiguous(),
                          i32(Ns), settings, seed, 0)
    np.testing.assert_array_equal(again, choice)


def test_filtered_forward_records_a_bad_setting(models):
    _, tm, _ = models
    k = torch.zeros(TS.n_layers, 2, TS.n_kv_heads, 64, 128, dtype=torch.bfloat16, device=DEV)
    choice, _, status = forward(tm, 2, 3, i32([[1, 2, 3]] * 2), None, None, k, k.transpose(-1, -2).contiguous(), i32([0, 0]),
                                [(1.0, 5, 1.0, 0.0), (1.0, 5, 2.0, 0.0)], 1, 0)
    assert status == -1 and (choice[1] == -1).all() and (choice[0] >= 0).all()


@pytest.mark.parametrize("mode,B", [("tree", 24), ("chain", 0)])
def test_steps_that_teach(models, mode, B):
    _, tm, dm = models
    b, P, cap, seed, K = 2, 40, 512, 99, 32
    prompt = synth.uniform_ints(2202, "prompt", (b, P), 0, TS.vocab)
    dec = engine.SpecDecoder(tm, dm, b, B, cap, prompt_len=P, mode=mode, temperature=0.8, seed=seed, top_k=K, top_p=0.97, teach=K)
    dec.settings["temperature"][1] = 0.0              # one sequence decodes greedily
    dec.prefill(torch.from_numpy(prompt).cuda())
    weight = f32(np.exp(-np.arange(dec.D) / 4.0)).expand(b, -1).contiguous()
    rng, n_acc = np.random.default_rng(7), 0

    def plant(d):      # lean the drafter on the target's next choices: an untimed pass along them
        for s in range(b):
            for j in range(d.D):
                if rng.random() < 0.7 and want[s][j] is not None:
                    d.logprobs[s, j, want[s][j]] += 14.0

    for _ in range(5):
        # what the target chooses from here, token after token
        want = [[None] * dec.D for _ in range(b)]
        N, tok = dec.cache_len.clone(), dec.bonus.clone()
        kc, vc = dec.k_cache.clone(), dec.v_cache.clone()
        ws = _lib.Workspace(_lib.target_tree_forward_filtered_workspace_size(tm.cfg, b, 1))
        for j in range(dec.D):
            c = torch.zeros(b, 1, dtype=torch.int32, device=DEV)
            _lib.target_tree_forward_filtered(tm.cfg, tm.weights, tok[:, None].contiguous(), None, None, kc, vc, N, c, None, ws,
                                              seed=seed, **dec.settings)
            for s in range(b):
                want[s][j] = int(c[s, 0])
            tok, N = c[:, 0].contiguous(), N + 1
        dec.plant = plant
        N0 = dec.cache_len.cpu().numpy()
        dec.step()
        loss = dec.distill(weight)
        torch.cuda.synchronize()
        assert dec.status() == 0
        ids, vals, lse = (dec.top[n].cpu().numpy() for n in ("top_id", "top_val", "top_lse"))
        depth = dec.tree["depth"].cpu().numpy()
        settings = [(0.8, K, 0.97, 0.0), (0.0, K, 0.97, 0.0)]
        check_draws(dec.choice.cpu().numpy(), ids, vals, settings, seed, N0[:, None] + depth)
        acc = dec.acc["acc_tok"].cpu().numpy()
        for s in range(b):
            a = int(dec.acc["n_acc"][s])
            n_acc += a
            parent, tokens, choice = (t[s].cpu().numpy() for t in (dec.tree["parent"], dec.tree["tok"], dec.choice))
            path = [0]
            while True:
                nxt = [i for i in range(dec.T) if parent[i] == path[-1] and tokens[i] == choice[path[-1]]]
                if not nxt:
                    break
                path.append(nxt[0])
            assert len(path) == a + 1
            assert [int(choice[i]) for i in path] == acc[s][:a + 1].tolist()
            row = dec.teacher_row[s].tolist()
            assert row == [s * dec.T + i for i in path[:dec.D]] + [-1] * (dec.D - len(path[:dec.D]))
            for d in range(dec.D):
                if row[d] < 0:
                    assert float(loss[s, d]) == 0 and not dec.grad[s, d].any()
                    continue
                i = path[d]
                z = dec.logprobs[s, d].double().cpu().numpy()
                l, g, _ = rows.distill(z, ids[s, i], vals[s, i], float(lse[s, i]), 1.0, float(weight[s, d]))
                # fp32 sums of 4000 terms: 2^-24 (4000 / 512 + 48) of the masses, ln's of up to 2^5
                assert abs(float(loss[s, d]) - l) <= 2.0 ** -17 * max(1.0, abs(l))
                assert np.abs(dec.grad[s, d].double().cpu().numpy() - g).max() <= 2.0 ** -17
    assert n_acc > 5


def test_captured_step_follows_its_settings(models):
    _, tm, dm = models
    b, P, seed, K = 2, 24, 5, 8
    prompt = synth.uniform_ints(2203, "prompt", (b, P), 0, TS.vocab)
    dec = engine.SpecDecoder(tm, dm, b, 12, 512, prompt_len=P, temperature=0.9, seed=seed, top_k=K, teach=K)
    dec.prefill(torch.from_numpy(prompt).cuda())
    dec.step()
    dec.distill()
    g = dec.capture()
    for temps in ((0.9, 0.9), (0.0, 1.4), (2.0, 0.0)):
        dec.settings["temperature"].copy_(f32(temps))
        N0 = dec.cache_len.cpu().numpy()
        g.replay()
        torch.cuda.synchronize()
        check_draws(dec.choice.cpu().numpy(), dec.top["top_id"].cpu().numpy(), dec.top["top_val"].cpu().numpy(),
                    [(t, K, 1.0, 0.0) for t in temps], seed, N0[:, None] + dec.tree["depth"].cpu().numpy())
    assert dec.status() == 0


def test_path_rows():
    b, D, T, max_src = 4, 7, 30, 8
    n_new, N = [3, 1, 8, 0], [10, 0, 100, 7]
    src = np.full((b, max_src), -1, np.int32)
    src[0, :2] = [10 + 4, 10 + 9]
    src[2, :7] = 100 + np.array([1, 2, 29, 30, 31, -5, 0])    # the last four are no nodes behind the root
    out = torch.full((b, D), 99, dtype=torch.int32, device=DEV)
    _lib.path_rows(i32(n_new), torch.from_numpy(src).cuda(), i32([n + k for n, k in zip(N, n_new)]), T, out)
    assert out.tolist() == [[0, 4, 9, -1, -1, -1, -1], [T] + [-1] * 6, [2 * T, 2 * T + 1, 2 * T + 2, 2 * T + 29, -1, -1, -1], [-1] * 7]
