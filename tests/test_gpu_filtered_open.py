"""The target forward under settings that cut nothing: it says what the forward without settings says, so neither a mask of
settings nor lists for a drafter change a text.  And what a prompt pass records reaches SpecDecoder.status()."""
import math

import numpy as np
import pytest
import torch

import synth
from block_diffusion_draft_dflash_gb300 import _lib, engine
from test_gpu_filtered import DEV, DS, TS, f32, i32, models  # noqa: F401

pytestmark = pytest.mark.gpu


def caches(b, cap, Ns, seed):
    k, v = (torch.from_numpy(synth.normal(seed, n, (TS.n_layers, b, TS.n_kv_heads, cap, 128))).to(DEV, torch.bfloat16) for n in "kv")
    for s, n in enumerate(Ns):
        k[:, s, :, n:] = 0
        v[:, s, :, n:] = 0
    return k, v.transpose(-1, -2).contiguous()


def filtered(tm, tok, kv, clen, seed, K=0, **settings):
    b, T = tok.shape
    ws = _lib.Workspace(_lib.target_tree_forward_filtered_workspace_size(tm.cfg, b, T))
    choice = torch.full((b, T), -7, dtype=torch.int32, device=DEV)
    top = dict(top_id=torch.zeros(b, T, K, dtype=torch.int32, device=DEV), top_val=torch.zeros(b, T, K, device=DEV)) if K else {}
    _lib.target_tree_forward_filtered(tm.cfg, tm.weights, tok, None, None, *(t.clone() for t in kv), clen, choice, None, ws,
                                      seed=seed, **settings, **top)
    assert ws.status() == 0
    return choice.tolist()


def plain(tm, tok, kv, clen, seed, temperature):
    b, T = tok.shape
    ws = _lib.Workspace(_lib.target_tree_forward_workspace_size(tm.cfg, b, T))
    choice = torch.full((b, T), -7, dtype=torch.int32, device=DEV)
    _lib.target_tree_forward(tm.cfg, tm.weights, tok, None, None, *(t.clone() for t in kv), clen, choice, None, ws, temperature, seed)
    assert ws.status() == 0
    return choice.tolist()


@pytest.mark.parametrize("b,T", [(1, 1), (3, 17), (5, 300)])      # one block of logits and two
def test_settings_that_cut_nothing(models, b, T):  # noqa: F811
    _, tm, _ = models
    Ns, seed = [30, 7, 100, 0, 61][:b], 0x55AA
    kv, clen = caches(b, 512, Ns, b), i32(Ns)
    tok = i32(synth.uniform_ints(b, "tok", (b, T), 0, TS.vocab))
    want = {t: plain(tm, tok, kv, clen, seed, t) for t in (0.0, 0.7, 1.0, 2.0)}
    for t in (0.7, 1.0, 2.0):
        assert filtered(tm, tok, kv, clen, seed, temperature=f32([t] * b)) == want[t]
        assert filtered(tm, tok, kv, clen, seed, K=5, temperature=f32([t] * b), top_k=i32([0] * b), top_p=f32([1.0] * b),
                        min_p=f32([0.0] * b)) == want[t]
    assert filtered(tm, tok, kv, clen, seed, K=5) == want[1.0]
    # sequences of their own: some cut, some not, one greedy
    temps = [1.0, 0.0, 2.0, 0.7, 1.0][:b]
    mixed = filtered(tm, tok, kv, clen, seed, temperature=f32(temps), top_k=i32([0, 0, 0, 0, 1][:b]))
    for s in range(b):
        assert mixed[s] == (want[0.0] if s == 4 else want[temps[s]])[s]


def test_settings_that_cut_nothing_leave_bad_rows_out(models):  # noqa: F811
    """A sequence with a NaN among its rows' inputs is recorded; the others choose as they do alone."""
    _, tm, _ = models
    b, T, Ns = 2, 4, [20, 20]
    k, v = caches(b, 64, Ns, 9)
    v[:, 1, :, :, 3] = math.nan
    tok = i32(synth.uniform_ints(9, "tok", (b, T), 0, TS.vocab))
    want = plain(tm, tok[:1].contiguous(), (k[:, :1].contiguous(), v[:, :1].contiguous()), i32(Ns[:1]), 3, 1.0)
    ws = _lib.Workspace(_lib.target_tree_forward_filtered_workspace_size(tm.cfg, b, T))
    choice = torch.full((b, T), -7, dtype=torch.int32, device=DEV)
    _lib.target_tree_forward_filtered(tm.cfg, tm.weights, tok, None, None, k, v, i32(Ns), choice, None, ws, seed=3)
    assert ws.status() == -6 and choice[0].tolist() == want[0] and (choice[1] == -1).all()


@pytest.mark.parametrize("mode,B", [("tree", 24), ("chain", 0)])
@pytest.mark.parametrize("temperature", [0.0, 1.0])
def test_teaching_does_not_change_the_text(models, mode, B, temperature):  # noqa: F811
    _, tm, dm = models
    b, P = 2, 30
    prompt = torch.from_numpy(synth.uniform_ints(11, "prompt", (b, P), 0, TS.vocab)).cuda()
    texts = []
    for teach in (0, 16):
        dec = engine.SpecDecoder(tm, dm, b, B, 512, prompt_len=P, mode=mode, temperature=temperature, seed=77, teach=teach)
        dec.prefill(prompt)
        text = [dec.bonus.tolist()]
        for _ in range(6):
            dec.step()
            if teach:
                dec.distill()
            acc, n = dec.acc["acc_tok"], dec.acc["n_acc"]
            text.append([acc[s, :int(n[s]) + 1].tolist() for s in range(b)])
        assert dec.status() == 0
        texts.append(text)
    assert texts[0] == texts[1]


# ------------------------------------------------------------------------------ what a prompt pass records
def test_status_tells_of_the_prompt_pass(models):  # noqa: F811
    _, tm, dm = models
    b, P = 2, 20
    prompt = torch.from_numpy(synth.uniform_ints(12, "prompt", (b, P), 0, TS.vocab)).cuda()
    dec = engine.SpecDecoder(tm, dm, b, 12, 256, prompt_len=P, temperature=0.8, top_k=5, seed=1)
    assert dec.status() == 0
    dec.prefill(prompt)
    assert dec.status() == 0
    dec.settings["top_p"][1] = 2.0
    dec.prefill(prompt)
    assert dec.bonus[1] == -1 and dec.status() == -1
    dec.settings["top_p"][1] = 1.0
    dec.prefill(prompt)
    assert dec.status() == 0
    dec.ws_prefill.buf[:4].view(torch.int32).fill_(-6)       # each call's own error, in the order of the calls
    dec.ws_draft0.buf[:4].view(torch.int32).fill_(-1)
    assert dec.status() == -6


def test_status_without_a_prompt_pass(models):  # noqa: F811
    """Decoders without those workspaces, or whose owner has given them up, still answer."""
    _, tm, dm = models
    assert engine.SpecDecoder(tm, dm, 1, 12, 256).status() == 0
    dec = engine.SpecDecoder(tm, dm, 1, 12, 256, prompt_len=8)
    del dec.ws_prefill, dec.ws_draft0, dec.prompt_feat
    assert dec.status() == 0
