"""What a prompt pass under settings records reaches SpecDecoder.status()."""
import pytest
import torch

import synth
from block_diffusion_draft_dflash_gb300 import engine
from test_gpu_filtered import TS, models  # noqa: F401

pytestmark = pytest.mark.gpu


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
