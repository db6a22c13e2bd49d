"""The recurrent example: speculative rounds give what plain decoding gives."""

import importlib.util
import os

import numpy as np
import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("recurrent_rounds", os.path.join(ROOT, "examples", "recurrent_rounds.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.sv.build_library()
    return mod


def test_rounds_equal_plain_decoding(example):
    model = example.RecurrentModel(seed=3)
    rng = np.random.default_rng(2)
    prompts = [rng.integers(0, model.vocab, n).tolist() for n in (2, 33, 140, 300)]
    new, logps, alternatives, rounds = example.speculate(model, prompts, 40)
    plain = example.decode(model, prompts, max(len(n) for n in new))
    for b, n in enumerate(new):
        assert n == plain[b][:len(n)], b
        assert len(logps[b]) == len(n) and all(lp <= 0 for lp in logps[b])
    assert rounds < 40  # some drafts were kept
    # greedy: the first alternative is the committed token's, and the alternatives descend
    lps = [lp for _, lp in alternatives]
    assert lps == sorted(lps, reverse=True)


def test_states_after_rounds_equal_a_prefill_of_the_same_tokens(example):
    model = example.RecurrentModel(seed=4)
    prompts = [list(range(50, 90)), list(range(7, 60))]
    whole = example.prefill(model, prompts)
    live = example.prefill(model, [p[:20] for p in prompts])
    off = torch.arange(3, dtype=torch.int32, device=model.device)

    def attend(layer, q, k, v, decay):
        out = torch.empty_like(v)
        example.sv.spec_linear_verify(q, k, v, decay, off, live[:, layer], live[:, layer].unsqueeze(1), out)
        return out

    for t in range(19, 39):
        model.forward(torch.tensor([p[t] for p in prompts], dtype=torch.int32, device=model.device), attend)
    # (the lanes' lengths differ: the first is at its end)
    torch.testing.assert_close(live[0, 0], whole[0, 0], rtol=1e-3, atol=1e-4)
