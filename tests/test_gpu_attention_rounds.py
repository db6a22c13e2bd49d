"""The attention example: the cache's calls together, as rounds use them, give what plain
decoding gives."""

import importlib.util
import os

import numpy as np
import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("attention_rounds", os.path.join(ROOT, "examples", "attention_rounds.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.sv.build_library()
    return mod


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "int8"])
def test_rounds_equal_plain_decoding(example, cache):
    model = example.AttentionModel(seed=3)
    rng = np.random.default_rng(2)
    prompts = [rng.integers(0, model.vocab, n).tolist() for n in (2, 33, 140, 300)]
    new, rounds = example.speculate(model, prompts, 40, cache=cache)
    plain = example.decode(model, prompts, max(len(n) for n in new), cache)
    for b, n in enumerate(new):
        assert len(n) >= 40 and n == plain[b][:len(n)], b
    assert rounds < 40  # some drafts were kept


@pytest.mark.parametrize("cache", ["bf16", "int8"])
def test_a_prompt_in_parts_equals_the_whole(example, cache):
    """Logits of a prompt's last token, the prompt taken whole or in parts of many sizes: both are a
    model's values up to the outputs' roundings (2^-8 of a value each, twice a layer, through weights of norm
    about 1), far below the 12 between the likeliest token and others."""
    model = example.AttentionModel(seed=5)
    prompt = np.random.default_rng(1).integers(0, model.vocab, 333).tolist()
    whole = example.Lanes(model, 1, 400, cache)
    want = whole.run([prompt])[0][-1]
    lanes, at = example.Lanes(model, 1, 400, cache), 0
    for n in (1, 2, 100, 13, 1, 64, 150, 2):
        got, _, status = lanes.run([prompt[at:at + n]])
        assert status.tolist() == [0]
        lanes.keep(torch.tensor([n], dtype=torch.int32, device="cuda"))
        at += n
    assert at == len(prompt) and torch.equal(lanes.cached, torch.tensor([333], dtype=torch.int32, device="cuda"))
    assert (got[-1] - want).norm() <= 2.0 ** -5 * want.norm()
