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


def test_decoding_continues_a_prefill(example):
    """A prompt's state, and the state after its first tokens' prefill and single steps over
    the rest, on the same activations: within 2^-15 (bf16 prefill) and 5 * steps * 2^-24 of
    the state's magnitude, twice over."""
    sv, n, cut = example.sv, 60, 37
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    q, k, v = (torch.randn(n, 2, 128, generator=g, device="cuda").div(11).to(torch.bfloat16) for _ in range(3))
    decay = torch.tensor([-0.01, -0.3], device="cuda").expand(n, 2)

    def offsets(*lens):
        return torch.tensor(np.cumsum((0, *lens)), dtype=torch.int32, device="cuda")

    whole, live = (torch.empty(1, 2, 128, 128, device="cuda") for _ in range(2))
    out, part = torch.empty_like(v), torch.empty_like(v)
    sv.spec_linear_prefill(q, k, v, decay, offsets(n), None, out, whole, n)
    sv.spec_linear_prefill(q[:cut], k[:cut], v[:cut], decay[:cut], offsets(cut), None, part[:cut], live, cut)
    for t in range(cut, n):
        r = slice(t, t + 1)
        sv.spec_linear_verify(q[r], k[r], v[r], decay[r], offsets(1), live, live.unsqueeze(1), part[r])
    mag = torch.zeros(2, 128, 128, dtype=torch.float64, device="cuda")
    for t in range(n):
        mag = mag * decay[t].double().exp()[:, None, None] + (k[t].double()[:, :, None] * v[t].double()[:, None, :]).abs()
    bound = 2 * (2.0 ** -15 + 5 * n * 2.0 ** -24) * mag
    assert ((live[0].double() - whole[0].double()).abs() <= bound).all()
