"""GPU: a prefill without a workspace takes its scratch memory on the stream that it runs on,
where the allocator orders it behind the memory's earlier uses."""

import numpy as np
import pytest
import torch

import speculative_decoding_verify_bf16_gb300 as sv
from oracle.linear import linear_attention

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    sv.build_library()
    sv.load_library()


@pytest.mark.parametrize("side", [True, False])
def test_scratch_memory_belongs_to_the_stream(side, monkeypatch):
    n, h, d = 3000, 2, 128  # few heads and a long lane: it is split
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    q, k, v = (torch.randn(n, h, d, generator=g, device=DEV).div(11).to(torch.bfloat16) for _ in range(3))
    decay = -0.05 * torch.rand(n, h, generator=g, device=DEV)
    want, wfinal, _, mag, fmag = linear_attention(*[t.double().cpu().numpy() for t in (q, k, v, decay)], [0, n], scale=d ** -0.5)
    offsets = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    out, final = torch.empty_like(v), torch.empty(1, h, d, d, device=DEV)
    size = sv.spec_linear_workspace(1, h, d, d, n)
    assert size > 0
    seen = []
    make = sv.new_linear_workspace
    monkeypatch.setattr(sv, "new_linear_workspace", lambda *a: seen.append(torch.cuda.current_stream()) or make(*a))
    stream = torch.cuda.Stream() if side else None
    torch.cuda.synchronize()
    # A block of that size that the current stream is still to write when it is given back.
    busy = torch.empty(size, dtype=torch.uint8, device=DEV)
    torch.cuda._sleep(20_000_000)
    busy.fill_(255)
    del busy
    sv.spec_linear_prefill(q, k, v, decay, offsets, None, out, final, n, stream=stream)
    torch.cuda.synchronize()
    assert seen == [stream or torch.cuda.current_stream()]
    # two bf16 parts of scores and states, fp32 products and sums, one rounding of an output
    assert (np.abs(out.double().cpu().numpy() - want) <= 2.0 ** -15 * mag + 2.0 ** -8 * np.abs(want)).all()
    assert (np.abs(final.double().cpu().numpy() - wfinal) <= 2.0 ** -15 * fmag).all()


def test_arguments_are_checked_before_scratch_memory_is_taken():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device=DEV)
    decay = torch.zeros(4, 2, device=DEV)
    with pytest.raises(ValueError):
        sv.spec_linear_prefill(x, x, x, decay, None, None, x.clone(), None, 4)
    with pytest.raises(ValueError):
        sv.spec_linear_prefill(x, x, x[0], decay, torch.tensor([0, 4], dtype=torch.int32, device=DEV), None, x.clone(), None, 4)
