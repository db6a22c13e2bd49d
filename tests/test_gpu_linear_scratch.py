"""A prefill takes scratch memory where it can use some: for bf16 prompts."""

import pytest
import torch

import speculative_decoding_verify_bf16_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype,taken", [(torch.bfloat16, 1), (torch.float32, 0)])
def test_scratch_memory_by_type(dtype, taken, monkeypatch):
    sv.build_library()
    calls = []
    make = sv.new_linear_workspace
    monkeypatch.setattr(sv, "new_linear_workspace", lambda *a: calls.append(a) or make(*a))
    n, h, d = 1100, 1, 64
    x = torch.zeros(n, h, d, dtype=dtype, device=DEV)
    out, final = torch.full_like(x, 7.0), torch.full((1, h, d, d), 7.0, device=DEV)
    sv.spec_linear_prefill(x, x, x, torch.zeros(n, h, device=DEV), torch.tensor([0, n], dtype=torch.int32, device=DEV), None,
                           out, final, n)
    assert len(calls) == taken and not out.any() and not final.any()
