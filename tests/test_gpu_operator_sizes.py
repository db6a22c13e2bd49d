"""Sizes and scales that do not fit the C structures are refused as bad arguments."""

import pytest
import torch

import speculative_decoding_verify_bf16_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    sv.build_library()
    sv.load_library()


@pytest.mark.parametrize("max_len,scale", [(2 ** 31, None), (2 ** 40, None), (-2 ** 31 - 1, None), (8, "1"), (8, 1e39)])
def test_prefill(max_len, scale):
    x = torch.zeros(8, 2, 64, dtype=torch.bfloat16, device=DEV)
    off = torch.tensor([0, 8], dtype=torch.int32, device=DEV)
    for workspace in (None, torch.empty(64, dtype=torch.uint8, device=DEV)):
        with pytest.raises(ValueError):
            sv.spec_linear_prefill(x, x, x, torch.zeros(8, 2, device=DEV), off, None, x.clone(), None, max_len, scale=scale,
                                   workspace=workspace)


@pytest.mark.parametrize("scale", ["1", 1e39])
def test_verify(scale):
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device=DEV)
    off = torch.tensor([0, 2], dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        sv.spec_linear_verify(x, x, x, torch.zeros(2, 2, device=DEV), off, None, torch.empty(1, 2, 2, 64, 64, device=DEV),
                              x.clone(), scale=scale)


def test_logprobs():
    x = torch.zeros(2, 8, device=DEV)
    tok, lp = torch.zeros(2, dtype=torch.int32, device=DEV), torch.empty(2, device=DEV)
    with pytest.raises(ValueError):
        sv.spec_token_logprobs(x, tok, lp, rows=-2 ** 40)
    with pytest.raises(sv.SpecError):
        sv.spec_token_logprobs(x, tok, lp, rows=-1)
