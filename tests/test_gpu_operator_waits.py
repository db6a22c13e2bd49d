"""The operators' bounded waits: a copy that never comes ends in a status, not in a hang.

The withheld copy is a switch of the kernels made for this; nothing faults, and the same
process goes on computing right results afterwards."""

import numpy as np
import pytest
import torch

import speculative_decoding_verify_bf16_gb300 as sv
from oracle.logprobs import token_logprobs

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    sv.build_library()
    sv.load_library()


def test_logprobs_wait_gives_up(monkeypatch):
    x = torch.randn(3, 40000, device=DEV)
    tok = torch.tensor([5, 6, 7], dtype=torch.int32, device=DEV)
    lp, status = torch.empty(3, device=DEV), torch.empty(3, dtype=torch.int32, device=DEV)
    monkeypatch.setenv("SPEC_LOGPROBS_TEST_WITHHOLD_COPY", "1")
    sv.spec_token_logprobs(x, tok, lp, row_status=status)
    torch.cuda.synchronize()
    want = token_logprobs(x.cpu().numpy(), [5, 6, 7])[1]
    assert status.tolist() == [sv.SPEC_ERR_TIMEOUT, 0, 0]
    assert torch.isnan(lp[0]) and np.allclose(lp[1:].cpu().numpy(), want[1:], atol=1e-5)
    monkeypatch.delenv("SPEC_LOGPROBS_TEST_WITHHOLD_COPY")
    sv.spec_token_logprobs(x, tok, lp, row_status=status)
    torch.cuda.synchronize()
    assert status.tolist() == [0, 0, 0] and np.allclose(lp.cpu().numpy(), want, atol=1e-5)


def test_prefill_wait_gives_up(monkeypatch):
    n, h = 200, 2
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    q, k, v = (torch.randn(2 * n, h, 128, generator=g, device=DEV).div(11).to(torch.bfloat16) for _ in range(3))
    decay = torch.full((2 * n, h), -0.1, device=DEV)
    off = torch.tensor([0, n, 2 * n], dtype=torch.int32, device=DEV)

    def run():
        out, state = torch.empty_like(v), torch.empty(2, h, 128, 128, device=DEV)
        status = torch.zeros(2, dtype=torch.int32, device=DEV)
        sv.spec_linear_prefill(q, k, v, decay, off, None, out, state, n, lane_status=status)
        torch.cuda.synchronize()
        return out, state, status.tolist()

    good = run()
    assert good[2] == [0, 0]
    monkeypatch.setenv("SPEC_LINEAR_TEST_WITHHOLD_COPY", "1")
    late = run()
    assert late[2] == [sv.SPEC_ERR_TIMEOUT, 0]
    assert torch.equal(late[0][n:], good[0][n:]) and torch.equal(late[1][1], good[1][1])
    monkeypatch.delenv("SPEC_LINEAR_TEST_WITHHOLD_COPY")
    again = run()
    assert again[2] == [0, 0] and torch.equal(again[0], good[0]) and torch.equal(again[1], good[1])
