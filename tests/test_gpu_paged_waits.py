"""The attention's bounded waits: a copy that never comes ends in a status, not in a hang.

The withheld copy (tile, in the kernel for many rows) is a switch of the kernels made for this; nothing faults, and the same
process goes on computing right results afterwards."""

import pytest
import torch

import speculative_decoding_verify_bf16_gb300 as sv
from paged_harness import Lanes, attend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    sv.build_library()
    sv.load_library()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 4, 300])
def test_attention_wait_gives_up(monkeypatch, kind, n):
    L = Lanes([n, n], [9000, 9000], kind=kind, kv=1, seed=1)
    q = L.queries(8)

    def run():
        out, lse, status = attend(L, q)
        torch.cuda.synchronize()
        return out, lse, status.tolist()

    good = run()
    assert good[2] == [0, 0]
    monkeypatch.setenv("SPEC_PAGED_TEST_WITHHOLD_COPY", "1")
    late = run()
    assert late[2] == [sv.SPEC_ERR_TIMEOUT, 0]
    assert torch.equal(late[0][n:], good[0][n:]) and torch.equal(late[1][n:], good[1][n:])
    monkeypatch.delenv("SPEC_PAGED_TEST_WITHHOLD_COPY")
    again = run()
    assert again[2] == [0, 0] and torch.equal(again[0], good[0]) and torch.equal(again[1], good[1])
