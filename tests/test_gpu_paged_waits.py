"""The tile kernel's bounded waits: a tile that is never handed on ends in a status, not in a hang.

The withheld tile is a switch of the kernel made for this; nothing faults, and the same
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
def test_attention_wait_gives_up(monkeypatch, kind):
    L = Lanes([300, 300], [9000, 9000], kind=kind, kv=1, seed=1)
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
    assert torch.equal(late[0][300:], good[0][300:]) and torch.equal(late[1][300:], good[1][300:])
    monkeypatch.delenv("SPEC_PAGED_TEST_WITHHOLD_COPY")
    again = run()
    assert again[2] == [0, 0] and torch.equal(again[0], good[0]) and torch.equal(again[1], good[1])
