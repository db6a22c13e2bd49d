"""The log probabilities' bounded waits: a copy that never comes fails its row as a whole.

The withheld copy is a switch of the kernel made for this; nothing faults, and the same
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


@pytest.mark.parametrize("which,rows,V,top", [("2", 3, 40960, 5), ("2", 200, 8192, 20), ("1", 3, 40960, 5)])
@pytest.mark.parametrize("with_status", [True, False])
def test_a_row_whose_copy_does_not_come(monkeypatch, which, rows, V, top, with_status):
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    x = torch.randn(rows, V, generator=g, device=DEV).to(torch.bfloat16)
    tok = torch.arange(rows, dtype=torch.int32, device=DEV)
    want = token_logprobs(x.float().cpu().numpy(), tok.tolist(), None, top)

    def run():
        lp, ent = torch.full((rows,), 7.0, device=DEV), torch.full((rows,), 7.0, device=DEV)
        ids = torch.full((rows, top), 7, dtype=torch.int32, device=DEV)
        alt = torch.full((rows, top), 7.0, device=DEV)
        st = torch.full((rows,), 7, dtype=torch.int32, device=DEV) if with_status else None
        sv.spec_token_logprobs(x, tok, lp, entropy=ent, top_ids=ids, top_logprobs=alt, row_status=st)
        torch.cuda.synchronize()
        return [None if t is None else t.cpu().numpy() for t in (st, lp, ent, ids, alt)]

    def right(got, first):
        np.testing.assert_allclose(got[1][first:], want[1][first:], rtol=2.0 ** -22, atol=1e-5)
        np.testing.assert_allclose(got[2][first:], want[2][first:], rtol=2.0 ** -22, atol=2e-5)
        np.testing.assert_array_equal(got[3][first:], want[3][first:])
        np.testing.assert_allclose(got[4][first:], want[4][first:], rtol=2.0 ** -22, atol=1e-5)
        assert got[0] is None or not got[0][first:].any()

    monkeypatch.setenv("SPEC_LOGPROBS_TEST_WITHHOLD_COPY", which)
    late = run()
    monkeypatch.delenv("SPEC_LOGPROBS_TEST_WITHHOLD_COPY")
    assert np.isnan(late[1][0]) and np.isnan(late[2][0]) and np.isnan(late[4][0]).all() and (late[3][0] == -1).all()
    assert late[0] is None or late[0][0] == sv.SPEC_ERR_TIMEOUT
    right(late, 1)
    right(run(), 0)
