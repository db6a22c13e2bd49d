"""An infinite temperature: every token that is not masked is as likely as any other."""

import numpy as np
import pytest
import torch

import speculative_decoding_verify_bf16_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [float("inf"), 1e38])
def test_uniform_over_what_is_not_masked(dtype, T):
    sv.build_library()
    V, top = 5000, 20
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    x = torch.randn(3, V, generator=g, device=DEV)
    x[1, 1000:] = float("-inf")
    x[2, 7:] = float("-inf")
    x = x.to(dtype)
    tok = torch.tensor([3, 4000, 2], dtype=torch.int32, device=DEV)
    lp, ent = torch.empty(3, device=DEV), torch.empty(3, device=DEV)
    ids, alt = torch.empty(3, top, dtype=torch.int32, device=DEV), torch.empty(3, top, device=DEV)
    st = torch.full((3,), 9, dtype=torch.int32, device=DEV)
    sv.spec_token_logprobs(x, tok, lp, entropy=ent, top_ids=ids, top_logprobs=alt, row_status=st,
                           temperatures=torch.full((3,), T, device=DEV))
    torch.cuda.synchronize()
    assert st.tolist() == [0, 0, 0]
    n = np.array([V, 1000, 7])
    np.testing.assert_allclose(ent.cpu().numpy(), np.log(n), rtol=1e-6)
    np.testing.assert_allclose(lp.cpu().numpy(), [-np.log(V), -np.inf, -np.log(7)], rtol=1e-6)
    order = np.argsort(-x.float().cpu().numpy(), axis=1, kind="stable")[:, :top]
    np.testing.assert_array_equal(ids.cpu().numpy(), order)
    want = np.where(np.arange(top) < n[:, None], -np.log(n)[:, None], -np.inf)
    np.testing.assert_allclose(alt.cpu().numpy(), want, rtol=1e-6)
