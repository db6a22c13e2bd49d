"""GPU parity: rows whose alternatives lie among more blocks than a warp's ring holds, so that
they come in several batches, the row's partial block (filled element by element) among them.

Ids are exact; tolerances as for the log probabilities elsewhere (1e-5, and four roundings
of a number's own size)."""

import numpy as np
import pytest
import torch

import speculative_decoding_verify_bf16_gb300 as sv
from oracle.logprobs import token_logprobs

pytestmark = pytest.mark.gpu
DEV = "cuda"
BLOCK = 512


@pytest.fixture(scope="module", autouse=True)
def _built():
    sv.build_library()
    sv.load_library()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("blocks,tail", [(2343, 100), (2343, 511), (3000, 0), (1400, 9)])
def test_best_blocks_in_one_column(dtype, blocks, tail):
    """Every 32nd block holds a high token: far more than 20 blocks are as good as the bound
    that the other blocks' maxima give."""
    V = blocks * BLOCK + tail
    g = torch.Generator(device=DEV)
    g.manual_seed(blocks + tail)
    x = torch.randn(2, V, generator=g, device=DEV).clamp_(-3, 3)
    last = (V - 1) // BLOCK  # the partial block's column
    for b in range(last % 32, last + 1, 32):
        x[:, b * BLOCK + 3] = 8.0
        x[1, b * BLOCK + 5] = 9.0
    x = x.to(dtype)
    tok = torch.tensor([last * BLOCK + 3, 5], dtype=torch.int32, device=DEV)
    want = token_logprobs(x.float().cpu().numpy(), tok.tolist(), None, 20)
    for _ in range(3):
        lp, ent = torch.empty(2, device=DEV), torch.empty(2, device=DEV)
        ids = torch.empty(2, 20, dtype=torch.int32, device=DEV)
        alt = torch.empty(2, 20, device=DEV)
        st = torch.full((2,), 9, dtype=torch.int32, device=DEV)
        sv.spec_token_logprobs(x, tok, lp, entropy=ent, top_ids=ids, top_logprobs=alt, row_status=st)
        torch.cuda.synchronize()
        assert st.tolist() == [0, 0]
        np.testing.assert_array_equal(ids.cpu().numpy(), want[3])
        np.testing.assert_allclose(alt.cpu().numpy(), want[4], rtol=2.0 ** -22, atol=1e-5)
        np.testing.assert_allclose(lp.cpu().numpy(), want[1], rtol=2.0 ** -22, atol=1e-5)
