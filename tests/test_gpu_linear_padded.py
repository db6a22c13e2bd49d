"""GPU: a prefill writes the columns of its outputs and nothing beside them.

Outputs (and q, k, v) are views of buffers with wider heads or rows; what lies between the
views keeps its bits, for whole chunks and for the shorter ones at a lane's end."""

import numpy as np
import pytest
import torch

import speculative_decoding_verify_bf16_gb300 as sv
from oracle.linear import linear_attention

pytestmark = pytest.mark.gpu
DEV = "cuda"
MARK = 11.0


@pytest.fixture(scope="module", autouse=True)
def _built():
    sv.build_library()
    sv.load_library()


def wide(x, size):
    """x as a view of a buffer whose heads are `size` wide, and that buffer."""
    buf = torch.full((x.shape[0], x.shape[1], size), MARK, dtype=x.dtype, device=DEV)
    buf[:, :, :x.shape[2]] = x
    return buf[:, :, :x.shape[2]], buf


@pytest.mark.parametrize("dv,size", [(4, 8), (12, 16), (20, 24), (28, 40), (60, 64), (100, 104), (124, 128), (16, 24), (128, 136)])
@pytest.mark.parametrize("lens", [[40], [130, 9, 0, 256], [128, 1, 77]])
@pytest.mark.parametrize("heads", [1, 2])
def test_columns_beside_the_outputs_stay(dv, size, lens, heads):
    g = torch.Generator(device=DEV)
    g.manual_seed(dv + sum(lens))
    n, dk, lanes = sum(lens), 64, len(lens)
    q, k = (torch.nn.functional.normalize(torch.randn(n, heads, dk, generator=g, device=DEV), dim=-1).to(torch.bfloat16)
            for _ in range(2))
    v, _ = wide(torch.randn(n, heads, dv, generator=g, device=DEV).to(torch.bfloat16), size)
    out, buf = wide(torch.full((n, heads, dv), MARK, dtype=torch.bfloat16, device=DEV), size)
    decay = -torch.rand(n, heads, generator=g, device=DEV)
    ends = np.cumsum([0] + lens)
    final = torch.empty(lanes, heads, dk, dv, device=DEV)
    status = torch.zeros(lanes, dtype=torch.int32, device=DEV)
    sv.spec_linear_prefill(q, k, v, decay, torch.tensor(ends, dtype=torch.int32, device=DEV), None, out, final, max(lens),
                           lane_status=status)
    torch.cuda.synchronize()
    assert status.tolist() == [0] * lanes
    assert (buf[:, :, dv:] == MARK).all()
    host = [t.double().cpu().numpy() for t in (q, k, v, decay)]
    want, wfinal, _, mag, fmag = linear_attention(*host, ends, scale=dk ** -0.5)
    # two bf16 parts of scores and states, products and sums in fp32, one rounding of an output
    assert (np.abs(out.double().cpu().numpy() - want) <= 2.0 ** -15 * mag + 2.0 ** -8 * np.abs(want)).all()
    assert (np.abs(final.double().cpu().numpy() - wfinal) <= 2.0 ** -15 * fmag).all()
