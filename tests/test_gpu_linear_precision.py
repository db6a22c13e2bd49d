"""GPU parity: the chunked prefill's outputs carry one bf16 rounding, their own.

Scores and states enter the outputs' products in two bf16 parts: the upper by truncation
(what is left is below 2^-7 of the number), the lower rounded (2^-9 of that), so each term
is within 2^-16, and a factor of two covers that a term has a score or a state and that
their products add up in fp32 with truncation (some 40 additions of 2^-23).  An output is
then within 2^-15 of its magnitude A (every term by its absolute value), and 2^-8 of its
value for its own rounding.  Errors of 2^-15 added to a rounding of 2^-9 (rms, relative)
raise its root mean square by far less than a hundredth."""

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


@pytest.mark.parametrize("lens,hk,hv,dk,dv", [([128], 2, 2, 128, 128), ([384, 128], 2, 4, 128, 128), ([1024], 1, 2, 128, 128),
                                              ([640] * 3, 2, 2, 64, 96), ([2048, 1280], 1, 1, 128, 128)])
@pytest.mark.parametrize("state", [True, False])
def test_outputs_are_rounded_once(lens, hk, hv, dk, dv, state):
    g = torch.Generator(device=DEV)
    g.manual_seed(sum(lens) + dk)
    n, lanes = sum(lens), len(lens)
    q, k = (torch.nn.functional.normalize(torch.randn(n, hk, dk, generator=g, device=DEV), dim=-1).to(torch.bfloat16)
            for _ in range(2))
    v = torch.randn(n, hv, dv, generator=g, device=DEV).to(torch.bfloat16)
    decay = -torch.logspace(-3, 0, hv, device=DEV) * torch.rand(n, hv, generator=g, device=DEV)
    S = torch.randn(lanes, hv, dk, dv, generator=g, device=DEV) if state else None
    ends = np.cumsum([0] + lens)
    out, final = torch.empty_like(v), torch.empty(lanes, hv, dk, dv, device=DEV)
    status = torch.zeros(lanes, dtype=torch.int32, device=DEV)
    sv.spec_linear_prefill(q, k, v, decay, torch.tensor(ends, dtype=torch.int32, device=DEV), S, out, final, max(lens),
                           lane_status=status)
    torch.cuda.synchronize()
    assert status.tolist() == [0] * lanes
    host = [None if t is None else t.double().cpu().numpy() for t in (q, k, v, decay)]
    want, _, _, mag, _ = linear_attention(*host, ends, None if S is None else S.double().cpu().numpy(), scale=dk ** -0.5)
    err = out.double().cpu().numpy() - want
    assert (np.abs(err) <= 2.0 ** -15 * mag + 2.0 ** -8 * np.abs(want)).all()
    own = torch.from_numpy(want).to(torch.bfloat16).double().numpy() - want
    rms = lambda x: np.sqrt(np.mean(x * x))
    assert rms(err) <= 1.01 * rms(own), (rms(err) / rms(want), rms(own) / rms(want))
