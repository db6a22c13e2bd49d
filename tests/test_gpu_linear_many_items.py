"""GPU parity: many short lanes, so that each thread block takes item after item and its
tiles, whose rows past a lane are set to zero, are filled by copies again.

Bounds as for the chunked form elsewhere: two bf16 parts of scores and states (2^-15 of an
output's magnitude), its own rounding (2^-8 of its value), states within 2^-15."""

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


@pytest.mark.parametrize("lanes,hk,hv,state", [(300, 2, 4, True), (170, 4, 4, False), (64, 8, 16, True)])
def test_many_short_lanes(lanes, hk, hv, state):
    rng = np.random.default_rng(lanes)
    lens = rng.integers(1, 200, lanes)
    lens[rng.random(lanes) < 0.3] = 128  # whole tiles behind shorter ones
    ends = np.concatenate([[0], np.cumsum(lens)])
    n, d = int(ends[-1]), 32
    g = torch.Generator(device=DEV)
    g.manual_seed(lanes)
    q, k = (torch.nn.functional.normalize(torch.randn(n, hk, d, generator=g, device=DEV), dim=-1).to(torch.bfloat16)
            for _ in range(2))
    v = torch.randn(n, hv, d, generator=g, device=DEV).to(torch.bfloat16)
    decay = -0.2 * torch.rand(n, hv, generator=g, device=DEV)
    S = torch.randn(lanes, hv, d, d, generator=g, device=DEV) if state else None
    host = [None if t is None else t.double().cpu().numpy() for t in (q, k, v, decay, S)]
    want, wfinal, _, mag, fmag = linear_attention(*host[:4], ends, host[4], scale=d ** -0.5)
    offsets = torch.tensor(ends, dtype=torch.int32, device=DEV)
    first = None
    for _ in range(5):
        out, final = torch.full_like(v, 7.0), torch.full((lanes, hv, d, d), 7.0, device=DEV)
        status = torch.zeros(lanes, dtype=torch.int32, device=DEV)
        sv.spec_linear_prefill(q, k, v, decay, offsets, S, out, final, 199, lane_status=status)
        torch.cuda.synchronize()
        assert not status.any()
        assert (np.abs(out.double().cpu().numpy() - want) <= 2.0 ** -15 * mag + 2.0 ** -8 * np.abs(want)).all()
        assert (np.abs(final.double().cpu().numpy() - wfinal) <= 2.0 ** -15 * fmag).all()
        first = first or (out, final)
        assert torch.equal(out, first[0]) and torch.equal(final, first[1])
