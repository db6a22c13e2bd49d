"""GPU parity: what a reset takes stays away, however the state grows after it; decays that
large growth follows count in full.

Bounds as for the chunked form elsewhere, against the 64-bit recurrence: 2^-15 of a state's
magnitude (every term by its absolute value, which a reset clears too), and for an output
that of its magnitude and its own rounding, 2^-8 of its value.  Sums of log decays hold
32 fractional bits of a base-2 logarithm, and each of at most 128 decays is read in fp32 with
an error of 2^-24 of itself in the product with log2(e); the strongest finite case is checked to 2^-9."""

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


def run(n, decay, key_scale, seed=1):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    h, d = 2, 128
    q, k, v = (torch.randn(n, h, d, generator=g, device=DEV).div(11).to(torch.bfloat16) for _ in range(3))
    k = k * key_scale[:, None, None].to(torch.bfloat16)
    S = torch.randn(1, h, d, d, generator=g, device=DEV)
    decay = decay[:, None].expand(n, h)
    out, final = torch.empty_like(v), torch.empty_like(S)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    sv.spec_linear_prefill(q, k, v, decay, torch.tensor([0, n], dtype=torch.int32, device=DEV), S, out, final, n,
                           lane_status=status)
    torch.cuda.synchronize()
    assert status.tolist() == [0]
    host = [t.double().cpu().numpy() for t in (q, k, v, decay, S)]
    want, wfinal, _, mag, fmag = linear_attention(*host[:4], [0, n], host[4], scale=d ** -0.5)
    return out.double().cpu().numpy(), final.double().cpu().numpy(), want, wfinal, mag, fmag


@pytest.mark.parametrize("n", [40, 128, 300])
@pytest.mark.parametrize("reset", [float("-inf"), -3.4e38, -1e5])
@pytest.mark.parametrize("at", [3, 17, 30])
def test_growth_does_not_bring_back_what_a_reset_took(n, reset, at):
    """No keys from the reset on: everything after it is exactly 0, also behind growth of e^80
    (2^115; a factor of 2^128 or more is infinite in fp32 and fails the lane)."""
    decay = torch.full((n,), -0.01, device=DEV)
    decay[at] = reset
    decay[at + 1:at + 9] = 10.0
    keys = (torch.arange(n, device=DEV) < at).float()
    out, final, want, wfinal, mag, _ = run(n, decay, keys)
    assert not wfinal.any() and not final.any()
    assert not want[at:].any() and not out[at:].any()
    assert (np.abs(out - want)[:at] <= 2.0 ** -15 * mag[:at] + 2.0 ** -8 * np.abs(want)[:at]).all()


@pytest.mark.parametrize("n", [40, 128, 300])
def test_reset_between_documents_with_growth(n):
    decay = torch.full((n,), 0.02, device=DEV)
    decay[[5, 20, n - 3]] = float("-inf")
    out, final, want, wfinal, mag, fmag = run(n, decay, torch.ones(n, device=DEV), seed=2)
    assert (np.abs(final - wfinal) <= 2.0 ** -15 * fmag).all()
    assert (np.abs(out - want) <= 2.0 ** -15 * mag + 2.0 ** -8 * np.abs(want)).all()


@pytest.mark.parametrize("n", [40, 128])
def test_strong_finite_decays_count_in_full(n):
    """e^-115 behind which e^80 follows: what was there before is there to e^-35."""
    decay = torch.zeros(n, device=DEV)
    decay[10] = -115.0
    decay[12:16] = 20.0
    out, final, want, wfinal, mag, fmag = run(n, decay, (torch.arange(n, device=DEV) < 10).float(), seed=3)
    assert (np.abs(final - wfinal) <= 2.0 ** -9 * fmag).all()
    seen = mag > 1e-30  # (between the two the numbers are below fp32's)
    assert (np.abs(out - want) <= 2.0 ** -9 * mag + 2.0 ** -8 * np.abs(want))[seen].all()
