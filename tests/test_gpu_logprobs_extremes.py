"""GPU parity: log probabilities where logits over temperature are huge numbers: tiny
temperatures, large logits, large negative fills in masked places.

Tolerances: a weight's exponent (x - m) log2(e) / T is a difference that fp32 holds to 2^-24 of
itself, times a factor held to 2^-23, so weights that count (exponents above -24) are within
2^-18 of themselves; sums add 2^-20, so a log probability is within 1e-5 and four roundings of
its own size, and an entropy, the difference of two such numbers, within 2e-5."""

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


def check(x, tokens, temps, top=5):
    rows = x.shape[0]
    tok = torch.as_tensor(tokens, dtype=torch.int32, device=DEV)
    t = None if temps is None else torch.as_tensor(temps, dtype=torch.float32, device=DEV)
    lp, ent = (torch.full((rows,), 77.0, device=DEV) for _ in range(2))
    ids = torch.full((rows, top), 77, dtype=torch.int32, device=DEV)
    alt = torch.full((rows, top), 77.0, device=DEV)
    st = torch.full((rows,), 77, dtype=torch.int32, device=DEV)
    sv.spec_token_logprobs(x, tok, lp, entropy=ent, top_ids=ids, top_logprobs=alt, temperatures=t, row_status=st)
    torch.cuda.synchronize()
    want = token_logprobs(x.float().cpu().numpy(), tok.cpu().numpy(), None if t is None else t.cpu().numpy(), top)
    assert not want[0].any() and st.tolist() == [0] * rows
    np.testing.assert_allclose(lp.cpu().numpy(), want[1], rtol=2.0 ** -22, atol=1e-5)
    np.testing.assert_allclose(ent.cpu().numpy(), want[2], rtol=2.0 ** -22, atol=2e-5)
    np.testing.assert_array_equal(ids.cpu().numpy(), want[3])
    np.testing.assert_allclose(alt.cpu().numpy(), want[4], rtol=2.0 ** -22, atol=1e-5)


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [1e-4, 1e-6, 1e-7, 1e-8, 1e-9, 2e-9, 1e-10, 1e-15, 1e-20, 1e-30])
def test_tiny_temperatures(T, dtype):
    rows, V, g = 200, 9000, gen(3)
    x = torch.randn(rows, V, generator=g, device=DEV) * 2
    x[torch.arange(rows), torch.randint(0, V, (rows,), generator=g, device=DEV)] += 8
    x = x.to(dtype)
    best = x.float().argmax(1)
    other = torch.randint(0, V, (rows,), generator=g, device=DEV)
    tok = torch.where(torch.arange(rows, device=DEV) % 4 == 0, other, best)
    temps = T * (1 + torch.rand(rows, generator=g, device=DEV))
    check(x, tok, temps)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size", [1e6, 1e7, 1e8, 1e9, 3e9, 1e10, 1e12, 1e20, 1e30])
def test_large_logits(size, dtype):
    rows, V, g = 60, 9000, gen(4)
    x = (torch.randn(rows, V, generator=g, device=DEV) * size).to(dtype)
    tok = x.float().argmax(1)
    tok[::5] = 17
    check(x, tok, None)
    check(x, tok, 0.3 + torch.rand(rows, generator=g, device=DEV))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fill", [-1e4, -1e6, -1e9, -2e9, -1e10, -1e12, -1e20, -1e30, -3e38])
@pytest.mark.parametrize("first", [True, False])
def test_large_fills_in_masked_places(fill, dtype, first):
    """Most of a row at one large negative number, in long runs, the live tokens behind them or
    before; many temperatures."""
    rows, V, g = 120, 60000, gen(5)
    x = torch.randn(rows, V, generator=g, device=DEV) * 3
    live = torch.randint(100, 9000, (rows,), generator=g, device=DEV)
    at = torch.arange(V, device=DEV)
    keep = at >= V - live[:, None] if first else at < live[:, None]
    keep[7::10] &= at % 97 == 0
    x = torch.where(keep, x, torch.tensor(fill, device=DEV)).to(dtype)
    tok = x.float().argmax(1)
    tok[3::10] = 0 if not first else V - 1
    temps = torch.where(torch.arange(rows, device=DEV) % 6 == 0, 0.0, 0.05 + 1.2 * torch.rand(rows, generator=g, device=DEV))
    check(x, tok, temps)


@pytest.mark.parametrize("middle", [2.0 ** 22, -2.0 ** 22, 2.0 ** 31, -2.0 ** 31])
@pytest.mark.parametrize("down", [True, False])
def test_running_maximum_across_the_forms_border(middle, down):
    """fp32 logits whose running maximum, in units of log 2, passes a border slowly, with
    weights on both sides that count."""
    V, g = 40000, gen(6)
    m = middle / 1.4426950408889634
    step = float(np.spacing(np.float32(abs(m))))
    ramp = torch.linspace(-60, 60, V, device=DEV, dtype=torch.float64)
    rows = []
    for i in range(16):
        noise = torch.rand(V, generator=g, device=DEV, dtype=torch.float64) * 3
        rows.append(m + step * torch.round((ramp * (1 + i / 8) + noise) * max(1.0, 0.1 / step)))
    x = torch.stack(rows)
    x = (x.flip(1) if down else x).to(torch.float32)
    tok = x.argmax(1)
    tok[::4] = V // 2
    check(x, tok, None)
    # and with the ramp at a few tens, however coarse the numbers are
    spread = (x.max(1).values - x.min(1).values) / 40
    check(x, tok, torch.where(spread > 1, spread, torch.ones_like(spread)))
