"""GPU parity: log probabilities of given tokens against the float64 oracle.

Tolerances: a weight e^(z - m) carries the roundings of x - m, of the product with
log2(e) / T and of the exponential (2 ulp), about |z - m| * 2^-22 relative, and fp32
sums of up to a few thousand terms a thread; 1e-5 in log space covers both, as for the
verify round's log probabilities.  A reported log probability also carries the
rounding of its own magnitude, up to 4 roundings of 2^-24 of it.  The entropy is a
difference of two such numbers: 2e-5.  Ids are exact."""

import numpy as np
import pytest
import torch

import speculative_decoding_verify_bf16_gb300 as sv
from oracle.logprobs import token_logprobs

pytestmark = pytest.mark.gpu
DEV = "cuda"
ATOL, RTOL, ENT_ATOL = 1e-5, 2.0 ** -22, 2e-5


@pytest.fixture(scope="module", autouse=True)
def _built():
    sv.build_library()
    sv.load_library()


def check(logits, tokens, temps=None, top=5, stream=None):
    rows = logits.shape[0]
    dev = logits.device
    tok = torch.as_tensor(tokens, dtype=torch.int32, device=dev)
    tt = None if temps is None else torch.as_tensor(temps, dtype=torch.float32, device=dev)
    lp, ent = (torch.full((rows,), 77.0, device=dev) for _ in range(2))
    ids = torch.full((rows, top), 77, dtype=torch.int32, device=dev)
    alt = torch.full((rows, top), 77.0, device=dev)
    st = torch.full((rows,), 77, dtype=torch.int32, device=dev)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    sv.spec_token_logprobs(logits, tok, lp, entropy=ent, top_ids=ids if top else None,
                           top_logprobs=alt if top else None, temperatures=tt, row_status=st, stream=stream)
    torch.cuda.synchronize()
    x = logits.float().cpu().numpy()
    want = token_logprobs(x, tok.cpu().numpy(), None if tt is None else tt.cpu().numpy(), top)
    np.testing.assert_array_equal(st.cpu().numpy(), want[0])
    np.testing.assert_allclose(lp.cpu().numpy(), want[1], rtol=RTOL, atol=ATOL)
    np.testing.assert_allclose(ent.cpu().numpy(), want[2], rtol=RTOL, atol=ENT_ATOL)
    np.testing.assert_array_equal(ids.cpu().numpy(), want[3])
    np.testing.assert_allclose(alt.cpu().numpy(), want[4], rtol=RTOL, atol=ATOL)
    return want


def rand(rows, V, dtype, seed, pad=0, shift=0, sigma=2.0):
    """[rows, V] logits in a wider buffer; `shift` moves the base off its alignment,
    the padding around the rows holds +inf that must not be read."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    buf = torch.full((rows * (V + pad) + shift,), float("inf"), device=DEV, dtype=dtype)
    x = buf[shift:].view(rows, V + pad)[:, :V]
    x.copy_((torch.randn(rows, V, generator=g, device=DEV) * sigma).to(dtype))
    return x


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1, 2, 7, 19, 20, 31, 511, 512, 513, 1024, 4099, 16384, 50001, 151936])
def test_sizes(V, dtype):
    rows = 5
    x = rand(rows, V, dtype, V)
    rng = np.random.default_rng(V)
    check(x, rng.integers(0, V, rows), [0.0, 0.7, 1.0, 0.3, -1.0], top=min(20, 3 + V % 18))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,V", [(1, 10104), (5, 50000), (1, 50000), (5, 50008), (2, 99992), (9, 57496), (3, 262136)])
def test_clusters_whose_last_blocks_have_nothing(rows, V, dtype):
    """Aligned rows that end inside a block, over more thread blocks than divide them evenly:
    the last ones have no part, and the partial block counts once."""
    x = rand(rows, V, dtype, V)
    check(x, np.random.default_rng(V).integers(0, V, rows), [(0.0, 0.7)[i % 2] for i in range(rows)], top=20)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad,shift", [(1, 0), (3, 1), (8, 0), (8, 3), (5, 7)])
def test_strides_and_alignment(dtype, pad, shift):
    x = rand(4, 3001, dtype, 11, pad, shift)
    check(x, [0, 3000, 17, 1234], top=20)


@pytest.mark.parametrize("rows,V", [(1, 262144), (3, 100003), (40, 20000), (160, 9000), (700, 3000)])
def test_row_counts(rows, V):
    x = rand(rows, V, torch.bfloat16, rows)
    rng = np.random.default_rng(rows)
    tok = rng.integers(0, V, rows)
    tok[rng.random(rows) < 0.3] = -1
    check(x, tok, rng.uniform(-0.5, 1.5, rows), top=7)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_masks_and_extreme_values(dtype):
    V, low = 6000, torch.finfo(dtype).min
    x = rand(9, V, dtype, 5)
    x[0, :5990] = float("-inf")       # ten tokens left
    x[1, 1:] = float("-inf")          # one token left
    x[2, :] = low                     # every token at the lowest value: uniform
    x[3, 100:] = low
    x[4, :512] = float("-inf")        # a whole block masked, the first
    x[5, 300:] = float("-inf")
    x[5, :300] = 0.0
    x[6, :] = 0.0
    x[6, ::2] = -0.0                  # -0 counts as +0
    x[7, :] = torch.linspace(-30, 30, V, device=DEV).to(dtype)
    x[8, :] = torch.linspace(30, -30, V, device=DEV).to(dtype)
    check(x, [5995, 0, 17, 5, 3000, 2, 5999, 5999, 0], top=20)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [3000, 90000])
def test_many_equal_logits(dtype, V):
    """Ties go to the lowest id, however many there are."""
    x = torch.round(rand(4, V, dtype, 3) * 0.5)
    x[1] = 2.5
    x[2] = -1.0
    x[2, V - 5:] = 1.0
    x[3, ::7] = 9.0
    check(x, [0, 1, V - 1, 7], top=20)


@pytest.mark.parametrize("dtype,width", [(torch.bfloat16, 8), (torch.float32, 4)])
def test_best_tokens_crowded(dtype, width):
    """The best tokens all at the places of one lane: hundreds tie for the last place."""
    x = rand(2, 70001, dtype, 6, sigma=0.5)
    ids = torch.arange(70001, device=DEV)
    x[0, ids % (32 * width) < width] = 7.0
    x[1, ids % (32 * width) == 3] = 7.0
    check(x, [0, 3], top=20)


def test_sharp_and_flat_rows():
    x = rand(4, 70000, torch.float32, 8, sigma=30.0)
    x[2] = 0.0
    x[3] = -1000.0
    x[3, 69999] = 1000.0
    check(x, [1, 2, 3, 69999], [0.05, 0.0, 0.5, 1.0], top=3)


def test_failed_rows_are_reported():
    x = rand(8, 5000, torch.float32, 9)
    x[1, 4999] = float("nan")
    x[2, 0] = float("inf")
    x[3] = float("-inf")
    x[6, 77] = float("nan")
    want = check(x, [1, 1, 1, 1, 5000, -1, -1, 2 ** 31 - 1], top=4)
    assert want[0].tolist() == [0, 4, 4, 4, 5, 0, 0, 5]


def test_no_alternatives_optional_outputs_and_stream():
    x = rand(3, 800, torch.bfloat16, 2)
    check(x, [1, 2, 3], top=0)
    check(x, [1, 2, 3], top=4, stream=torch.cuda.Stream())
    lp = torch.empty(3, device=DEV)
    sv.spec_token_logprobs(x, torch.tensor([1, 2, 3], dtype=torch.int32, device=DEV), lp)
    want = token_logprobs(x.float().cpu().numpy(), [1, 2, 3])
    np.testing.assert_allclose(lp.cpu().numpy(), want[1], rtol=RTOL, atol=ATOL)


def test_rows_past_two_gigabytes():
    """Row offsets beyond 32 bits."""
    V, rows = 1 << 19, 2100  # 2.2 GB of bf16
    x = torch.empty(rows, V, dtype=torch.bfloat16, device=DEV)
    for r in (0, 2060, 2099):
        x[r] = rand(1, V, torch.bfloat16, r)[0]
    tok = torch.full((rows,), -1, dtype=torch.int32, device=DEV)
    for r in (0, 2060, 2099):
        tok[r] = r
    lp = torch.empty(rows, device=DEV)
    sv.spec_token_logprobs(x, tok, lp)
    for r in (0, 2060, 2099):
        want = token_logprobs(x[r:r + 1].float().cpu().numpy(), [r])[1]
        np.testing.assert_allclose(lp[r:r + 1].cpu().numpy(), want, rtol=RTOL, atol=ATOL)


def test_the_same_call_gives_the_same_bits():
    x = rand(64, 30000, torch.bfloat16, 4)
    tok = torch.zeros(64, dtype=torch.int32, device=DEV)
    outs = []
    for _ in range(3):
        lp, ent = torch.empty(64, device=DEV), torch.empty(64, device=DEV)
        sv.spec_token_logprobs(x, tok, lp, entropy=ent)
        outs.append((lp, ent))
    for lp, ent in outs[1:]:
        assert torch.equal(lp, outs[0][0]) and torch.equal(ent, outs[0][1])


def test_binding_refusals():
    x = rand(3, 100, torch.float32, 1)
    tok, lp = torch.zeros(3, dtype=torch.int32, device=DEV), torch.empty(3, device=DEV)
    ids, alt = torch.empty(3, 4, dtype=torch.int32, device=DEV), torch.empty(3, 4, device=DEV)
    bad = [dict(logits=x.double()), dict(logits=x.t()), dict(logits=x.cpu()), dict(tokens=tok.long()),
           dict(tokens=tok[:2]), dict(logprobs=lp.double()), dict(rows=4), dict(top_ids=ids),
           dict(top_ids=ids, top_logprobs=alt[:, :3]), dict(entropy=lp[:2]), dict(temperatures=tok),
           dict(row_status=lp)]
    for kw in bad:
        with pytest.raises(ValueError):
            sv.spec_token_logprobs(**{**dict(logits=x, tokens=tok, logprobs=lp), **kw})
    wide = torch.empty(3, 21, dtype=torch.int32, device=DEV), torch.empty(3, 21, device=DEV)
    with pytest.raises(sv.SpecError):
        sv.spec_token_logprobs(x, tok, lp, top_ids=wide[0], top_logprobs=wide[1])
