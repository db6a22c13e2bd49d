"""GPU parity: query rows of zeros or of tiny numbers, and tiny scales, against the float64 oracle (bounds
in paged_harness), in both kernels: a score's factor must not vanish beside the scores that are hidden."""

import pytest
import torch

import speculative_decoding_verify_bf16_gb300 as sv
from paged_harness import Lanes, attend, check, check_lane

pytestmark = pytest.mark.gpu
KINDS = ["bf16", "e4m3", "int8"]
# Few rows; 24 rows of a head in one lane (tiles); a prompt's part, its last position anywhere in a tile of 128.
LENS = [([3], [500]), ([12], [150]), ([200], [0]), ([200, 5], [40, 300]), ([130], [31])]


@pytest.fixture(scope="module", autouse=True)
def _built():
    sv.build_library()
    sv.load_library()


def run(L, q, window=0, scale=None):
    out, lse, status = attend(L, q, window, scale)
    torch.cuda.synchronize()
    assert status.tolist() == [0] * len(L.lens)
    for b in range(len(L.lens)):
        check_lane(L, b, q, out, lse, window, scale)
    return out


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,before", LENS)
def test_rows_of_zeros(kind, window, d, lens, before):
    """A row, a head and (at last) all of the queries: each output is the mean of what it sees."""
    L = Lanes(lens, before, kind=kind, d=d, seed=sum(lens))
    q = L.queries(4)
    q[1] = 0.0
    q[:, 2] = 0.0
    run(L, q, window)
    run(L, torch.zeros_like(q), window)


@pytest.mark.parametrize("kind", KINDS)
def test_a_cache_of_zeros(kind):
    """A warm-up call: everything is zero."""
    sizes = dict(lens=[200, 3], before=[70, 9])
    L = Lanes(kind=kind, seed=2, **sizes)
    for b, n in enumerate([270, 12]):
        for name in "kv":
            getattr(L, name)[b] = L.put(name, b, 0, torch.zeros(n, L.kv, L.d, device="cuda"))
    out = run(L, torch.zeros_like(L.queries(4)))
    assert (out == 0).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens,before", LENS)
def test_tiny_queries_and_scales(kind, lens, before):
    check(lens, before, kind=kind, q_scale=1e-30, seed=3)
    check(lens, before, kind=kind, q_scale=2.0 ** -90, window=70, seed=4)
    check(lens, before, kind=kind, scale=1e-28, seed=5)
    check(lens, before, kind=kind, scale=2.0 ** -100, seed=6)
    check(lens, before, kind=kind, q_scale=1e-30, scale=1e28, seed=7)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens,before", LENS)
def test_scores_of_zero_between_huge_numbers(kind, lens, before):
    """Queries and keys whose numbers' product is beyond fp32, in components that the other does not have."""
    L = Lanes(lens, before, kind=kind, seed=8)
    for b, n in enumerate(len(x) for x in L.k):
        x = torch.randn(n, L.kv, L.d, generator=L.g, device="cuda") * 2.0 ** 40
        x[..., 0] = 0.0
        L.k[b] = L.put("k", b, 0, x)
    q = torch.zeros_like(L.queries(4))
    q[..., 0] = 2.0 ** 120
    run(L, q)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [3, 200])
def test_an_infinite_scale_is_reported(kind, n):
    L = Lanes([n], [70], kind=kind, seed=9)
    _, _, status = attend(L, L.queries(4), scale=float("inf"))
    torch.cuda.synchronize()
    assert status.tolist() == [sv.SPEC_ERR_NONFINITE]
