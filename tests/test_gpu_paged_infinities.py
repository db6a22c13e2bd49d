"""GPU: infinities in a bf16 cache.  A score of -inf is a weight of 0, as in the formula; what makes an output
NaN or infinite is reported."""

import numpy as np
import pytest
import torch

import speculative_decoding_verify_bf16_gb300 as sv
from paged_harness import DEV, Lanes, attend, check_lane

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    sv.build_library()
    sv.load_library()


def lanes(n, seed):
    """Two lanes; every query's component 3 is 1."""
    L = Lanes([n, 2], [90, 33], seed=seed)
    q = L.queries(4)
    q[..., 3] = 1.0
    return L, q


def with_number(L, name, pos, component, x):
    t = torch.tensor(getattr(L, name)[0][pos:pos + 1]).to(DEV)
    t[..., component] = x
    L.put(name, 0, pos, t)


def call(L, q, whole):
    out, lse, status = attend(L, q, workspace=torch.empty(0, dtype=torch.uint8, device=DEV) if whole else None)
    torch.cuda.synchronize()
    check_lane(L, 1, q, out, lse)
    return out, lse, status.tolist()


@pytest.mark.parametrize("whole", [False, True])
@pytest.mark.parametrize("n", [1, 4, 12, 200])
@pytest.mark.parametrize("positions", [[17], [0], [89], [16, 17, 40, 41, 42]])
def test_a_key_whose_scores_are_minus_infinity_weighs_nothing(n, positions, whole):
    L, q = lanes(n, 1)
    for p in positions:
        with_number(L, "k", p, 3, -INF)
    out, lse, status = call(L, q, whole)
    assert status == [0, 0]
    # the same without these positions
    L.k[0], L.v[0] = np.delete(L.k[0], positions, 0), np.delete(L.v[0], positions, 0)
    L.before[0] -= len(positions)
    check_lane(L, 0, q, out, lse)


@pytest.mark.parametrize("whole", [False, True])
@pytest.mark.parametrize("n", [1, 4, 12, 200])
@pytest.mark.parametrize("name,number", [("k", INF), ("v", INF), ("v", -INF), ("q", INF), ("q", -INF)])
def test_infinities_that_reach_an_output_are_reported(n, name, number, whole):
    L, q = lanes(n, 2)
    if name == "q":
        q[n - 1, 1, 5] = number
    else:
        with_number(L, name, 17, 3, number)
    assert call(L, q, whole)[2] == [sv.SPEC_ERR_NONFINITE, 0]


@pytest.mark.parametrize("whole", [False, True])
@pytest.mark.parametrize("n", [1, 4, 12, 200])
def test_a_row_that_gives_nothing_any_weight_is_reported(n, whole):
    L, q = lanes(n, 3)
    for p in range(90 + n):
        with_number(L, "k", p, 3, -INF)
    assert call(L, q, whole)[2] == [sv.SPEC_ERR_NONFINITE, 0]


@pytest.mark.parametrize("n", [1, 4, 12, 200])
def test_a_key_of_infinities_that_a_query_does_not_have_is_reported(n):
    """0 * inf is NaN."""
    L, q = lanes(n, 4)
    q[..., 3] = 0.0
    with_number(L, "k", 17, 3, -INF)
    assert call(L, q, False)[2] == [sv.SPEC_ERR_NONFINITE, 0]
