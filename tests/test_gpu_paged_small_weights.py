"""GPU parity: weights far below a row's largest, which many positions together make count (8-bit
caches, whose weights enter a product as fp16 numbers)."""

import pytest
import torch

import speculative_decoding_verify_bf16_gb300 as sv
from paged_floors import check_lane
from paged_harness import DEV, Lanes, attend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    sv.build_library()
    sv.load_library()


def run(L, q, window=0, scale=None, workspace=None, floor=2.0 ** -32):
    out, lse, status = attend(L, q, window, scale, workspace)
    torch.cuda.synchronize()
    assert status.tolist() == [0] * len(L.lens)
    for b in range(len(L.lens)):
        check_lane(L, b, q, out, lse, window, scale, floor)
    return out


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,before", [(1, 300), (3, 20000), (12, 1000), (200, 800)])
@pytest.mark.parametrize("loud", [0, 37, 290])
def test_one_position_far_above_the_others(kind, d, n, before, loud):
    """2^25.6 or 2^26 times the others' weight, and a value in another component: without the many small
    weights that component would be empty.  (The rows' second half sees them alone.)"""
    L = Lanes([n], [before], kind=kind, kv=1, d=d, seed=loud)
    k, v = (torch.zeros(before + n, 1, d, device=DEV) for _ in range(2))
    k[loud, 0, 0] = 17.75
    v[:, 0, 1] = 1.0
    v[loud, 0, 0], v[loud, 0, 1] = 1.0, 0.0
    L.k[0], L.v[0] = L.put("k", 0, 0, k), L.put("v", 0, 0, v)
    q = torch.zeros(n, 4, d, dtype=torch.bfloat16, device=DEV)
    q[:, :2, 0] = 1.0
    for workspace in (None, torch.empty(0, dtype=torch.uint8, device=DEV)):
        out = run(L, q, scale=1.0, workspace=workspace).double()
        assert (out[:, :2, 1] >= 0.9 * before * 2.0 ** -26).all()


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("lens,before", [([3, 1], [500, 90]), ([12], [700]), ([180, 9], [300, 0])])
@pytest.mark.parametrize("q_scale", [1.0, 4.0, 12.0])
@pytest.mark.parametrize("window", [0, 100])
def test_peaked_rows(kind, lens, before, q_scale, window):
    L = Lanes(lens, before, kind=kind, seed=5)
    # (tiles of many rows have one exponent for 32 positions: up to 7 above a position's own, and so M)
    run(L, L.queries(4, q_scale), window, floor=2.0 ** -25 if lens[0] > 4 else 2.0 ** -32)
