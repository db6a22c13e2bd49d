"""GPU: the attention leaves lanes out that had failed before the call, and a lane's first error stays."""

import numpy as np
import pytest
import torch

import speculative_decoding_verify_bf16_gb300 as sv
from paged_harness import DEV, Lanes, attend, check_lane, i32

pytestmark = pytest.mark.gpu
KINDS = ["bf16", "e4m3", "int8"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    sv.build_library()
    sv.load_library()


def scratch(whole):
    return torch.empty(0, dtype=torch.uint8, device=DEV) if whole else None


def verify(L, q, entry, got, b_checked=None):
    """Left-out lanes' rows and codes as they were, the others right."""
    out, lse, status = got
    torch.cuda.synchronize()
    assert status.tolist() == entry
    ends = np.cumsum([0] + L.lens)
    for b, code in enumerate(entry):
        rows = slice(ends[b], ends[b + 1])
        if code:
            assert (out[rows] == 7).all() and (lse[rows] == 7).all(), b
        elif L.lens[b] and (b_checked is None or b in b_checked):
            check_lane(L, b, q, out, lse)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 3, 12, 200])
@pytest.mark.parametrize("whole", [False, True])
def test_failed_lanes_are_left_out(kind, d, n, whole):
    lens = [n, n, 2, 0, n, 1, n]
    L = Lanes(lens, [40, 300, 700, 9, 0, 33, 500], kind=kind, d=d, seed=n)
    q = L.queries(4)
    entry = [0, sv.SPEC_ERR_TOKEN_RANGE, 0, sv.SPEC_ERR_LAYOUT, sv.SPEC_ERR_TIMEOUT, 0, -5]
    q[n:2 * n] = float("nan")  # nothing of a left-out lane is looked at
    L.host_tables[4] = -1
    L.tables = torch.tensor(L.host_tables, device=DEV)
    L.cached[6] = -3
    verify(L, q, entry, attend(L, q, status=i32(entry), workspace=scratch(whole)))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [2, 200])
@pytest.mark.parametrize("whole", [False, True])
def test_long_lanes_beside_left_out_ones(kind, n, whole):
    L = Lanes([n, n, n], [9000, 4000, 3000], kind=kind, seed=n, d=64)
    q = L.queries(4)
    for entry in ([4, 0, 0], [0, 4, 0], [0, 0, 4], [4, 0, 4], [4, 4, 4]):
        verify(L, q, entry, attend(L, q, status=i32(entry), workspace=scratch(whole)), b_checked=[] if n > 2 else None)


@pytest.mark.parametrize("lanes", [150, 700, 1400])
def test_many_lanes(lanes):
    rng = np.random.default_rng(lanes)
    lens = rng.integers(0, 3, lanes).tolist()
    L = Lanes(lens, rng.integers(0, 60, lanes).tolist(), kind="int8", kv=1, d=64, seed=lanes)
    q = L.queries(2)
    entry = (rng.integers(0, 3, lanes) == 0).astype(int) * 5
    for whole in (False, True):
        verify(L, q, entry.tolist(), attend(L, q, status=i32(entry), workspace=scratch(whole)))


@pytest.mark.parametrize("n", [2, 200])
def test_captured_and_replayed_with_other_lanes_left_out(n):
    L = Lanes([n, n, n], [400, 30, 1000], kind="e4m3", seed=1)
    q = L.queries(4)
    out, lse, status = torch.empty_like(q), torch.empty(3 * n, 4, device=DEV), i32([0, 0, 0])
    ws = sv.new_paged_attention_workspace(4, L.kv, L.d, n, DEV)
    call = lambda: sv.spec_paged_attention(q, *L.where(), out, n, lse=lse, lane_status=status, workspace=ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for entry in ([0, 0, 0], [0, 5, 0], [4, 0, 6], [0, 0, 0]):
        out.fill_(7), lse.fill_(7), status.copy_(i32(entry))
        graph.replay()
        verify(L, q, entry, (out, lse, status))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [2, 200])
@pytest.mark.parametrize("whole", [False, True])
def test_codes_of_this_call_are_plain(kind, n, whole):
    """What a call reports is a code of the header, and it keeps the next call from the lane."""
    L = Lanes([n, n, n, n], [400, 300, 1000, 5000], kind=kind, d=64, seed=2)
    q = L.queries(4)
    q[n + 1, 2, 5] = float("nan")
    L.host_tables[2, 1] = 10 ** 6
    L.tables = torch.tensor(L.host_tables, device=DEV)
    L.cached[3] = -1
    want = [0, sv.SPEC_ERR_NONFINITE, sv.SPEC_ERR_LAYOUT, sv.SPEC_ERR_LAYOUT]
    out, lse, status = attend(L, q, workspace=scratch(whole))
    torch.cuda.synchronize()
    assert status.tolist() == want
    verify(L, q, want, attend(L, q, status=status, workspace=scratch(whole)))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 300])
@pytest.mark.parametrize("whole", [False, True])
def test_a_wait_that_gives_up_keeps_an_earlier_error(monkeypatch, kind, n, whole):
    """The first lane names a page that is none, then its copy does not come."""
    L = Lanes([n, n], [9000, 9000], kind=kind, kv=1, seed=1)
    q = L.queries(8)
    L.host_tables[0, 0] = -1
    L.tables = torch.tensor(L.host_tables, device=DEV)
    monkeypatch.setenv("SPEC_PAGED_TEST_WITHHOLD_COPY", "1")
    out, lse, status = attend(L, q, workspace=scratch(whole))
    torch.cuda.synchronize()
    assert status.tolist()[0] == sv.SPEC_ERR_LAYOUT
