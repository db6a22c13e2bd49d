"""GPU: lanes that fail in some of their heads, while other thread blocks of the same lanes
start: each lane is reported, and no other lane's numbers change."""

import pytest
import torch

import speculative_decoding_verify_bf16_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    sv.build_library()
    sv.load_library()


@pytest.mark.parametrize("form", ["prefill", "verify"])
@pytest.mark.parametrize("lanes,heads,d", [(48, 16, 128), (7, 64, 64)])
def test_failing_heads_leave_other_lanes_alone(form, lanes, heads, d):
    g = torch.Generator(device=DEV)
    g.manual_seed(lanes)
    n = 6
    q, k, v = (torch.randn(lanes * n, heads, d, generator=g, device=DEV).div(8) for _ in range(3))
    decay = -torch.rand(lanes * n, heads, generator=g, device=DEV)
    offsets = torch.arange(0, lanes * n + 1, n, dtype=torch.int32, device=DEV)
    live = torch.randn(lanes, heads, d, d, generator=g, device=DEV)

    def run(v):
        out, status = torch.full_like(v, 7.0), torch.zeros(lanes, dtype=torch.int32, device=DEV)
        if form == "prefill":
            to = torch.full_like(live, 7.0)
            sv.spec_linear_prefill(q, k, v, decay, offsets, live, out, to, n, lane_status=status)
        else:
            to = torch.full((lanes, n, heads, d, d), 7.0, device=DEV)
            sv.spec_linear_verify(q, k, v, decay, offsets, live, to, out, lane_status=status)
        torch.cuda.synchronize()
        return out.view(lanes, n, heads, d), to, status

    good = run(v)
    assert not good[2].any()
    bad = v.clone().view(lanes, n, heads, d)
    bad[::3, 0, 0, 1] = float("nan")
    bad[::3, 2, heads // 2, 5] = float("inf")
    for _ in range(10):
        got = run(bad.view_as(v))
        want = torch.zeros(lanes, dtype=torch.int32, device=DEV)
        want[::3] = sv.SPEC_ERR_NONFINITE
        assert torch.equal(got[2], want)
        well = want == 0
        assert torch.equal(got[0][well], good[0][well]) and torch.equal(got[1][well], good[1][well])
