"""GPU: the prefill's scratch memory.  A buffer for the largest call serves every smaller one,
and one of any size is taken as it is, without a byte touched behind it.

Bounds as for the chunked form elsewhere: states within 2^-15 of their magnitude, outputs within
that and their own rounding, 2^-8 of their value."""

import numpy as np
import pytest
import torch

import speculative_decoding_verify_bf16_gb300 as sv
from oracle.linear import linear_attention

pytestmark = pytest.mark.gpu
DEV = "cuda"
STATE = (128 * 128 + 4) * 4  # a segment's state and decay


@pytest.fixture(scope="module", autouse=True)
def _built():
    sv.build_library()
    sv.load_library()


def test_it_grows_with_lanes_and_lengths_up_to_a_bound():
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    lens = [8, 900, 1000, 1024, 1500, 2049, 2304, 2432, 4096, 16384, 1 << 20]
    for heads in (1, 2, 3, 5, 16, 40, 76, 77, 300):
        size = [[sv.spec_linear_workspace(b, heads, 128, 128, n) for n in lens] for b in (1, 2, 3, 4, 5, 8, 20, 64, 300)]
        size = np.array(size)
        assert (np.diff(size, axis=0) >= 0).all() and (np.diff(size, axis=1) >= 0).all()
        assert size.max() <= sms * STATE and (size[:, 0] == 0).all()
        assert (size.max() > 0) == (2 * heads <= sms)


def prompts(lens, h, seed=1):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    n = sum(lens)
    q, k, v = (torch.randn(n, h, 128, generator=g, device=DEV).div(11).to(torch.bfloat16) for _ in range(3))
    decay = -0.01 * torch.rand(n, h, generator=g, device=DEV)
    S = torch.randn(len(lens), h, 128, 128, generator=g, device=DEV)
    return q, k, v, decay, S


def check(lens, h, workspace, want):
    q, k, v, decay, S = prompts(lens, h)
    out, final = torch.empty_like(v), torch.empty_like(S)
    status = torch.zeros(len(lens), dtype=torch.int32, device=DEV)
    ends = np.cumsum([0] + lens)
    sv.spec_linear_prefill(q, k, v, decay, torch.tensor(ends, dtype=torch.int32, device=DEV), S, out, final, max(lens),
                           lane_status=status, workspace=workspace)
    torch.cuda.synchronize()
    assert not status.any()
    if want is None:
        want = linear_attention(*[t.double().cpu().numpy() for t in (q, k, v, decay)], ends, S.double().cpu().numpy(),
                                scale=128 ** -0.5)
    o, s, _, mag, fmag = want
    assert (np.abs(out.double().cpu().numpy() - o) <= 2.0 ** -15 * mag + 2.0 ** -8 * np.abs(o)).all()
    assert (np.abs(final.double().cpu().numpy() - s) <= 2.0 ** -15 * fmag).all()
    return want


def test_a_buffer_for_the_largest_call_serves_smaller_ones():
    h = 2
    workspace = sv.new_linear_workspace(8, h, 128, 128, 4000, DEV)
    for lens in ([2304], [2432], [1100], [4000], [1500, 40, 0, 1300], [1024] * 8, [2500, 2500, 100], [7]):
        check(lens, h, workspace, None)
    # (a lane of 2304 tokens is cut into more segments than one of 2432)
    check([2304], 16, sv.new_linear_workspace(1, 16, 128, 128, 2432, DEV), None)


@pytest.mark.parametrize("lens,h", [([3000], 2), ([1500, 0, 2200], 1)])
def test_any_size_will_do(lens, h):
    full = sv.spec_linear_workspace(len(lens), h, 128, 128, max(lens))
    assert full > 0
    want, pairs = None, len(lens) * h
    for size in (0, 16, pairs * STATE, 2 * pairs * STATE - 16, 2 * pairs * STATE, 5 * pairs * STATE + 48, full, full + (1 << 20)):
        buf = torch.full((size + 4096,), 171, dtype=torch.uint8, device=DEV)
        want = check(lens, h, buf[:size], want)
        assert (buf[size:] == 171).all()


def test_misaligned_scratch_memory_is_refused():
    q, k, v, decay, S = prompts([3000], 1)
    buf = torch.zeros(sv.spec_linear_workspace(1, 1, 128, 128, 3000) + 16, dtype=torch.uint8, device=DEV)
    with pytest.raises(sv.SpecError):
        sv.spec_linear_prefill(q, k, v, decay, torch.tensor([0, 3000], dtype=torch.int32, device=DEV), S, torch.empty_like(v),
                               S.clone(), 3000, workspace=buf[4:])
