"""GPU parity: linear attention with decay against the float64 recurrence.

Bounds, with A the recurrence's magnitudes (every term by its absolute value), u = 2^-24:

* recurrent form (spec_linear_verify, fp32 prompts): each step rounds the decay (expf,
  2 ulp), a product and a sum, so after t steps a state is within (5 t + 2) u A, and an
  output sums dk products of it: (5 t + dk + 10) u of its magnitude.
* chunked form (bf16 prompts): the weights of a state's terms are held to 2^-16
  (two bf16 parts), products and sums in fp32, a chunk's 128 products in one sum: a
  state is within 2^-15 A.  An output's scores and states may each be rounded once to
  bf16 on the way: 2^-8 of its magnitude in the worst case; over many outputs these
  roundings are independent, and the root mean square error is held to 2^-8 of the
  root mean square output.
* an output in bf16 (8 significant bits) adds its own rounding, 2^-8 of its value, and inputs are taken
  exactly as the kernel gets them (bf16 or fp32).
"""

import numpy as np
import pytest
import torch

import speculative_decoding_verify_bf16_gb300 as sv
from oracle.linear import linear_attention

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    sv.build_library()
    sv.load_library()


def offsets_of(lens):
    return torch.tensor(np.cumsum([0] + list(lens)), dtype=torch.int32, device=DEV)


def make(lens, hk, hv, dk, dv, dtype, seed, state=True, resets=0.0, slow=1e-3, fast=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    n = sum(lens)
    unit = lambda h: torch.nn.functional.normalize(torch.randn(n, h, dk, generator=g, device=DEV), dim=-1).to(dtype)
    q, k = unit(hk), unit(hk)
    v = torch.randn(n, hv, dv, generator=g, device=DEV).to(dtype)
    rate = torch.logspace(np.log10(slow), np.log10(fast), hv, device=DEV)
    decay = -rate * torch.nn.functional.softplus(torch.randn(n, hv, generator=g, device=DEV))
    if resets:
        decay[torch.rand(n, generator=g, device=DEV) < resets] = float("-inf")
    S = torch.randn(len(lens), hv, dk, dv, generator=g, device=DEV) if state else None
    return q, k, v, decay, S


def host(*ts):
    return [None if t is None else t.double().cpu().numpy() for t in ts]


def check_prefill(lens, hk=2, hv=2, dk=128, dv=128, dtype=torch.bfloat16, seed=0, state=True, scale=None, inputs=None,
                  in_place=False, stream=None, **kw):
    q, k, v, decay, S = inputs or make(lens, hk, hv, dk, dv, dtype, seed, state, **kw)
    lanes = len(lens)
    out = torch.full(v.shape, 7.0, dtype=dtype, device=DEV)
    final = S.clone() if in_place else torch.full((lanes, hv, dk, dv), 7.0, device=DEV)
    status = torch.zeros(lanes, dtype=torch.int32, device=DEV)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    sv.spec_linear_prefill(q, k, v, decay, offsets_of(lens), final if in_place else S, out, final, max(lens), scale=scale,
                           lane_status=status, stream=stream)
    torch.cuda.synchronize()
    assert status.tolist() == [0] * lanes
    want, wfinal, _, mag, fmag = linear_attention(*host(q, k, v, decay), np.cumsum([0] + list(lens)), *host(S),
                                                  scale=dk ** -0.5 if scale is None else scale)
    got, gfinal = host(out, final)
    t = max(lens)
    rec_s, rec_o = (5 * t + 2) * U, (5 * t + dk + 10) * U
    if dtype == torch.bfloat16:
        bound_o = (2.0 ** -8 + rec_o) * mag + 2.0 ** -8 * np.abs(want)
        bound_s = (2.0 ** -15 + rec_s) * fmag
    else:
        bound_o, bound_s = rec_o * mag, rec_s * fmag
    assert (np.abs(gfinal - wfinal) <= bound_s + 1e-30).all(), np.max(np.abs(gfinal - wfinal) / (bound_s + 1e-30))
    if want.size:
        assert (np.abs(got - want) <= bound_o + 1e-30).all(), np.max(np.abs(got - want) / (bound_o + 1e-30))
        if want.size >= 4096:
            assert np.sqrt(np.mean((got - want) ** 2)) <= 2.0 ** -8 * np.sqrt(np.mean(want ** 2))
    return out, final


@pytest.mark.parametrize("n", [1, 2, 15, 16, 63, 64, 65, 127, 128, 129, 191, 255, 256, 257, 400, 1000])
def test_prefill_lengths(n):
    check_prefill([n], seed=n)


@pytest.mark.parametrize("lens", [[0, 5, 0, 130, 1], [128, 128, 128], [300, 1, 77, 0], [1] * 9, [513, 12, 260, 128, 127]])
@pytest.mark.parametrize("state", [True, False])
def test_prefill_ragged_lanes(lens, state):
    check_prefill(lens, hv=4, seed=len(lens), state=state)


def test_prefill_long_and_split():
    """Few heads and a long axis: the work of one head is split."""
    check_prefill([3000], hk=1, hv=2, seed=1)
    check_prefill([2049, 130], hk=1, hv=1, seed=2, slow=1e-4, fast=1e-4)
    check_prefill([2000, 0, 700], hk=1, hv=1, dk=64, dv=96, seed=3)
    check_prefill([1500], hk=1, hv=1, dk=72, dv=64, seed=4, in_place=True)
    check_prefill([1500], hk=1, hv=1, seed=5, in_place=True)


@pytest.mark.parametrize("hk,hv", [(1, 1), (2, 4), (3, 9), (16, 16)])
def test_prefill_head_layouts(hk, hv):
    check_prefill([200, 37], hk=hk, hv=hv, seed=hv)


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (256, 256), (48, 20), (1, 4), (130, 132), (24, 40),
                                   (104, 8), (128, 128)])
def test_prefill_head_sizes(dk, dv):
    check_prefill([150, 20], dk=dk, dv=dv, seed=dk + dv)


@pytest.mark.parametrize("n", [1, 40, 300])
def test_prefill_fp32(n):
    check_prefill([n, 3], dtype=torch.float32, seed=n)


def test_prefill_strong_decays_and_resets():
    check_prefill([700], seed=1, resets=0.02)
    check_prefill([300], seed=2, resets=0.6)
    check_prefill([300], seed=3, slow=20.0, fast=400.0)
    q, k, v, decay, S = make([300], 2, 2, 128, 128, torch.bfloat16, 4)
    decay[100:110] = torch.finfo(torch.float32).min
    decay[0] = -150.0
    decay[299] = float("-inf")
    check_prefill([300], inputs=(q, k, v, decay, S))


def test_prefill_no_decay_and_growth():
    q, k, v, decay, S = make([400], 2, 2, 128, 128, torch.bfloat16, 5)
    check_prefill([400], inputs=(q, k, v, torch.zeros_like(decay), S))
    check_prefill([400], inputs=(q, k, v, torch.full_like(decay, 0.01), S))


def test_prefill_strides_and_shared_decay():
    """q, k, v as slices of one projection, head-major v, a decay a head by expand."""
    n, h, d = 333, 4, 128
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    proj = (torch.randn(n, 2 * h * d + 8, generator=g, device=DEV) / 11).to(torch.bfloat16)
    q = proj[:, :h * d].view(n, h, d)
    k = proj[:, h * d:2 * h * d].view(n, h, d)
    v = torch.randn(h, n, d, generator=g, device=DEV).to(torch.bfloat16).transpose(0, 1)
    decay = -torch.tensor([0.001, 0.01, 0.1, 1.0], device=DEV).expand(n, h)
    check_prefill([300, 33], hk=h, hv=h, inputs=(q, k, v, decay, None), state=False, scale=0.5)
    # rows that no 16-byte load can take
    odd = (torch.randn(n, h, d + 1, generator=g, device=DEV) / 11).to(torch.bfloat16)
    check_prefill([300, 33], hk=h, hv=h, inputs=(odd[:, :, :d], k, v, decay, None), state=False)
    flat = torch.randn(n * h * d + 1, generator=g, device=DEV).to(torch.bfloat16)[1:].view(n, h, d)
    check_prefill([300, 33], hk=h, hv=h, inputs=(q, k, flat, decay, None), state=False)


def test_prefill_in_place_and_on_another_stream():
    a = check_prefill([200, 64], seed=7, in_place=True)
    b = check_prefill([200, 64], seed=7, stream=torch.cuda.Stream())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_prefill_in_pieces_equals_whole():
    """A prompt taken in two calls through the state."""
    q, k, v, decay, S = make([500], 2, 2, 128, 128, torch.bfloat16, 8)
    whole = check_prefill([500], inputs=(q, k, v, decay, S))
    cut = 190
    mid = torch.empty_like(S)
    out = torch.empty_like(v)
    sv.spec_linear_prefill(q[:cut], k[:cut], v[:cut], decay[:cut], offsets_of([cut]), S, out[:cut], mid, cut)
    sv.spec_linear_prefill(q[cut:], k[cut:], v[cut:], decay[cut:], offsets_of([500 - cut]), mid, out[cut:], mid, 500 - cut)
    torch.cuda.synchronize()
    want, wfinal, _, mag, fmag = linear_attention(*host(q, k, v, decay), [0, 500], *host(S), scale=128 ** -0.5)
    assert (np.abs(host(mid)[0] - wfinal) <= (2.0 ** -14 + 2502 * U) * fmag).all()
    assert (np.abs(host(out)[0] - want) <= (2.0 ** -8 + 2700 * U) * mag + 2.0 ** -8 * np.abs(want)).all()
    assert whole[0].shape == out.shape


def test_prefill_rows_behind_a_lane_do_not_leak():
    """NaN and infinities in rows of no lane, or of the next lane, stay there."""
    lens = [70, 90]
    q, k, v, decay, S = make([70, 90, 60], 2, 2, 128, 128, torch.bfloat16, 9)
    S = S[:2].contiguous()
    clean = [x[:160].clone() for x in (q, k, v, decay)]
    want = check_prefill(lens, inputs=(*clean, S))
    for x in (q, k, v):
        x[160:] = float("nan")
        x[200:] = float("inf")
    decay[160:] = float("nan")
    out, final = torch.empty_like(v), torch.empty_like(S)
    status = torch.zeros(2, dtype=torch.int32, device=DEV)
    sv.spec_linear_prefill(q, k, v, decay, offsets_of(lens), S, out, final, 90, lane_status=status)
    torch.cuda.synchronize()
    assert status.tolist() == [0, 0]
    assert torch.equal(out[:160], want[0]) and torch.equal(final, want[1])
    # a bad lane does not touch its neighbour
    v2 = v.clone()
    v2[30] = float("inf")
    sv.spec_linear_prefill(q, k, v2, decay, offsets_of(lens), S, out, final, 90, lane_status=status)
    torch.cuda.synchronize()
    assert status.tolist() == [sv.SPEC_ERR_NONFINITE, 0]
    assert torch.equal(out[70:160], want[0][70:]) and torch.equal(final[1], want[1][1])


@pytest.mark.parametrize("n", [40, 300])
@pytest.mark.parametrize("what", ["k", "v", "decay", "state"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_prefill_nonfinite_inputs_are_reported(n, what, bad):
    q, k, v, decay, S = make([n, n], 2, 2, 128, 128, torch.bfloat16, 10)
    {"k": k, "v": v, "decay": decay}.get(what, S[0, 1])[(3,) if what == "state" else (n // 2, 1)] = bad
    status = torch.zeros(2, dtype=torch.int32, device=DEV)
    out, final = torch.empty_like(v), torch.empty_like(S)
    sv.spec_linear_prefill(q, k, v, decay, offsets_of([n, n]), S, out, final, n, lane_status=status)
    torch.cuda.synchronize()
    assert status.tolist() == [sv.SPEC_ERR_NONFINITE, 0]


@pytest.mark.parametrize("n", [3, 300])
def test_lanes_left_out(n):
    """Bad offsets and lanes that failed before leave outputs and states alone."""
    q, k, v, decay, S = make([n] * 4, 2, 2, 128, 128, torch.bfloat16, 11)
    off = offsets_of([n] * 4)
    off[4] = 4 * n + 5                    # the last lane reaches past the rows
    status = torch.tensor([0, 4, 0, 0], dtype=torch.int32, device=DEV)
    out, final = torch.full_like(v, 7.0), torch.full_like(S, 7.0)
    sv.spec_linear_prefill(q, k, v, decay, off, S, out, final, n + 9, lane_status=status)
    torch.cuda.synchronize()
    assert status.tolist() == [0, 4, 0, sv.SPEC_ERR_LAYOUT]
    for b in (1, 3):
        assert (out[b * n:(b + 1) * n] == 7).all() and (final[b] == 7).all()
    for b in (0, 2):
        assert not (out[b * n:(b + 1) * n] == 7).all() and not (final[b] == 7).all()
    status.zero_()
    sv.spec_linear_prefill(q, k, v, decay, offsets_of([n] * 4), S, out, final, n - 1, lane_status=status)
    torch.cuda.synchronize()
    assert status.tolist() == [sv.SPEC_ERR_LAYOUT] * 4   # longer than max_len says


# ---------------------------------------------------------------------------
# Columns of a round
# ---------------------------------------------------------------------------
def check_verify(lens, cols, hk=2, hv=2, dk=128, dv=128, dtype=torch.bfloat16, seed=0, state=True, **kw):
    q, k, v, decay, S = make(lens, hk, hv, dk, dv, dtype, seed, state, **kw)
    lanes = len(lens)
    out = torch.full(v.shape, 7.0, dtype=dtype, device=DEV)
    staged = torch.full((lanes, cols, hv, dk, dv), 7.0, device=DEV)
    live = None if S is None else S.clone()
    status = torch.zeros(lanes, dtype=torch.int32, device=DEV)
    sv.spec_linear_verify(q, k, v, decay, offsets_of(lens), live, staged, out, lane_status=status)
    torch.cuda.synchronize()
    assert status.tolist() == [0] * lanes
    assert live is None or torch.equal(live, S)
    want, _, snaps, mag, fmag = linear_attention(*host(q, k, v, decay), np.cumsum([0] + list(lens)), *host(S),
                                                 scale=dk ** -0.5)
    got, gst = host(out, staged)
    round_o = 2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0.0
    assert (np.abs(got - want) <= (5 * cols + dk + 10) * U * mag + round_o).all()
    S0 = np.zeros((lanes, hv, dk, dv)) if S is None else host(S)[0]
    for b, n in enumerate(lens):
        # magnitudes of a snapshot: bounded by the largest a prefix reaches
        top = np.abs(S0[b]).max() + sum(np.abs(host(k)[0]).max() * np.abs(host(v)[0]).max() for _ in range(n))
        assert (np.abs(gst[b, :n] - snaps[b]) <= (5 * n + 2) * U * top).all()
        assert (gst[b, n:] == 7).all()
    return q, k, v, decay, S, out, staged


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", [1, 2, 4, 8, 9, 16, 17])
def test_verify_columns(cols, dtype):
    check_verify([cols, 1, max(1, cols - 1)], cols, seed=cols, dtype=dtype)


@pytest.mark.parametrize("dk,dv,hk,hv", [(64, 64, 1, 4), (256, 256, 1, 1), (96, 32, 2, 2), (8, 100, 1, 3), (3, 4, 1, 1)])
def test_verify_shapes(dk, dv, hk, hv):
    check_verify([3, 0, 5], 5, hk, hv, dk, dv, torch.float32, seed=dk)
    check_verify([3, 0, 5], 5, hk, hv, dk, dv, torch.bfloat16, seed=dk, state=False)


@pytest.mark.parametrize("lanes,hv", [(1, 16), (64, 16), (5, 1), (300, 2)])
def test_verify_lane_and_head_counts(lanes, hv):
    rng = np.random.default_rng(lanes)
    check_verify(rng.integers(1, 4, lanes).tolist(), 3, hv, hv, 64, 32, seed=lanes)


def test_verify_columns_equal_single_token_decoding_bit_for_bit():
    lens = [6, 3]
    q, k, v, decay, S, out, staged = check_verify(lens, 6, hk=1, hv=2, seed=12, resets=0.1)
    first = [0, 6]
    for b, n in enumerate(lens):
        live = S[b:b + 1].clone()
        for t in range(n):
            r = slice(first[b] + t, first[b] + t + 1)
            o = torch.empty_like(v[r])
            sv.spec_linear_verify(q[r], k[r], v[r], decay[r], offsets_of([1]), live, live.unsqueeze(1), o)
            assert torch.equal(o, out[r]) and torch.equal(live[0], staged[b, t]), (b, t)


def test_verify_on_layer_views_then_commit():
    """Snapshots and live states of one layer inside [lanes][cols][layers]..., rolled by
    the commit."""
    lanes, cols, layers, h, d = 3, 4, 2, 2, 64
    g = torch.Generator(device=DEV)
    g.manual_seed(13)
    live = torch.randn(lanes, layers, h, d, d, generator=g, device=DEV)
    staged = torch.zeros(lanes, cols, layers, h, d, d, device=DEV)
    snaps = []
    for layer in range(layers):
        q, k, v, decay, _ = make([cols] * lanes, h, h, d, d, torch.float32, 14 + layer)
        out = torch.empty_like(v)
        sv.spec_linear_verify(q, k, v, decay, offsets_of([cols] * lanes), live[:, layer], staged[:, :, layer], out)
        snaps.append(linear_attention(*host(q, k, v, decay), [0, 4, 8, 12], *host(live[:, layer]), scale=d ** -0.5)[2])
    committed = torch.tensor([1, 4, 2], dtype=torch.int32, device=DEV)
    sv.spec_commit_state(staged, live, committed)
    torch.cuda.synchronize()
    for b, c in enumerate(committed.tolist()):
        for layer in range(layers):
            np.testing.assert_allclose(live[b, layer].cpu().numpy(), snaps[layer][b][c - 1], rtol=1e-5, atol=1e-5)


def test_verify_reports_and_leaves_out():
    q, k, v, decay, S = make([2, 3, 2], 2, 2, 128, 128, torch.float32, 15)
    v[1, 0, 5] = float("nan")
    out = torch.full_like(v, 7.0)
    staged = torch.full((3, 2, 2, 128, 128), 7.0, device=DEV)
    status = torch.zeros(3, dtype=torch.int32, device=DEV)
    sv.spec_linear_verify(q, k, v, decay, offsets_of([2, 3, 2]), S, staged, out, lane_status=status)
    torch.cuda.synchronize()
    assert status.tolist() == [sv.SPEC_ERR_NONFINITE, sv.SPEC_ERR_LAYOUT, 0]  # the second has more columns than fit
    assert (out[2:5] == 7).all() and (staged[1] == 7).all()


def test_state_offsets_past_32_bits():
    """Lane strides beyond 2^31 elements."""
    lanes, h, d = 2, 1, 128
    stride = (1 << 31) + 1024
    big = torch.empty(stride + h * d * d, device=DEV)
    live = big.as_strided((lanes, h, d, d), (stride, d * d, d, 1))
    live.normal_()
    S = live.clone()
    q, k, v, decay, _ = make([1, 1], h, h, d, d, torch.float32, 16)
    out = torch.empty_like(v)
    sv.spec_linear_verify(q, k, v, decay, offsets_of([1, 1]), live, live.unsqueeze(1), out)
    torch.cuda.synchronize()
    want = linear_attention(*host(q, k, v, decay), [0, 1, 2], *host(S), scale=d ** -0.5)
    np.testing.assert_allclose(live.cpu().numpy(), want[1], rtol=1e-5, atol=1e-5)
    del big, live


def test_binding_refusals():
    q, k, v, decay, S = make([4, 4], 2, 4, 64, 64, torch.bfloat16, 17)
    off, out = offsets_of([4, 4]), torch.empty_like(v)
    good = dict(q=q, k=k, v=v, log_decay=decay, row_offsets=off, out=out)
    bad = [dict(q=q.float()), dict(k=k[:, :1]), dict(k=k[:7]), dict(v=v[:, :3], out=out[:, :3]), dict(out=out[:, :2]),
           dict(v=v.transpose(1, 2)), dict(log_decay=decay.double()), dict(log_decay=decay[:, :2]),
           dict(row_offsets=off.long()), dict(q=q.cpu())]
    for kw in bad:
        with pytest.raises(ValueError):
            sv.spec_linear_prefill(**{**good, **kw}, state_in=S, state_out=S, max_len=4)
        with pytest.raises(ValueError):
            sv.spec_linear_verify(**{**good, **kw}, live=S, staged=S.unsqueeze(1).repeat(1, 4, 1, 1, 1))
    for st in (S[:1], S.double(), S.transpose(2, 3), S[..., :32]):
        with pytest.raises(ValueError):
            sv.spec_linear_prefill(**good, state_in=st, state_out=None, max_len=4)
        with pytest.raises(ValueError):
            sv.spec_linear_prefill(**good, state_in=None, state_out=st, max_len=4)
    with pytest.raises(ValueError):
        sv.spec_linear_verify(**good, live=S, staged=S)
    with pytest.raises(sv.SpecError):
        sv.spec_linear_prefill(**good, state_in=S, state_out=S, max_len=-1)
