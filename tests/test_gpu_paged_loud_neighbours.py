"""GPU parity: keys and values of very different sizes beside each other in an 8-bit cache, in both kernels.
What a row does not see, or gives no weight, must not change what it sees of others."""

import numpy as np
import pytest
import torch

import speculative_decoding_verify_bf16_gb300 as sv
from paged_floors import check_lane
from paged_harness import DEV, Lanes, attend

pytestmark = pytest.mark.gpu
KINDS = ["e4m3", "int8"]
# Few rows; tiles: 24 rows of a head in one lane, prompts' parts.
LENS = [([3], [130]), ([12], [150]), ([200], [40]), ([150, 7], [33, 700])]


@pytest.fixture(scope="module", autouse=True)
def _built():
    sv.build_library()
    sv.load_library()


def tokens(L, n):
    return torch.randn(n, L.kv, L.d, generator=L.g, device=DEV)


def run(L, q, window=0, scale=None, workspace=None):
    out, lse, status = attend(L, q, window, scale, workspace)
    torch.cuda.synchronize()
    assert status.tolist() == [0] * len(L.lens)
    for b, n in enumerate(L.lens):
        # (tiles: one exponent for 32 positions, at most 7 above a position's own)
        check_lane(L, b, q, out, lse, window, scale, floor=2.0 ** -25 if max(L.lens) > 4 else 2.0 ** -32)
    return out


def fill(L, name, b, x, first=0):
    stored = L.put(name, b, first, x)
    getattr(L, name)[b][first:first + x.shape[0]] = stored


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("up", [8, 16, 26, 45])
@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("lens,before", LENS)
def test_a_loud_last_column(kind, d, up, what, lens, before):
    """The last column's key or value is 2^up times the others': earlier columns, in its group of
    positions too, do not see it."""
    L = Lanes(lens, before, kind=kind, d=d, seed=up)
    for b, n in enumerate(lens):
        fill(L, what, b, tokens(L, 1) * 2.0 ** up, before[b] + n - 1)
    run(L, L.queries(4))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("up", [8, 26, 40])
@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("lens,before", LENS)
def test_loud_values_without_weight(kind, up, window, lens, before):
    """Every 13th position's value is loud, its score 200 below the others'."""
    L = Lanes(lens, before, kind=kind, seed=up + 1)
    for b, n in enumerate(len(x) for x in L.k):
        k, v = tokens(L, n), tokens(L, n)
        k[..., 0] = 0.0
        k[::13] = 0.0
        k[::13, :, 0] = -20.0
        v[::13] *= 2.0 ** up
        fill(L, "k", b, k), fill(L, "v", b, v)
    q = L.queries(4)
    q[..., 0] = 10.0
    run(L, q, window, scale=1.0 if up == 8 else None)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("lens,before", LENS)
def test_values_of_all_sizes(kind, window, lens, before):
    """Each token has sizes of its own, 2^-40 to 2^40, some are zero."""
    L = Lanes(lens, before, kind=kind, seed=3)
    for b, n in enumerate(len(x) for x in L.k):
        e = torch.randint(-40, 41, (n, L.kv, 1), generator=L.g, device=DEV).float()
        fill(L, "v", b, tokens(L, n) * torch.exp2(e) * (e % 5 != 0))
        e = torch.randint(-45, 1, (n, L.kv, 1), generator=L.g, device=DEV).float()
        fill(L, "k", b, tokens(L, n) * torch.exp2(e) * (e % 5 != 0))
    run(L, L.queries(4), window)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("step", [6, 7, 8, 9, 14, 15, 16, 17])
@pytest.mark.parametrize("lens,before", LENS)
def test_at_the_border_of_what_one_exponent_serves(kind, step, lens, before):
    """Two sizes by turns, 2^step apart."""
    L = Lanes(lens, before, kind=kind, seed=step)
    for b, n in enumerate(len(x) for x in L.k):
        up = torch.where(torch.arange(n, device=DEV) % 3 == 0, 2.0 ** step, 1.0)[:, None, None]
        fill(L, "v", b, tokens(L, n) * up)
        fill(L, "k", b, tokens(L, n) * up * 2.0 ** -step)
    run(L, L.queries(4))


@pytest.mark.parametrize("kind", KINDS)
def test_long_contexts_split_and_whole(kind):
    L = Lanes([150, 2], [9000, 20000], kind=kind, kv=1, d=64, seed=5)
    for b, n in enumerate(len(x) for x in L.k):
        loud = torch.where(torch.rand(n, generator=L.g, device=DEV) < 0.002, 2.0 ** 30, 1.0)[:, None, None]
        k = tokens(L, n) * 0.5
        k[..., 0] = torch.where(loud[..., 0] > 1, -40.0, 0.0)
        fill(L, "k", b, k), fill(L, "v", b, tokens(L, n) * loud + 1.0)
    q = L.queries(2)
    q[..., 0] = 10.0
    for workspace in (None, torch.empty(0, dtype=torch.uint8, device=DEV)):
        out, lse, status = attend(L, q, workspace=workspace, scale=1.0)
        torch.cuda.synchronize()
        assert status.tolist() == [0, 0]
        for i, rows in ((0, slice(0, 3)), (1, slice(150, 152))):  # (the oracle takes a second a column)
            M = Lanes([rows.stop - rows.start], [L.before[i]], kind=kind, kv=1, d=64, seed=6)
            n = L.before[i] + rows.stop - rows.start
            M.host_tables, M.cache, M.k, M.v = L.host_tables[i:i + 1], L.cache, [L.k[i][:n]], [L.v[i][:n]]
            check_lane(M, 0, q[rows], out[rows], lse[rows], scale=1.0, floor=2.0 ** -25)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens,before", LENS)
@pytest.mark.parametrize("what", ["k", "v"])
def test_numbers_that_are_not_finite_among_them(kind, lens, before, what):
    L = Lanes(lens + [4], before + [60], kind=kind, seed=7)
    fill(L, what, 0, tokens(L, 1) * 2.0 ** 30, 21)
    fill(L, what, 0, tokens(L, 1) * np.nan, 22)
    fill(L, "v", len(lens), tokens(L, 1) * 2.0 ** 30, 62)
    q = L.queries(4)
    out, lse, status = attend(L, q)
    torch.cuda.synchronize()
    assert status.tolist() == [sv.SPEC_ERR_NONFINITE] + [0] * len(lens)
    check_lane(L, len(lens), q, out, lse, floor=2.0 ** -25)
