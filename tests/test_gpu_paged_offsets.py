"""GPU: rows into slots and back where some lanes' offsets are wrong.  A lane whose own offsets hold is dealt
with, wherever the others' stand."""

import numpy as np
import pytest
import torch

import speculative_decoding_verify_bf16_gb300 as sv
from oracle import paged
from paged_harness import DEV, Lanes, i32

pytestmark = pytest.mark.gpu
LAY = sv.SPEC_ERR_LAYOUT


@pytest.fixture(scope="module", autouse=True)
def _built():
    sv.build_library()
    sv.load_library()


def pools(L):
    return [t.float().cpu().numpy() for t in L.cache if t is not None]


def run(offsets, rows, max_len, kind, seed=0):
    """Writes and reads with these offsets; what each lane's offsets say is what has to happen."""
    lanes = len(offsets) - 1
    ok = [0 <= a <= b <= rows and b - a <= max_len for a, b in zip(offsets, offsets[1:])]
    rng = np.random.default_rng(seed)
    L = Lanes([max_len] * lanes, rng.integers(0, 40, lanes).tolist(), kind=kind, kv=2, d=64, page=8, seed=seed)
    L.offsets = torch.tensor(np.array(offsets, np.int64).astype(np.int32), device=DEV)
    k, v = (torch.randn(rows, 2, 64, generator=L.g, device=DEV).to(torch.bfloat16) for _ in range(2))
    status = torch.zeros(lanes, dtype=torch.int32, device=DEV)
    before = pools(L)
    sv.spec_cache_write(*L.where(), k, v, max_len, lane_status=status)
    torch.cuda.synchronize()
    assert status.tolist() == [0 if good else LAY for good in ok]
    after = pools(L)
    touched = np.zeros(L.cache.k.shape[:2], bool)
    held = {}
    for b in range(lanes):
        if not ok[b]:
            continue
        a, n = offsets[b], offsets[b + 1] - offsets[b]
        page, slot = paged.lane_slots(L.host_tables[b], L.page, L.before[b], n)
        touched[page, slot] = True
        for name, x, pool, i in (("k", k, after[0], 2), ("v", v, after[1], 3)):
            want = x[a:a + n].double().cpu().numpy()
            got = pool[page, slot]
            if kind != "bf16":
                y, byte = paged.quantise(want, kind)
                assert np.array_equal(got, y) and np.array_equal(after[i][page, slot], byte), (b, name)
                want = paged.values(y, byte)
            else:
                assert np.array_equal(got, want), (b, name)
            held[b, name] = want
    for x, y in zip(before, after):
        assert np.array_equal(x[~touched], y[~touched], equal_nan=True)
    rk, rv = (torch.full((rows, 2, 64), 7.0, device=DEV) for _ in range(2))
    status.zero_()
    sv.spec_cache_read(*L.where(), rk, rv, max_len, lane_status=status)
    torch.cuda.synchronize()
    assert status.tolist() == [0 if good else LAY for good in ok]
    owners = np.zeros(rows, int)
    for b in range(lanes):
        if ok[b]:
            owners[offsets[b]:offsets[b + 1]] += 1
    for name, got in (("k", rk), ("v", rv)):
        got = got.double().cpu().numpy()
        assert (got[owners == 0] == 7).all()
        for b in range(lanes):
            if ok[b]:
                rows_b = np.arange(offsets[b], offsets[b + 1])
                alone = owners[rows_b] == 1  # (a row of two lanes holds the one's token or the other's)
                assert np.array_equal(got[rows_b[alone]], held[b, name][alone]), (b, name)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("offsets", [[0, 5, 3, 8], [0, 100, 3, 8], [-1, 2, 4, 8], [0, 2, -7, 3, 8], [0, 2 ** 31 - 1, 0, 8], [8, 0, 8], [3, 8, 0, 3],
                                     [-2 ** 31, 2, 2 ** 31 - 1, 1, 6], [0, 3, 3, 2, 6, 6]])
def test_lanes_beside_wrong_offsets(kind, offsets):
    run(offsets, 8, 8, kind)


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("lanes", [40, 127, 128, 129, 500])
@pytest.mark.parametrize("wrong", [1, 5, 30])
def test_many_lanes(kind, lanes, wrong):
    rng = np.random.default_rng(lanes + wrong)
    offsets = np.cumsum(rng.integers(0, 9, lanes + 1))
    offsets -= offsets[0]
    rows = int(offsets[-1])
    at = rng.choice(lanes + 1, wrong, replace=False)
    offsets[at] = rng.choice([-1, -2 ** 31, 2 ** 31 - 1, rows + 1, 0, rows // 2], wrong)
    run([int(x) for x in offsets], rows, 8, kind, seed=wrong)
