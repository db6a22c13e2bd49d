"""GPU: rows into the slots of a paged cache and back, bit for bit what the oracle says."""

import numpy as np
import pytest
import torch

import speculative_decoding_verify_bf16_gb300 as sv
from oracle import paged
from paged_harness import DEV, TYPES, Lanes, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    sv.build_library()
    sv.load_library()


def raw(t):
    return None if t is None else t.view(torch.uint8).clone()


def write(L, k, v, status=None):
    status = torch.zeros(len(L.lens), dtype=torch.int32, device=DEV) if status is None else status
    sv.spec_cache_write(*L.where(), k, v, L.max_len, lane_status=status)
    torch.cuda.synchronize()
    return status.tolist()


def read(L, dtype, rows=None):
    rows = sum(L.lens) if rows is None else rows
    k, v = (torch.full((rows, L.kv, L.d), 7.0, dtype=dtype, device=DEV) for _ in range(2))
    status = torch.zeros(len(L.lens), dtype=torch.int32, device=DEV)
    sv.spec_cache_read(*L.where(), k, v, L.max_len, lane_status=status)
    torch.cuda.synchronize()
    return k, v, status.tolist()


def expect(L, before, k, v):
    """The pools' bytes after the write, from those before it: only the rows' slots change."""
    want = [None if t is None else t.cpu().numpy().copy() for t in before]
    row = 0
    for b, n in enumerate(L.lens):
        page, slot = paged.lane_slots(L.host_tables[b], L.page, L.before[b], n)
        for j, x in enumerate((k, v)):
            part = x[row:row + n]
            if L.kind == "bf16":
                bits = part.to(torch.bfloat16).contiguous().view(torch.uint8).cpu().numpy()
                want[j][page, slot] = bits
            else:
                y, byte = paged.quantise(part.double().cpu().numpy(), L.kind)
                if L.kind == "int8":
                    bits = y.astype(np.int8).view(np.uint8)
                else:
                    table = paged.e4m3_values()
                    code = np.array([np.flatnonzero(table[:127] == m)[0] for m in np.abs(y).ravel()], np.uint8).reshape(y.shape)
                    bits = code | (np.signbit(y).astype(np.uint8) << 7)
                want[j][page, slot] = bits
                want[2 + j][page, slot] = byte.astype(np.uint8)
        row += n
    return want


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,kv,page,layout", [(128, 2, 16, "slots"), (64, 1, 24, "heads"), (16, 3, 1, "slots"), (256, 2, 7, "joined"),
                                              (80, 5, 64, "heads"), (144, 1, 100, "slots"), (128, 8, 16, "joined")])
def test_slots_and_back(kind, dtype, d, kv, page, layout):
    L = Lanes([1, 0, 5, 37, 2], [0, 9, 15, 100, 63], kind=kind, d=d, kv=kv, page=page, layout=layout, seed=d + page)
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    k, v = ((torch.randn(45, kv, d, generator=g, device=DEV) * torch.exp2(
        torch.randint(-20, 20, (45, kv, 1), generator=g, device=DEV).float())).to(dtype) for _ in range(2))
    k[3], v[7, 0] = 0.0, -0.0
    before = [raw(t) for t in L.cache]
    want = expect(L, before, k, v)
    assert write(L, k, v) == [0] * 5
    for t, w in zip(L.cache, want):
        if t is not None:
            assert np.array_equal(t.view(torch.uint8).cpu().numpy(), w)
    for out in (torch.bfloat16, torch.float32):
        rk, rv, status = read(L, out)
        assert status == [0] * 5
        for got, x in ((rk, k), (rv, v)):
            held = x.to(torch.bfloat16).double().cpu().numpy() if kind == "bf16" else \
                paged.values(*paged.quantise(x.double().cpu().numpy(), kind))
            assert np.array_equal(got.double().cpu().numpy(), held)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_roundings_and_borders(kind):
    """Every e4m3 number and the halves between them, ties, and largest numbers on both
    sides of a power of two's border."""
    top = paged.TOP[kind]
    d, rows = 128, []
    grid = paged.e4m3_values()[:127]
    pts = np.concatenate([grid, (grid[1:] + grid[:-1]) / 2, np.arange(0, 127.5, 0.5)])
    pts = np.concatenate([pts, np.nextafter(pts.astype(np.float32), np.float32(1e9)), np.nextafter(pts.astype(np.float32), np.float32(-1))])
    pts = pts[np.abs(pts) <= top]
    for i in range(0, len(pts), d - 1):
        x = np.zeros(d)
        part = pts[i:i + d - 1]
        x[1:1 + len(part)] = part * np.where(np.arange(len(part)) % 2, -1, 1)
        x[0] = top
        rows.append(x)
    for e in (-60, -48, -47, -10, -1, 0, 3, 47, 48):
        for m in (top, np.nextafter(np.float32(top), np.float32(1e9)), np.nextafter(np.float32(top), np.float32(0)), top * 0.75, 1.0):
            if m * 2.0 ** e <= top * 2.0 ** 48:
                x = np.zeros(d)
                x[5], x[6], x[7] = m * 2.0 ** e, -m * 2.0 ** e / 3, m * 2.0 ** e / 1000
                rows.append(x)
    k = torch.tensor(np.array(rows), device=DEV).float()[:, None].contiguous()
    L = Lanes([len(rows)], [3], kind=kind, kv=1, d=d, seed=2)
    assert write(L, k, -k) == [0]
    rk, rv, _ = read(L, torch.float32)
    want = paged.values(*paged.quantise(k.double().cpu().numpy(), kind))
    assert np.array_equal(rk.double().cpu().numpy(), want) and np.array_equal(rv.double().cpu().numpy(), -want)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf"), 3.4e38, -2.0 ** 58])
def test_numbers_that_it_cannot_hold(kind, bad):
    for which in range(2):
        L = Lanes([2, 3, 1], [4, 30, 0], kind=kind, seed=3)
        kv = [torch.randn(6, L.kv, L.d, device=DEV) for _ in range(2)]
        kv[which][3, 1, 77] = bad
        held = kind == "bf16" and abs(bad) == 2.0 ** 58
        assert write(L, *kv) == [0, 0 if held else sv.SPEC_ERR_NONFINITE, 0]
        got = read(L, torch.float32)
        assert got[2] == [0, 0, 0]
        if kind != "bf16":  # the whole head reads back as NaN, and nothing else
            for b in (0, 2):
                rows = slice(0, 2) if b == 0 else slice(5, 6)
                assert torch.isfinite(got[0][rows]).all() and torch.isfinite(got[1][rows]).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
def test_failed_lanes_leave_the_others_alone(kind):
    n = 3
    L = Lanes([n] * 8, [40, 50, 60, 70, 80, 90, 30, 16], kind=kind, seed=4)
    k, v = (torch.randn(8 * n, L.kv, L.d, device=DEV) for _ in range(2))
    good = L.host_tables.copy()
    bad = good.copy()
    bad[1, 50 // 16] = L.cache.k.shape[0]
    bad[2, 60 // 16] = -1
    L.tables = torch.tensor(bad, device=DEV)
    L.cached[3] = -1
    L.cached[4] = L.tables.shape[1] * L.page - n + 1
    L.cached[5] = 2 ** 31 - 1
    status = torch.zeros(8, dtype=torch.int32, device=DEV)
    status[6] = sv.SPEC_ERR_TIMEOUT
    before = [raw(t) for t in L.cache]
    lay = sv.SPEC_ERR_LAYOUT
    assert write(L, k, v, status) == [0, lay, lay, lay, lay, lay, sv.SPEC_ERR_TIMEOUT, 0]
    kept = L.lens
    want = expect(L, before, k, v)
    for b in (0, 7):  # written; what the failed lanes own is theirs
        page, slot = paged.lane_slots(good[b], L.page, L.before[b], n)
        for t, w in zip(L.cache, want):
            if t is not None:
                assert np.array_equal(t.view(torch.uint8).cpu().numpy()[page, slot], w[page, slot])
    for b in (3, 4, 5, 6):  # not touched at all
        page, slot = paged.lane_slots(good[b], L.page, 0, L.before[b] + n)
        for t, w in zip(L.cache, before):
            if t is not None:
                assert np.array_equal(t.view(torch.uint8).cpu().numpy()[page, slot], w.cpu().numpy()[page, slot])
    assert kept == [n] * 8


def test_bad_offsets_and_rows_behind_the_last_lane():
    L = Lanes([2, 2, 2, 2], [4, 30, 0, 16], seed=5)
    k, v = (torch.randn(12, L.kv, L.d, device=DEV) for _ in range(2))
    L.offsets = i32([0, 2, 1, 6, 13])  # lane 1 descends, 2 is too long, 3 leaves the rows
    lay = sv.SPEC_ERR_LAYOUT
    assert write(L, k, v) == [0, lay, lay, lay]
    L = Lanes([2, 1], [4, 30], seed=5)
    rk, rv, status = read(L, torch.float32, rows=6)
    assert status == [0, 0] and (rk[3:] == 7).all() and (rv[3:] == 7).all()
    L = Lanes([0], [4], seed=5)
    assert write(L, k[:0], v[:0]) == [0]


def test_strided_rows():
    L = Lanes([4, 2], [4, 30], kind="e4m3", kv=4, d=64, seed=6)
    fused = torch.randn(6, 4 + 2 * 4, 64, device=DEV).to(torch.bfloat16)
    k, v = fused[:, 4:8], fused[:, 8:]
    assert write(L, k, v) == [0, 0]
    back = torch.full((6, 4, 3 * 64), 7.0, dtype=torch.bfloat16, device=DEV)
    status = torch.zeros(2, dtype=torch.int32, device=DEV)
    sv.spec_cache_read(*L.where(), back[..., :64], back[..., 128:], 4, lane_status=status)
    torch.cuda.synchronize()
    for got, x in ((back[..., :64], k), (back[..., 128:], v)):
        assert np.array_equal(got.double().cpu().numpy(), paged.values(*paged.quantise(x.double().cpu().numpy(), "e4m3")))
    assert (back[..., 64:128] == 7).all()


def test_many_rows_and_lanes():
    rng = np.random.default_rng(7)
    lens = rng.integers(0, 60, 400).tolist()
    L = Lanes(lens, rng.integers(0, 50, 400).tolist(), kind="int8", kv=2, d=64, page=24, seed=7)
    k, v = (torch.randn(sum(lens), 2, 64, device=DEV).to(torch.bfloat16) for _ in range(2))
    assert write(L, k, v) == [0] * 400
    rk, rv, _ = read(L, torch.bfloat16)
    for got, x in ((rk, k), (rv, v)):
        assert np.array_equal(got.double().cpu().numpy(), paged.values(*paged.quantise(x.double().cpu().numpy(), "int8")))


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
def test_new_cache(kind):
    c = sv.new_paged_cache(5, 16, 2, 64, TYPES[kind], DEV)
    assert c.k.shape == c.v.shape == (5, 16, 2, 64) and c.k.dtype == TYPES[kind]
    assert not c.k.view(torch.uint8).any() and not c.v.view(torch.uint8).any()
    assert (c.k_exps is None) == (kind == "bf16")
    with pytest.raises(ValueError):
        sv.new_paged_cache(5, 16, 2, 64, torch.float16, DEV)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
def test_captured_write_and_read(kind):
    L = Lanes([2, 3], [4, 30], kind=kind, seed=8)
    k, v = (torch.randn(5, L.kv, L.d, device=DEV) for _ in range(2))
    rk, rv = torch.empty_like(k), torch.empty_like(v)
    status = torch.zeros(2, dtype=torch.int32, device=DEV)

    def both():
        sv.spec_cache_write(*L.where(), k, v, L.max_len, lane_status=status)
        sv.spec_cache_read(*L.where(), rk, rv, L.max_len, lane_status=status)

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for i in range(3):
        k.normal_(), v.normal_()
        L.cached.copy_(i32([i, 33 - i]))
        graph.replay()
        torch.cuda.synchronize()
        assert status.tolist() == [0, 0]
        for got, x in ((rk, k), (rv, v)):
            held = x.to(torch.bfloat16).double().cpu().numpy() if kind == "bf16" else \
                paged.values(*paged.quantise(x.double().cpu().numpy(), kind))
            assert np.array_equal(got.double().cpu().numpy(), held)
