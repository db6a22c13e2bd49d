"""GPU parity: attention over a paged cache against the float64 oracle (bounds in paged_harness)."""

import numpy as np
import pytest
import torch

import speculative_decoding_verify_bf16_gb300 as sv
from paged_harness import DEV, Lanes, attend, check, check_lane, i32, offsets_of

pytestmark = pytest.mark.gpu
KINDS = ["bf16", "e4m3", "int8"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    sv.build_library()
    sv.load_library()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("before", [0, 1, 14, 15, 16, 31, 63, 126, 127, 128, 254, 255, 256, 1000, 5000])
def test_one_token(kind, before):
    check([1], [before], kind=kind, seed=before)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [16, 48, 64, 80, 112, 128, 144, 240, 256])
def test_head_sizes(kind, d):
    check([1, 3], [200, 77], kind=kind, d=d, seed=d)
    check([2, 16, 0, 9], [200, 0, 5, 700], hq=6, kind=kind, d=d, seed=d + 1)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hq,kv", [(1, 1), (2, 2), (3, 1), (14, 2), (16, 1), (8, 8), (32, 4), (48, 1), (130, 1)])
def test_head_layouts(kind, hq, kv):
    check([1, 4], [130, 300], hq=hq, kv=kv, kind=kind, seed=hq)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows", [7, 8, 9, 12, 15, 16, 17, 24, 25, 31, 32, 33, 64, 65])
def test_rows_of_a_head(kind, d, rows):
    """Every number of rows that a kernel's blocks of 8, 16, 32 and 128 end at or beside."""
    check([1], [150], hq=rows, kv=1, d=d, kind=kind, seed=rows)
    check([rows], [40], hq=1, kv=1, d=d, kind=kind, seed=rows + 1)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [1, 3, 16, 24, 100, 128, 1000])
def test_page_sizes(kind, page):
    check([2, 5, 1], [300, 0, 999], page=page, kind=kind, seed=page)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("layout", ["slots", "heads", "joined"])
def test_cache_layouts(kind, layout):
    check([2, 5], [300, 40], layout=layout, kind=kind, kv=3, hq=6, seed=4)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window", [1, 2, 17, 128, 400, 100000])
def test_windows(kind, window):
    check([1, 8, 3], [900, 130, 0], window=window, kind=kind, seed=window % 1000)
    check([300], [500], window=window, kind=kind, kv=1, hq=2, seed=window % 999)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens", [[8] * 5, [0, 7, 0, 1, 16], [33, 2, 64], [129, 1], [1] * 40])
def test_columns(kind, lens):
    rng = np.random.default_rng(len(lens))
    check(lens, rng.integers(0, 600, len(lens)).tolist(), hq=8, kind=kind, seed=len(lens))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [48, 64, 128])
@pytest.mark.parametrize("window,whole", [(0, False), (50, False), (0, True)])
def test_rounds_of_many_lanes(kind, d, window, whole):
    """17 to 32 rows of a head and many lanes (few of them take the tiles), split and whole."""
    rng = np.random.default_rng(d)
    lens = rng.integers(0, 5, 44).tolist()
    before = rng.integers(0, 700, 44).tolist()
    workspace = torch.empty(0, dtype=torch.uint8, device=DEV) if whole else None
    check(lens, before, hq=8, kv=1, d=d, kind=kind, page=24, window=window, workspace=workspace, seed=d)
    check([4], [900], hq=8, kv=1, d=d, kind=kind, scale=-0.1, window=window, workspace=workspace, seed=d + 1)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,before,d", [(255, 0, 128), (256, 1, 64), (257, 300, 128), (700, 130, 96), (512, 1500, 128), (300, 10, 256)])
def test_prompts(kind, n, before, d):
    check([n], [before], hq=2, kv=1, d=d, kind=kind, seed=n)


@pytest.mark.parametrize("kind", KINDS)
def test_ragged_prompts(kind):
    check([130, 0, 1, 400, 17, 64], [0, 50, 700, 33, 128, 1000], hq=8, kv=2, kind=kind, page=24, seed=3)


def test_more_lanes_than_threads():
    rng = np.random.default_rng(1)
    lens = rng.integers(0, 3, 700)
    check(lens.tolist(), rng.integers(0, 40, 700).tolist(), hq=2, kv=1, d=64, kind="int8", seed=5)


@pytest.mark.parametrize("kind", KINDS)
def test_long_context_is_split_and_whole(kind):
    """With and without scratch memory for the parts, and with too little of it."""
    for workspace in (None, torch.empty(0, dtype=torch.uint8, device=DEV), torch.empty(4096, dtype=torch.uint8, device=DEV)):
        check([2, 1], [30000, 7000], kind=kind, kv=2, hq=8, workspace=workspace, seed=9)


@pytest.mark.parametrize("kind", KINDS)
def test_peaked_and_large_scores(kind):
    check([4], [800], q_scale=20.0, kind=kind, seed=1)
    check([4], [800], scale=0.0, kind=kind, seed=2)
    check([4], [800], scale=-0.2, kind=kind, seed=3)
    check([4], [800], q_scale=1e-30, kind=kind, seed=4)
    check([4], [800], q_scale=1e30, scale=1e-31, kind=kind, seed=5)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_values_of_very_different_sizes(kind):
    """Exponents at both ends of the range beside each other, and heads of zeros."""
    L = Lanes([3], [500], kind=kind, seed=11)
    x = torch.randn(40, L.kv, L.d, device=DEV).to(torch.bfloat16)
    L.v[0][100:140] = L.put("v", 0, 100, x * 2.0 ** 20)
    L.v[0][200:240] = L.put("v", 0, 200, x * 2.0 ** -35)
    L.v[0][300:340] = L.put("v", 0, 300, x * 0.0)
    L.k[0][400:440] = L.put("k", 0, 400, x * 0.0)
    q = L.queries(4)
    out, lse, status = attend(L, q)
    torch.cuda.synchronize()
    assert status.tolist() == [0]
    check_lane(L, 0, q, out, lse)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [1, 5, 200])
def test_strided_queries_and_outputs(kind, n):
    L = Lanes([n, 2], [100, 300], kind=kind, seed=12)
    wide = torch.randn(n + 2, 8, 3 * L.d, device=DEV).to(torch.bfloat16)
    q = wide[:, 1::2, L.d:2 * L.d]
    back = torch.full((n + 5, 4, L.d + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    wide_lse = torch.full((n + 2, 9), 7.0, device=DEV)
    status = torch.zeros(2, dtype=torch.int32, device=DEV)
    sv.spec_paged_attention(q, *L.where(), back[:n + 2, :, :L.d], L.max_len, lse=wide_lse[:, :4], lane_status=status)
    torch.cuda.synchronize()
    assert status.tolist() == [0, 0]
    for b in range(2):
        check_lane(L, b, q, back[:, :, :L.d], wide_lse[:, :4])
    assert (back[n + 2:] == 7).all() and (back[:, :, L.d:] == 7).all() and (wide_lse[:, 4:] == 7).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [2, 150])
def test_rows_behind_the_last_lane_stay(kind, n):
    L = Lanes([n, 1], [20, 40], kind=kind, seed=13)
    q = torch.cat([L.queries(4), torch.full((6, 4, L.d), float("nan"), dtype=torch.bfloat16, device=DEV)])
    out, lse, status = attend(L, q)
    torch.cuda.synchronize()
    assert status.tolist() == [0, 0] and (out[n + 1:] == 7).all() and (lse[n + 1:] == 7).all()
    for b in range(2):
        check_lane(L, b, q, out, lse)


@pytest.mark.parametrize("n", [1, 300])
def test_lanes_that_share_a_prefix(n):
    """Two lanes' tables name the same pages for their first tokens."""
    L = Lanes([n, n], [64, 64], seed=14)
    L.host_tables[1, :4] = L.host_tables[0, :4]
    L.tables = torch.tensor(L.host_tables, device=DEV)
    L.k[1][:64], L.v[1][:64] = L.k[0][:64], L.v[0][:64]
    q = L.queries(4)
    out, lse, status = attend(L, q)
    torch.cuda.synchronize()
    assert status.tolist() == [0, 0]
    for b in range(2):
        check_lane(L, b, q, out, lse)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [3, 200])
def test_failed_lanes_leave_the_others_alone(kind, n):
    """Layouts that do not hold, and pages that are none: each lane reports its own."""
    lens, before = [n] * 9, [40, 50, 60, 70, 80, 90, 30, 20, 10]
    L = Lanes(lens, before, kind=kind, seed=15)
    q = L.queries(4)
    L.host_tables[1, 1] = L.cache.k.shape[0]
    L.host_tables[2, 2] = -1
    L.tables = torch.tensor(L.host_tables, device=DEV)
    L.cached[3] = -1
    L.cached[4] = L.tables.shape[1] * L.page - n + 1
    L.cached[5] = 2 ** 31 - 1
    status = torch.zeros(9, dtype=torch.int32, device=DEV)
    status[6] = sv.SPEC_ERR_TOKEN_RANGE
    out, lse, status = attend(L, q, status=status)
    torch.cuda.synchronize()
    lay = sv.SPEC_ERR_LAYOUT
    assert status.tolist() == [0, lay, lay, lay, lay, lay, sv.SPEC_ERR_TOKEN_RANGE, 0, 0]
    for b in (0, 7, 8):
        check_lane(L, b, q, out, lse)


@pytest.mark.parametrize("n", [2, 140])
def test_bad_offsets(n):
    lens = [n, n, n, n]
    L = Lanes(lens, [10] * 4, seed=16)
    q = L.queries(4)
    L.offsets = i32([0, n, n - 1, 3 * n, 4 * n + 1])  # lane 1 descends, 2 is too long, 3 leaves the rows
    out, lse, status = attend(L, q)
    torch.cuda.synchronize()
    lay = sv.SPEC_ERR_LAYOUT
    assert status.tolist() == [0, lay, lay, lay]
    check_lane(L, 0, q, out, lse)


def test_max_context_bounds_the_lanes():
    L = Lanes([2, 2], [100, 50], seed=17)
    q = L.queries(4)
    out, lse, status = attend(L, q, max_context=60)
    torch.cuda.synchronize()
    assert status.tolist() == [sv.SPEC_ERR_LAYOUT, 0]
    check_lane(L, 1, q, out, lse)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [2, 150])
@pytest.mark.parametrize("what", ["q", "k", "v"])
def test_numbers_that_are_not_finite(kind, n, what):
    L = Lanes([n, n], [90, 33], kind=kind, seed=18)
    q = L.queries(4)
    if what == "q":
        q[1, 2, 5] = float("inf")
    else:
        L.put(what, 0, 17, torch.full((1, L.kv, L.d), float("nan"), dtype=torch.bfloat16, device=DEV))
    out, lse, status = attend(L, q)
    torch.cuda.synchronize()
    assert status.tolist() == [sv.SPEC_ERR_NONFINITE, 0]
    check_lane(L, 1, q, out, lse)


@pytest.mark.parametrize("n", [1, 200])
def test_no_status_and_no_lse(n):
    L = Lanes([n], [70], seed=19)
    q = L.queries(4)
    out = torch.zeros_like(q)
    sv.spec_paged_attention(q, *L.where(), out, n)
    torch.cuda.synchronize()
    check_lane(L, 0, q, out, None)


def test_nothing_to_do():
    L = Lanes([0, 0], [5, 0], seed=20)
    q = torch.zeros(0, 4, L.d, dtype=torch.bfloat16, device=DEV)
    out, _, status = attend(L, q, lse=False)
    torch.cuda.synchronize()
    assert status.tolist() == [0, 0]
    L = Lanes([], [], seed=20)
    attend(L, torch.zeros(3, 4, L.d, dtype=torch.bfloat16, device=DEV), lse=False)
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind", KINDS)
def test_pages_behind_four_gigabytes(kind):
    """Offsets of slots that pass 32 bits, in elements and in bytes."""
    d, kv, page = 128, 2, 16
    size = 2 if kind == "bf16" else 1
    pages = (2 ** 32 + 2 ** 27) // (page * kv * d) + 40
    L = Lanes([2], [70], kind=kind, kv=kv, d=d, page=page, seed=21)
    k = torch.empty(pages * page * kv * d * size, dtype=torch.uint8, device=DEV).view(L.cache.k.dtype).view(pages, page, kv, d)
    v = torch.empty_like(k)
    exps = [None, None]
    if kind != "bf16":
        exps = [torch.empty(pages, page, kv, dtype=torch.uint8, device=DEV) for _ in range(2)]
    far = pages - L.cache.k.shape[0]
    for new, old in zip((k, v, *exps), L.cache):
        if new is not None:
            new.view(torch.uint8)[far:] = old.view(torch.uint8)
    L.cache = sv.PagedCache(k, v, *exps)
    L.tables += far
    q = L.queries(4)
    out, lse, status = attend(L, q)
    torch.cuda.synchronize()
    assert status.tolist() == [0]
    check_lane(L, 0, q, out, lse)


@pytest.mark.parametrize("n", [1, 6, 150])
def test_captured_and_replayed_as_lanes_grow(n):
    """One captured launch serves rounds of other lengths; lengths are read on the device."""
    L = Lanes([n, n], [3000, 400], kind="e4m3", seed=22)
    q = L.queries(8)
    ws = sv.new_paged_attention_workspace(8, L.kv, L.d, n, DEV)
    attend(L, q, workspace=ws)
    torch.cuda.synchronize()
    out, lse, status = torch.empty_like(q), torch.empty(2 * n, 8, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.spec_paged_attention(q, *L.where(), out, n, lse=lse, lane_status=status, workspace=ws)
    for before in ([3000, 400], [0, 1], [129, 395], [2000, 0]):  # (within the lanes' pages)
        L.cached.copy_(i32(before))
        out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert status.tolist() == [0, 0]
        M = Lanes([n, n], before, kind="e4m3", seed=22)
        M.k = [a[:c + n] for a, c in zip(L.k, before)]
        M.v = [a[:c + n] for a, c in zip(L.v, before)]
        for b in range(2):
            check_lane(M, b, q, out, lse)


def test_streams_and_results_that_do_not_vary():
    """Calls on two streams at once, each with scratch memory of its own, give the same bits as
    calls after one another."""
    jobs = []
    for s in range(2):
        L = Lanes([3, 2, 1], [9000, 40, 2500], kind=KINDS[s], seed=23 + s)
        jobs.append((L, L.queries(8), sv.new_paged_attention_workspace(8, L.kv, L.d, 3, DEV), torch.cuda.Stream()))
    want = [attend(L, q, workspace=ws)[:2] for L, q, ws, _ in jobs]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [attend(L, q, workspace=ws, stream=st)[:2] for L, q, ws, st in jobs]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


def test_scratch_memory_is_kept_to():
    for n, hq, kv, d in ((1, 8, 2, 128), (4, 8, 1, 64), (300, 4, 2, 128), (9, 4, 2, 256)):
        L = Lanes([n], [20000], kv=kv, d=d, seed=25)
        q = L.queries(hq)
        size = sv.spec_paged_attention_workspace(hq, kv, d, n)
        assert size > 0
        want = None
        for have in (size, size - 16, 0, size + 4096):
            buf = torch.full((have + 8192,), 171, dtype=torch.uint8, device=DEV)
            out, lse, status = attend(L, q, workspace=buf[:have])
            torch.cuda.synchronize()
            assert status.tolist() == [0] and (buf[have:] == 171).all()
            if want is None:
                check_lane(L, 0, q, out, lse)
                want = out.double()
            assert (out.double() - want).abs().max() <= 2.0 ** -6 * want.abs().max()
    with pytest.raises(sv.SpecError):
        attend(L, q, workspace=torch.empty(1 << 20, dtype=torch.uint8, device=DEV)[4:])


def test_a_buffer_for_more_columns_serves_fewer():
    ws = sv.new_paged_attention_workspace(8, 2, 128, 600, DEV)
    for n in (1, 3, 8, 100, 600):
        check([n], [3000], hq=8, kv=2, workspace=ws, seed=n)


def test_scratch_memory_grows_with_the_columns():
    for hq, kv, d in ((8, 2, 128), (32, 8, 128), (16, 1, 64), (8, 8, 256), (24, 3, 96)):
        sizes = [sv.spec_paged_attention_workspace(hq, kv, d, n) for n in (1, 2, 3, 4, 8, 9, 16, 33, 64, 600, 5000)]
        assert sizes == sorted(sizes) and sizes[0] > 0


@pytest.mark.parametrize("n", [1, 3])
def test_strides_of_dimensions_of_one_are_free(n):
    """One head, one row, one slot a page: their strides are never used, whatever they are."""
    L = Lanes([n], [20], kv=1, d=64, page=1, seed=26)
    odd = lambda t, strides: torch.as_strided(t, t.shape, strides)
    L.cache = sv.PagedCache(odd(L.cache.k, (64, 7, 3, 1)), odd(L.cache.v, (64, 7, 3, 1)))
    q = odd(L.queries(1), (5 if n == 1 else 64, 3, 1))
    out, lse, status = attend(L, q, out=odd(torch.zeros(n, 1, 64, dtype=torch.bfloat16, device=DEV), (5 if n == 1 else 64, 3, 1)))
    torch.cuda.synchronize()
    assert status.tolist() == [0]
    check_lane(L, 0, q, out, lse)


def test_refusals_of_the_binding():
    L = Lanes([2], [20], seed=27)
    q = L.queries(4)
    out = torch.empty_like(q)
    bad = [dict(q=q.float()), dict(q=q[0]), dict(out=out[:1]), dict(out=out.float()), dict(q=q.transpose(1, 2), out=out.transpose(1, 2)),
           dict(q=q[:, :3], out=out[:, :3]), dict(q=q[..., :64], out=out[..., :64]), dict(lse=torch.empty(2, 3, device=DEV)),
           dict(lane_status=torch.zeros(1, device=DEV)), dict(tables=L.tables.long()), dict(tables=L.tables[0]),
           dict(tables=L.tables.repeat(2, 1)), dict(cached=None), dict(offsets=None), dict(cache=tuple(L.cache)), dict(scale="1"),
           dict(max_len=2 ** 40), dict(workspace=torch.empty(9, device=DEV))]
    for kw in bad:
        a = dict(q=q, cache=L.cache, tables=L.tables, cached=L.cached, offsets=L.offsets, out=out, max_len=2) | kw
        with pytest.raises((ValueError, TypeError)):
            sv.spec_paged_attention(a.pop("q"), a.pop("cache"), a.pop("tables"), a.pop("cached"), a.pop("offsets"), a.pop("out"),
                                    a.pop("max_len"), **a)
    k, v, _, _ = L.cache
    for args in ((k, v[:1]), (k, v.float()), (k.float(), v.float()), (k[0], v[0]), (k, v, torch.zeros(1)), (k.view(torch.int8), v.view(torch.int8))):
        with pytest.raises(ValueError):
            sv.PagedCache(*args)
    rows = torch.zeros(2, L.kv, L.d, device=DEV)
    for kk, vv in ((rows.half(), rows.half()), (rows[:, :1], rows[:, :1]), (rows, rows[:1]), (rows.transpose(1, 2), rows.transpose(1, 2))):
        with pytest.raises(ValueError):
            sv.spec_cache_write(*L.where(), kk, vv, 2)
