"""Refusals of the paged cache's entry points: on the host, before any CUDA call (no GPU
needed; the pointers are never dereferenced), and the oracle's rounding."""

import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

from conftest import ROOT

import speculative_decoding_verify_bf16_gb300 as sv
from oracle import paged

FAKE = 4096


@pytest.fixture(scope="module")
def lib():
    sv.build_library()
    return sv.load_library()


def cache(**kw):
    c = dict(k_pages=FAKE, v_pages=FAKE, page_stride=16 * 256, slot_stride=256, head_stride=128, k_exps=FAKE, v_exps=FAKE,
             exp_page_stride=32, exp_slot_stride=2, exp_head_stride=1, block_tables=FAKE, table_stride=9, cached_lens=FAKE,
             row_offsets=FAKE, lane_status=None, type=2, pages=5, page_size=16, table_width=9, lanes=2, rows=9, max_len=9,
             kv_heads=2, dim=128)
    c.update(kw)
    return sv._PagedCache(**c)


BAD_CACHES = [dict(type=0), dict(type=4), dict(lanes=-1), dict(rows=-1), dict(max_len=-1), dict(table_width=-1), dict(table_width=10),
              dict(pages=0), dict(page_size=0), dict(kv_heads=0), dict(dim=0), dict(dim=8), dict(dim=100), dict(dim=272),
              dict(page_stride=-16), dict(slot_stride=8), dict(head_stride=24), dict(k_pages=FAKE + 8), dict(v_pages=FAKE + 2),
              dict(exp_slot_stride=-1), dict(k_pages=None), dict(v_pages=None), dict(cached_lens=None), dict(row_offsets=None),
              dict(block_tables=None), dict(k_exps=None), dict(v_exps=None)]


def rows_args(c=None, **kw):
    a = sv._CacheRowsArgs(cache=c or cache(), k=FAKE, v=FAKE, k_row_stride=256, k_head_stride=128, v_row_stride=256,
                          v_head_stride=128, dtype=1)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def attention_args(c=None, **kw):
    a = sv._PagedAttentionArgs(cache=c or cache(), q=FAKE, out=FAKE, q_row_stride=512, q_head_stride=128, out_row_stride=512,
                               out_head_stride=128, lse=FAKE, lse_row_stride=4, q_heads=4, scale=1.0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_cache_refusals(lib, kw):
    bad = sv.SPEC_ERR_INVALID_ARG
    assert lib.spec_cache_write(ctypes.byref(rows_args(cache(**kw))), None) == bad
    assert lib.spec_cache_read(ctypes.byref(rows_args(cache(**kw))), None) == bad
    assert lib.spec_paged_attention(ctypes.byref(attention_args(cache(**kw))), None) == bad


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=None), dict(k=FAKE + 8), dict(v=FAKE + 4), dict(k_row_stride=-8),
                                dict(k_row_stride=12), dict(v_head_stride=4), dict(dtype=2)])
def test_rows_refusals(lib, kw):
    for f in (lib.spec_cache_write, lib.spec_cache_read):
        assert f(ctypes.byref(rows_args(**kw)), None) == sv.SPEC_ERR_INVALID_ARG
    # one row for all tokens can be read, not written
    assert lib.spec_cache_read(ctypes.byref(rows_args(k_row_stride=0)), None) == sv.SPEC_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(q=None), dict(out=None), dict(q=FAKE + 8), dict(out=FAKE + 2), dict(workspace=FAKE + 4),
                                dict(q_row_stride=-8), dict(q_head_stride=4), dict(out_row_stride=0), dict(out_head_stride=12),
                                dict(q_heads=0), dict(q_heads=3), dict(q_heads=-2), dict(window=-1), dict(max_context=-1),
                                dict(lse_row_stride=3)])
def test_attention_refusals(lib, kw):
    assert lib.spec_paged_attention(ctypes.byref(attention_args(**kw)), None) == sv.SPEC_ERR_INVALID_ARG


def test_special_cases_on_the_host(lib):
    for f in (lib.spec_cache_write, lib.spec_cache_read, lib.spec_paged_attention):
        assert f(None, None) == sv.SPEC_ERR_INVALID_ARG
    empty = cache(lanes=0, row_offsets=None, cached_lens=None, block_tables=None, k_pages=None, v_pages=None, k_exps=None, v_exps=None)
    assert lib.spec_cache_write(ctypes.byref(rows_args(empty)), None) == sv.SPEC_OK
    assert lib.spec_cache_read(ctypes.byref(rows_args(empty)), None) == sv.SPEC_OK
    assert lib.spec_paged_attention(ctypes.byref(attention_args(empty)), None) == sv.SPEC_OK
    # rows of a head group that do not fit 2^30
    big = cache(max_len=2 ** 29)
    assert lib.spec_paged_attention(ctypes.byref(attention_args(big, q_heads=8, lse_row_stride=8)), None) == sv.SPEC_ERR_INVALID_ARG
    for bad in [(0, 1, 128, 1), (4, 0, 128, 1), (4, 3, 128, 1), (4, 2, 100, 1), (4, 2, 512, 1), (4, 2, 128, 0), (4, 2, 128, -3)]:
        assert sv.spec_paged_attention_workspace(*bad) == 0


def test_binding_structs_and_constants_match_the_header(tmp_path):
    for struct, cls in (("spec_paged_cache", sv._PagedCache), ("spec_cache_rows_args", sv._CacheRowsArgs),
                        ("spec_paged_attention_args", sv._PagedAttentionArgs)):
        fields = [n for n, _ in cls._fields_]
        body = "".join(f'  printf("%zu\\n", offsetof({struct}, {f}));\n' for f in fields)
        src = tmp_path / "layout.c"
        src.write_text(f'#include <stddef.h>\n#include <stdio.h>\n#include "spec_cache.h"\n'
                       f'int main(void) {{\n  printf("%zu\\n", sizeof({struct}));\n{body}  return 0;\n}}\n')
        exe = tmp_path / "layout"
        subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
        vals = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
        assert ctypes.sizeof(cls) == vals[0]
        assert [getattr(cls, f).offset for f in fields] == vals[1:]
    text = open(os.path.join(ROOT, "include", "spec_cache.h")).read()
    defines = {m.group(1): int(m.group(2)) for m in re.finditer(r"#define\s+(SPEC_\w+)\s+\(?(-?\d+)\)?", text)}
    for name in ("SPEC_CACHE_MAX_DIM", "SPEC_CACHE_LEAST_EXP", "SPEC_CACHE_MOST_EXP"):
        assert getattr(sv, name) == defines[name]
    assert (paged.LEAST, paged.MOST) == (sv.SPEC_CACHE_LEAST_EXP, sv.SPEC_CACHE_MOST_EXP)


def test_packed_arguments_equal_the_structures():
    """The binding packs bytes; they are what filling the structure gives."""
    a = attention_args()
    flat = [getattr(a.cache, n) or 0 for n, _ in sv._PagedCache._fields_]
    flat += [getattr(a, n) or 0 for n, _ in sv._PagedAttentionArgs._fields_[1:]]
    assert sv._PAGED_ATTENTION_LAYOUT.pack(*flat) == bytes(a)
    a = rows_args()
    flat = [getattr(a.cache, n) or 0 for n, _ in sv._PagedCache._fields_] + [getattr(a, n) or 0 for n, _ in sv._CacheRowsArgs._fields_[1:]]
    assert sv._CACHE_ROWS_LAYOUT.pack(*flat) == bytes(a)


def test_oracle_rounding():
    table = paged.e4m3_values()
    ours = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(table, ours, equal_nan=True)
    x = np.random.default_rng(0).normal(size=(50, 64)).astype(np.float32) * np.exp2(np.arange(-25, 25))[:, None].astype(np.float32)
    for kind in ("e4m3", "int8"):
        y, byte = paged.quantise(x, kind)
        top, big = paged.TOP[kind], np.abs(x).max(-1)
        e = byte - 127
        assert (top * 2.0 ** e >= big).all() and (top * 2.0 ** (e - 1) < big).all()
        z = torch.tensor(x / 2.0 ** e[:, None])
        want = z.float().to(torch.float8_e4m3fn).double() if kind == "e4m3" else z.round()
        assert np.array_equal(y, want.numpy())
    y, byte = paged.quantise(np.array([[0.0, 0.0], [np.nan, 1.0], [np.inf, 0.0], [1e30, 0.0], [1e-30, 0.0]]), "int8")
    assert byte.tolist() == [79, 255, 255, 255, 79]
    assert np.isnan(paged.values(y, byte)[1:4]).all() and (paged.values(y, byte)[[0, 4]] == 0).all()


def test_oracle_attention_small_case():
    """Two positions, by hand."""
    q, k = np.ones((1, 1, 1)), np.array([[[0.0]], [[np.log(3.0)]]])
    v = np.array([[[4.0]], [[8.0]]])
    out, lse, _, _ = paged.attention(q, k, v, 1, 1.0)
    assert np.allclose(out, 7.0) and np.allclose(lse, np.log(4.0))
    assert np.allclose(paged.attention(q, k, v, 1, 1.0, window=1)[0], 8.0)
