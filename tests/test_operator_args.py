"""Refusals of the operators' entry points: on the host, before any CUDA call (no GPU
needed; the pointers are never dereferenced)."""

import ctypes
import os
import re

import pytest

from conftest import ROOT

import speculative_decoding_verify_bf16_gb300 as sv

FAKE = 4096


@pytest.fixture(scope="module")
def lib():
    sv.build_library()
    return sv.load_library()


def logprobs_args(**kw):
    a = sv._LogprobsArgs(logits=FAKE, dtype=1, ld=64, V=64, rows=4, tokens=FAKE, temperatures=None, logprobs=FAKE,
                         entropy=None, top=3, top_ids=FAKE, top_logprobs=FAKE, row_status=None)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def linear_args(**kw):
    a = sv._LinearArgs(q=FAKE, k=FAKE, v=FAKE, out=FAKE, log_decay=FAKE, row_offsets=FAKE, state_in=FAKE,
                       state_out=FAKE, dtype=1, lanes=2, rows=9, max_len=9, k_heads=2, v_heads=4, dk=128, dv=128,
                       scale=1.0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw", [dict(rows=-1), dict(V=0), dict(V=-4), dict(ld=63), dict(dtype=2), dict(top=-1),
                                dict(top=21), dict(logits=None), dict(tokens=None), dict(logprobs=None),
                                dict(top_ids=None), dict(top_logprobs=None), dict(rows=2 ** 31 - 1)])
def test_logprobs_refusals(lib, kw):
    assert lib.spec_token_logprobs(ctypes.byref(logprobs_args(**kw)), None) == sv.SPEC_ERR_INVALID_ARG


def test_logprobs_no_rows_is_no_work(lib):
    assert lib.spec_token_logprobs(None, None) == sv.SPEC_ERR_INVALID_ARG
    assert lib.spec_token_logprobs(ctypes.byref(logprobs_args(rows=0, logits=None)), None) == sv.SPEC_OK


@pytest.mark.parametrize("kw", [dict(lanes=-1), dict(rows=-1), dict(max_len=-1), dict(dtype=5), dict(k_heads=0),
                                dict(v_heads=0), dict(v_heads=3), dict(dk=0), dict(dk=257), dict(dv=0), dict(dv=260),
                                dict(dv=126), dict(q=None), dict(k=None), dict(v=None), dict(out=None),
                                dict(log_decay=None), dict(row_offsets=None), dict(q_row_stride=-1),
                                dict(out_head_stride=-4), dict(state_in=FAKE + 4), dict(state_out=FAKE + 8),
                                dict(state_in_lane_stride=2), dict(state_out_head_stride=1),
                                dict(lanes=2 ** 30, v_heads=64)])
@pytest.mark.parametrize("entry", ["spec_linear_prefill", "spec_linear_verify"])
def test_linear_refusals(lib, entry, kw):
    assert getattr(lib, entry)(ctypes.byref(linear_args(**kw)), None) == sv.SPEC_ERR_INVALID_ARG


def test_linear_special_cases_on_the_host(lib):
    assert lib.spec_linear_prefill(None, None) == sv.SPEC_ERR_INVALID_ARG
    assert lib.spec_linear_verify(None, None) == sv.SPEC_ERR_INVALID_ARG
    assert lib.spec_linear_verify(ctypes.byref(linear_args(state_out=None)), None) == sv.SPEC_ERR_INVALID_ARG
    for f in (lib.spec_linear_prefill, lib.spec_linear_verify):
        assert f(ctypes.byref(linear_args(lanes=0, row_offsets=None)), None) == sv.SPEC_OK
    # sizes the prefill refuses want no scratch memory
    for bad in [(-1, 4, 128, 128, 9), (2, 0, 128, 128, 9), (2, 4, 0, 128, 9), (2, 4, 128, 300, 9), (2, 4, 128, 128, -1)]:
        assert sv.spec_linear_workspace(*bad) == 0


def test_binding_structs_and_constants_match_the_headers(tmp_path):
    import subprocess
    for header, struct, cls in (("spec_logprobs.h", "spec_logprobs_args", sv._LogprobsArgs),
                                ("spec_linear.h", "spec_linear_args", sv._LinearArgs)):
        fields = [n for n, _ in cls._fields_]
        body = "".join(f'  printf("%zu\\n", offsetof({struct}, {f}));\n' for f in fields)
        src = tmp_path / "layout.c"
        src.write_text(f'#include <stddef.h>\n#include <stdio.h>\n#include "{header}"\n'
                       f'int main(void) {{\n  printf("%zu\\n", sizeof({struct}));\n{body}  return 0;\n}}\n')
        exe = tmp_path / "layout"
        subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
        vals = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
        assert ctypes.sizeof(cls) == vals[0]
        assert [getattr(cls, f).offset for f in fields] == vals[1:]
    text = open(os.path.join(ROOT, "include", "spec_logprobs.h")).read() + \
        open(os.path.join(ROOT, "include", "spec_linear.h")).read()
    defines = {m.group(1): int(m.group(2)) for m in re.finditer(r"#define\s+(SPEC_\w+)\s+(\d+)\b", text)}
    assert defines["SPEC_LOGPROBS_MAX_TOP"] == sv.SPEC_LOGPROBS_MAX_TOP
    assert defines["SPEC_LINEAR_MAX_DIM"] == sv.SPEC_LINEAR_MAX_DIM
