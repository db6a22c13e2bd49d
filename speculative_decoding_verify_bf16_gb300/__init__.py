"""Python binding of libspecverify, the GB300 verify-round library.

Argument marshalling only: every step of the verify round runs in the CUDA
kernels behind the C ABI of ``include/spec_verify.h``.  Tensors must already be
on the GPU; PyTorch provides device memory and the current stream.  If the
shared library has not been built every entry point raises -- there is no CPU
fallback.
"""

import ctypes
import os
import struct

import torch

from .build import LIB_PATH, build_library

__all__ = [
    "SPEC_OK", "SPEC_ERR_INVALID_ARG", "SPEC_ERR_UNSUPPORTED", "SPEC_ERR_CUDA",
    "SPEC_ERR_NONFINITE", "SPEC_ERR_TOKEN_RANGE", "SPEC_ERR_LAYOUT", "SPEC_ERR_TIMEOUT",
    "SPEC_MAX_DRAFTS", "SpecError", "ROW_STATS_FIELDS", "load_library", "build_library",
    "spec_row_budget", "spec_verify_accept", "spec_commit_state", "spec_status_string",
    "spec_verify_launch_shape", "spec_round_uniforms", "new_row_stats", "row_stats_view",
    "spec_accept_counts_update", "spec_accept_rates_from_counts", "new_accept_counts", "accept_counts_view",
    "spec_backoff_step", "new_backoff_states", "BACKOFF_FIELDS", "ACCEPT_COUNT_WORDS",
    "spec_ngram_draft", "SPEC_NGRAM_MAX_MATCH", "spec_apply_penalties", "SPEC_VERIFY_META_BEFORE_WAIT",
    "SPEC_VERIFY_TEST_WITHHOLD_COPY", "spec_token_logprobs", "SPEC_LOGPROBS_MAX_TOP", "spec_linear_prefill",
    "spec_linear_verify", "spec_linear_workspace", "new_linear_workspace", "SPEC_LINEAR_MAX_DIM",
    "PagedCache", "new_paged_cache", "spec_cache_write", "spec_cache_read", "spec_paged_attention",
    "spec_paged_attention_workspace", "new_paged_attention_workspace", "SPEC_CACHE_MAX_DIM", "SPEC_CACHE_LEAST_EXP",
    "SPEC_CACHE_MOST_EXP",
]

SPEC_OK = 0
SPEC_ERR_INVALID_ARG = 1
SPEC_ERR_UNSUPPORTED = 2
SPEC_ERR_CUDA = 3
SPEC_ERR_NONFINITE = 4
SPEC_ERR_TOKEN_RANGE = 5
SPEC_ERR_LAYOUT = 6
SPEC_ERR_TIMEOUT = 7
SPEC_MAX_DRAFTS = 15
SPEC_VERIFY_META_BEFORE_WAIT = 1
SPEC_VERIFY_TEST_WITHHOLD_COPY = 2

_DTYPES = {torch.float32: 0, torch.bfloat16: 1}

# spec_row_stats: 8 x 32-bit words per row.
ROW_STATS_FIELDS = ("argmax", "max_logit", "lse", "logp_d", "logq_d", "resid_mass", "drawn", "flags")
_ROW_STATS_INT = {"argmax", "drawn", "flags"}


class SpecError(RuntimeError):
    """A non-zero status returned by the library."""

    def __init__(self, code, what):
        self.code = code
        super().__init__(f"{what}: {spec_status_string(code)} ({code})")


class _Args(ctypes.Structure):
    _fields_ = [
        ("target_logits", ctypes.c_void_p),
        ("draft_logits", ctypes.c_void_p),
        ("dtype", ctypes.c_int),
        ("ld", ctypes.c_int64),
        ("V", ctypes.c_int32),
        ("lanes", ctypes.c_int32),
        ("rows", ctypes.c_int32),
        ("draft_tokens", ctypes.c_void_p),
        ("draft_lens", ctypes.c_void_p),
        ("row_offsets", ctypes.c_void_p),
        ("temperatures", ctypes.c_void_p),
        ("seed", ctypes.c_uint64),
        ("committed", ctypes.c_void_p),
        ("out_tokens", ctypes.c_void_p),
        ("lane_status", ctypes.c_void_p),
        ("row_stats", ctypes.c_void_p),
        ("lane_base", ctypes.c_uint32),
        ("flags", ctypes.c_uint32),
    ]


_lib = None


class _AcceptCounts(ctypes.Structure):
    _fields_ = [("rounds", ctypes.c_uint64), ("proposed", ctypes.c_uint64), ("accepted", ctypes.c_uint64),
                ("slot_reached", ctypes.c_uint64 * SPEC_MAX_DRAFTS), ("slot_kept", ctypes.c_uint64 * SPEC_MAX_DRAFTS)]


class _AcceptRates(ctypes.Structure):
    _fields_ = [("accepted_per_proposed", ctypes.c_double), ("tokens_per_round", ctypes.c_double),
                ("by_slot", ctypes.c_double * SPEC_MAX_DRAFTS), ("given_previous", ctypes.c_double * SPEC_MAX_DRAFTS),
                ("depth", ctypes.c_int32), ("reserved", ctypes.c_int32), ("implied_alpha", ctypes.c_double)]


class _LogprobsArgs(ctypes.Structure):
    _fields_ = [("logits", ctypes.c_void_p), ("dtype", ctypes.c_int), ("ld", ctypes.c_int64), ("V", ctypes.c_int32),
                ("rows", ctypes.c_int32), ("tokens", ctypes.c_void_p), ("temperatures", ctypes.c_void_p),
                ("logprobs", ctypes.c_void_p), ("entropy", ctypes.c_void_p), ("top", ctypes.c_int32),
                ("top_ids", ctypes.c_void_p), ("top_logprobs", ctypes.c_void_p), ("row_status", ctypes.c_void_p)]


class _LinearArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "k", "v", "out")] + \
        [(f"{n}_{s}_stride", ctypes.c_int64) for n in ("q", "k", "v", "out") for s in ("row", "head")] + \
        [("log_decay", ctypes.c_void_p), ("decay_row_stride", ctypes.c_int64), ("decay_head_stride", ctypes.c_int64),
         ("row_offsets", ctypes.c_void_p),
         ("state_in", ctypes.c_void_p), ("state_in_lane_stride", ctypes.c_int64), ("state_in_head_stride", ctypes.c_int64),
         ("state_out", ctypes.c_void_p), ("state_out_lane_stride", ctypes.c_int64),
         ("state_out_col_stride", ctypes.c_int64), ("state_out_head_stride", ctypes.c_int64),
         ("lane_status", ctypes.c_void_p), ("dtype", ctypes.c_int), ("lanes", ctypes.c_int32), ("rows", ctypes.c_int32),
         ("max_len", ctypes.c_int32), ("k_heads", ctypes.c_int32), ("v_heads", ctypes.c_int32), ("dk", ctypes.c_int32),
         ("dv", ctypes.c_int32), ("scale", ctypes.c_float), ("workspace", ctypes.c_void_p),
         ("workspace_bytes", ctypes.c_uint64)]


class _PagedCache(ctypes.Structure):
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("slot_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("k_exps", ctypes.c_void_p),
                ("v_exps", ctypes.c_void_p), ("exp_page_stride", ctypes.c_int64), ("exp_slot_stride", ctypes.c_int64),
                ("exp_head_stride", ctypes.c_int64), ("block_tables", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("cached_lens", ctypes.c_void_p), ("row_offsets", ctypes.c_void_p), ("lane_status", ctypes.c_void_p),
                ("type", ctypes.c_int)] + \
        [(n, ctypes.c_int32) for n in ("pages", "page_size", "table_width", "lanes", "rows", "max_len", "kv_heads", "dim")]


class _CacheRowsArgs(ctypes.Structure):
    _fields_ = [("cache", _PagedCache), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_row_stride", ctypes.c_int64),
                ("k_head_stride", ctypes.c_int64), ("v_row_stride", ctypes.c_int64), ("v_head_stride", ctypes.c_int64),
                ("dtype", ctypes.c_int)]


class _PagedAttentionArgs(ctypes.Structure):
    _fields_ = [("cache", _PagedCache), ("q", ctypes.c_void_p), ("out", ctypes.c_void_p), ("q_row_stride", ctypes.c_int64),
                ("q_head_stride", ctypes.c_int64), ("out_row_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64),
                ("lse", ctypes.c_void_p), ("lse_row_stride", ctypes.c_int64), ("q_heads", ctypes.c_int32),
                ("window", ctypes.c_int32), ("max_context", ctypes.c_int32), ("scale", ctypes.c_float),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_uint64)]


ACCEPT_COUNT_WORDS = 3 + 2 * SPEC_MAX_DRAFTS
BACKOFF_FIELDS = ("misses", "backoff", "wait", "reserved")


def load_library():
    """Load libspecverify.so (built in-tree); raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; call speculative_decoding_verify_bf16_gb300."
                           "build_library() (needs nvcc) -- there is no CPU fallback")
    lib = ctypes.CDLL(LIB_PATH)
    lib.spec_row_budget.restype = ctypes.c_int32
    lib.spec_row_budget.argtypes = [ctypes.c_int32] * 3
    lib.spec_verify_accept.restype = ctypes.c_int
    lib.spec_verify_accept.argtypes = [ctypes.POINTER(_Args), ctypes.c_void_p]
    lib.spec_commit_state.restype = ctypes.c_int
    lib.spec_commit_state.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.c_int32, ctypes.c_int32, ctypes.c_uint64,
                                      ctypes.c_uint64, ctypes.c_uint64, ctypes.c_uint64,
                                      ctypes.c_void_p, ctypes.c_void_p]
    lib.spec_status_string.restype = ctypes.c_char_p
    lib.spec_status_string.argtypes = [ctypes.c_int]
    lib.spec_round_uniforms.restype = ctypes.c_int
    lib.spec_round_uniforms.argtypes = [ctypes.c_uint64, ctypes.c_uint32, ctypes.c_int32, ctypes.c_int32,
                                        ctypes.c_void_p, ctypes.c_void_p]
    lib.spec_verify_launch_shape.restype = ctypes.c_int
    lib.spec_verify_launch_shape.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int,
                                             ctypes.c_int32] + [ctypes.POINTER(ctypes.c_int32)] * 4
    lib.spec_accept_counts_update.restype = ctypes.c_int
    lib.spec_accept_counts_update.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                              ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p]
    lib.spec_accept_rates_from_counts.restype = ctypes.c_int
    lib.spec_accept_rates_from_counts.argtypes = [ctypes.POINTER(_AcceptCounts), ctypes.POINTER(_AcceptRates)]
    lib.spec_backoff_init.restype = ctypes.c_int
    lib.spec_backoff_init.argtypes = [ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p]
    lib.spec_ngram_draft.restype = ctypes.c_int
    lib.spec_ngram_draft.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                     ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p]
    lib.spec_apply_penalties.restype = ctypes.c_int
    lib.spec_apply_penalties.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32] + \
        [ctypes.c_void_p] * 10
    lib.spec_backoff_step.restype = ctypes.c_int
    lib.spec_backoff_step.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p]
    lib.spec_token_logprobs.restype = ctypes.c_int
    lib.spec_token_logprobs.argtypes = [ctypes.c_void_p, ctypes.c_void_p]  # (packed bytes, or a structure)
    lib.spec_linear_workspace.restype = ctypes.c_uint64
    lib.spec_linear_workspace.argtypes = [ctypes.c_int32] * 5
    lib.spec_paged_attention_workspace.restype = ctypes.c_uint64
    lib.spec_paged_attention_workspace.argtypes = [ctypes.c_int32] * 4
    for f in (lib.spec_linear_prefill, lib.spec_linear_verify, lib.spec_cache_write, lib.spec_cache_read,
              lib.spec_paged_attention):
        f.restype = ctypes.c_int
        f.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    _lib = lib
    return lib


def spec_status_string(code):
    return load_library().spec_status_string(int(code)).decode()


def spec_row_budget(draft_tokens, row_budget, lanes):
    """Drafts per lane under a row budget; raises ValueError on bad arguments."""
    r = load_library().spec_row_budget(int(draft_tokens), int(row_budget), int(lanes))
    if r < 0:
        raise ValueError(f"spec_row_budget({draft_tokens}, {row_budget}, {lanes}): "
                         f"{spec_status_string(-r)}")
    return int(r)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t, name, dtype, device, numel=None):
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise ValueError(f"{name} must be a tensor on {device}")
    if t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name} needs at least {numel} elements")


def new_row_stats(rows, device):
    """An int32 [rows, 8] buffer laid out as spec_row_stats."""
    return torch.empty(rows, 8, dtype=torch.int32, device=device)


def row_stats_view(buf):
    """Dict of named columns of a row-stats buffer (float fields viewed as float32)."""
    out = {}
    for i, name in enumerate(ROW_STATS_FIELDS):
        col = buf[:, i].contiguous()
        out[name] = col if name in _ROW_STATS_INT else col.view(torch.float32)
    return out


def spec_verify_accept(target, draft, draft_tokens, draft_lens, row_offsets, temperatures, seed,
                       committed, out_tokens, lane_status=None, row_stats=None, stream=None,
                       rows=None, lane_base=0, meta_before_wait=False, test_flags=0):
    """Launch the fused verify kernel (see spec_verify_accept in include/spec_verify.h).

    target, draft: [rows, >= V] bf16 or float32 CUDA tensors with unit inner
    stride (draft may be None when no lane samples); the row stride is taken as
    ld.  draft_tokens, out_tokens: int32 [rows]; draft_lens, committed,
    lane_status: int32 [lanes]; row_offsets: int32 [lanes + 1]; temperatures:
    float32 [lanes]; row_stats: int32 [rows, 8] from new_row_stats().
    ``rows`` defaults to target.shape[0] (it must equal row_offsets[-1]).
    ``lane_base`` is the global index of lane 0 in the Philox counter (a batch
    split into parts draws the uniforms of the unsplit batch).
    ``meta_before_wait`` sets SPEC_VERIFY_META_BEFORE_WAIT: the caller promises
    that the kernel preceding this launch on the stream did not write
    draft_tokens, draft_lens, row_offsets or temperatures.  ``test_flags`` adds
    test-only flags (SPEC_VERIFY_TEST_WITHHOLD_COPY).
    """
    lib = load_library()
    if target.dim() != 2 or target.stride(1) != 1 or target.dtype not in _DTYPES:
        raise ValueError("target must be a 2-D bf16/float32 tensor with unit inner stride")
    dev = target.device
    if dev.type != "cuda":
        raise ValueError("target must be on a CUDA device")
    if draft is not None and (draft.dtype != target.dtype or draft.device != dev or draft.dim() != 2
                              or draft.stride(1) != 1 or draft.stride(0) != target.stride(0)):
        raise ValueError("draft must match target's dtype, device and row stride")
    lanes = draft_lens.numel()
    nrows = target.shape[0] if rows is None else int(rows)
    if nrows > target.shape[0] or (draft is not None and nrows > draft.shape[0]):
        raise ValueError("rows exceeds the rows of the logits tensors")
    _need(draft_tokens, "draft_tokens", torch.int32, dev, nrows)
    _need(draft_lens, "draft_lens", torch.int32, dev)
    _need(row_offsets, "row_offsets", torch.int32, dev, lanes + 1)
    _need(temperatures, "temperatures", torch.float32, dev, lanes)
    _need(committed, "committed", torch.int32, dev, lanes)
    _need(out_tokens, "out_tokens", torch.int32, dev, nrows)
    if lane_status is not None:
        _need(lane_status, "lane_status", torch.int32, dev, lanes)
    if row_stats is not None:
        _need(row_stats, "row_stats", torch.int32, dev, nrows * 8)
    a = _Args(
        target_logits=target.data_ptr(),
        draft_logits=None if draft is None else draft.data_ptr(),
        dtype=_DTYPES[target.dtype],
        ld=target.stride(0),
        V=target.shape[1],
        lanes=lanes,
        rows=nrows,
        draft_tokens=draft_tokens.data_ptr(),
        draft_lens=draft_lens.data_ptr(),
        row_offsets=row_offsets.data_ptr(),
        temperatures=temperatures.data_ptr(),
        seed=int(seed) & ((1 << 64) - 1),
        committed=committed.data_ptr(),
        out_tokens=out_tokens.data_ptr(),
        lane_status=None if lane_status is None else lane_status.data_ptr(),
        row_stats=None if row_stats is None else row_stats.data_ptr(),
        lane_base=int(lane_base),
        flags=(SPEC_VERIFY_META_BEFORE_WAIT if meta_before_wait else 0) | int(test_flags),
    )
    code = lib.spec_verify_accept(ctypes.byref(a), _stream(stream))
    if code != SPEC_OK:
        raise SpecError(code, "spec_verify_accept")


def spec_verify_accept_raw(args, stream):
    """Call spec_verify_accept with a prepared _Args (no checks); returns the status."""
    return load_library().spec_verify_accept(ctypes.byref(args), stream)


def make_args(target, draft, draft_tokens, draft_lens, row_offsets, temperatures, seed,
              committed, out_tokens, lane_status=None, row_stats=None, V=None, rows=None, lane_base=0,
              meta_before_wait=False):
    """Build the C argument struct once (for tight loops that call it repeatedly)."""
    return _Args(
        target_logits=target.data_ptr(),
        draft_logits=None if draft is None else draft.data_ptr(),
        dtype=_DTYPES[target.dtype],
        ld=target.stride(0),
        V=target.shape[1] if V is None else int(V),
        lanes=draft_lens.numel(),
        rows=target.shape[0] if rows is None else int(rows),
        draft_tokens=draft_tokens.data_ptr(),
        draft_lens=draft_lens.data_ptr(),
        row_offsets=row_offsets.data_ptr(),
        temperatures=temperatures.data_ptr(),
        seed=int(seed) & ((1 << 64) - 1),
        committed=committed.data_ptr(),
        out_tokens=out_tokens.data_ptr(),
        lane_status=None if lane_status is None else lane_status.data_ptr(),
        row_stats=None if row_stats is None else row_stats.data_ptr(),
        lane_base=int(lane_base),
        flags=SPEC_VERIFY_META_BEFORE_WAIT if meta_before_wait else 0,
    )


def spec_commit_state(staged, live, committed, lane_status=None, stream=None):
    """Copy staged[b, committed[b] - 1] into live[b] for every lane (on the GPU).

    staged: [lanes, cols, ...] and live: [lanes, ...] CUDA tensors of one dtype
    whose per-column snapshot is contiguous.
    """
    lib = load_library()
    lanes, cols = staged.shape[0], staged.shape[1]
    dev = staged.device
    if live.device != dev or live.dtype != staged.dtype or live.shape[0] != lanes:
        raise ValueError("live must match staged's device, dtype and lane count")
    if not staged[0, 0].is_contiguous() or not live[0].is_contiguous():
        raise ValueError("each snapshot must be contiguous")
    esize = staged.element_size()
    bytes_per_col = live[0].numel() * esize
    if staged[0, 0].numel() * esize != bytes_per_col:
        raise ValueError("staged and live snapshots differ in size")
    _need(committed, "committed", torch.int32, dev, lanes)
    if lane_status is not None:
        _need(lane_status, "lane_status", torch.int32, dev, lanes)
    code = lib.spec_commit_state(
        _ptr(staged), _ptr(live), _ptr(committed), lanes, cols, bytes_per_col,
        staged.stride(0) * esize, staged.stride(1) * esize, live.stride(0) * esize,
        _ptr(lane_status), _stream(stream))
    if code != SPEC_OK:
        raise SpecError(code, "spec_commit_state")


def spec_round_uniforms(seed, lanes, positions, lane_base=0, device=None, stream=None):
    """float32 [lanes, positions, 2]: the (u, u') pairs the verify kernel draws."""
    lib = load_library()
    device = device or torch.device("cuda", torch.cuda.current_device())
    out = torch.empty(lanes, positions, 2, dtype=torch.float32, device=device)
    code = lib.spec_round_uniforms(int(seed) & ((1 << 64) - 1), int(lane_base), int(lanes), int(positions),
                                   _ptr(out), _stream(stream))
    if code != SPEC_OK:
        raise SpecError(code, "spec_round_uniforms")
    return out


def spec_verify_launch_shape(lanes, rows, V, dtype=torch.bfloat16, with_draft=False):
    """Launch shape spec_verify_accept would pick (see include/spec_verify.h)."""
    lib = load_library()
    vals = [ctypes.c_int32() for _ in range(4)]
    code = lib.spec_verify_launch_shape(int(lanes), int(rows), int(V), _DTYPES[dtype], int(bool(with_draft)),
                                        *[ctypes.byref(v) for v in vals])
    if code != SPEC_OK:
        raise SpecError(code, "spec_verify_launch_shape")
    return dict(zip(("cluster_ctas", "threads", "slice", "smem_bytes"), (v.value for v in vals)))


# ---------------------------------------------------------------------------
# Acceptance metrics and miss back-off (include/spec_round_control.h)
# ---------------------------------------------------------------------------
def new_accept_counts(n, device):
    """Zeroed int64 [n, 33] buffer laid out as n spec_accept_counts."""
    return torch.zeros(n, ACCEPT_COUNT_WORDS, dtype=torch.int64, device=device)


def accept_counts_view(row):
    """Dict of one spec_accept_counts row (any int64 tensor or sequence of 33 words)."""
    w = [int(x) for x in (row.tolist() if isinstance(row, torch.Tensor) else row)]
    k = SPEC_MAX_DRAFTS
    return {"rounds": w[0], "proposed": w[1], "accepted": w[2],
            "slot_reached": w[3:3 + k], "slot_kept": w[3 + k:3 + 2 * k]}


def spec_accept_counts_update(committed, draft_lens, lane_status, counts, per_lane=False, stream=None):
    """Add one verify round's outputs to device counts (new_accept_counts(1) for the
    batch, new_accept_counts(lanes) with per_lane=True)."""
    lib = load_library()
    dev = committed.device
    lanes = committed.numel()
    _need(committed, "committed", torch.int32, dev)
    _need(draft_lens, "draft_lens", torch.int32, dev, lanes)
    if lane_status is not None:
        _need(lane_status, "lane_status", torch.int32, dev, lanes)
    _need(counts, "counts", torch.int64, dev, (lanes if per_lane else 1) * ACCEPT_COUNT_WORDS)
    rc = lib.spec_accept_counts_update(_ptr(committed), _ptr(draft_lens), _ptr(lane_status), lanes,
                                       _ptr(counts), 1 if per_lane else 0, _stream(stream))
    if rc != SPEC_OK:
        raise SpecError(rc, "spec_accept_counts_update")


def spec_accept_rates_from_counts(counts_row):
    """The page's rates from one set of counts (host call)."""
    c = accept_counts_view(counts_row)
    cs = _AcceptCounts(c["rounds"], c["proposed"], c["accepted"],
                       (ctypes.c_uint64 * SPEC_MAX_DRAFTS)(*c["slot_reached"]),
                       (ctypes.c_uint64 * SPEC_MAX_DRAFTS)(*c["slot_kept"]))
    r = _AcceptRates()
    rc = load_library().spec_accept_rates_from_counts(ctypes.byref(cs), ctypes.byref(r))
    if rc != SPEC_OK:
        raise SpecError(rc, "spec_accept_rates_from_counts")
    return {"accepted_per_proposed": r.accepted_per_proposed, "tokens_per_round": r.tokens_per_round,
            "by_slot": list(r.by_slot), "given_previous": list(r.given_previous), "depth": r.depth,
            "implied_alpha": r.implied_alpha}


def new_backoff_states(lanes, device, stream=None):
    """int32 [lanes, 4] back-off states, initialised on the device."""
    st = torch.empty(lanes, 4, dtype=torch.int32, device=device)
    rc = load_library().spec_backoff_init(_ptr(st), lanes, _stream(stream))
    if rc != SPEC_OK:
        raise SpecError(rc, "spec_backoff_init")
    return st


def spec_backoff_step(states, proposed, committed, lane_status, draft_tokens, next_draft_lens, stream=None):
    """Advance the back-off of every lane by one verify round; writes the next
    round's draft lengths."""
    lib = load_library()
    dev = states.device
    lanes = proposed.numel()
    _need(states, "states", torch.int32, dev, lanes * 4)
    _need(proposed, "proposed", torch.int32, dev)
    _need(committed, "committed", torch.int32, dev, lanes)
    if lane_status is not None:
        _need(lane_status, "lane_status", torch.int32, dev, lanes)
    _need(next_draft_lens, "next_draft_lens", torch.int32, dev, lanes)
    rc = lib.spec_backoff_step(_ptr(states), _ptr(proposed), _ptr(committed), _ptr(lane_status), lanes,
                               int(draft_tokens), _ptr(next_draft_lens), _stream(stream))
    if rc != SPEC_OK:
        raise SpecError(rc, "spec_backoff_step")


SPEC_NGRAM_MAX_MATCH = 16


def spec_ngram_draft(tokens, hist_offsets, k, drafts, draft_lens, match_min=1, match_max=4, stream=None):
    """Copy-from-the-conversation drafts for every lane: tokens int32 [total],
    hist_offsets int64 [lanes + 1], drafts int32 [lanes, >= k] (row stride taken
    as the draft stride), draft_lens int32 [lanes]."""
    lib = load_library()
    dev = tokens.device
    lanes = hist_offsets.numel() - 1
    _need(tokens, "tokens", torch.int32, dev)
    _need(hist_offsets, "hist_offsets", torch.int64, dev, lanes + 1)
    _need(draft_lens, "draft_lens", torch.int32, dev, lanes)
    if drafts.dim() != 2 or drafts.dtype != torch.int32 or drafts.device != dev or drafts.stride(1) != 1 \
            or drafts.shape[0] < lanes:
        raise ValueError("drafts must be an int32 [lanes, >= k] tensor with unit inner stride")
    rc = lib.spec_ngram_draft(_ptr(tokens), _ptr(hist_offsets), lanes, int(k), int(match_min), int(match_max),
                              _ptr(drafts), drafts.stride(0), _ptr(draft_lens), _stream(stream))
    if rc != SPEC_OK:
        raise SpecError(rc, "spec_ngram_draft")


def spec_apply_penalties(target, row_offsets, draft_tokens, draft_lens, pen_tokens, pen_counts, pen_offsets,
                         presence=None, frequency=None, lane_status=None, stream=None):
    """Per-row presence / frequency penalties on the target logits (see
    spec_apply_penalties in include/spec_round_control.h).  The logits in
    ``target`` are overwritten with the penalised values.  target: the round's
    [rows, >= V] bf16/float32 logits (V = target.shape[1], ld its row stride);
    pen_tokens / pen_counts int32 [n] (per lane ascending distinct ids, counts
    >= 1), pen_offsets int64 [lanes + 1]; presence / frequency float32 [lanes]
    or None; lane_status int32 [lanes] or None receives each lane's status (a
    lane whose list breaks the contract is left untouched)."""
    lib = load_library()
    if target.dim() != 2 or target.stride(1) != 1 or target.dtype not in _DTYPES:
        raise ValueError("target must be a 2-D bf16/float32 tensor with unit inner stride")
    dev = target.device
    lanes = draft_lens.numel()
    _need(row_offsets, "row_offsets", torch.int32, dev, lanes + 1)
    _need(draft_tokens, "draft_tokens", torch.int32, dev)
    _need(draft_lens, "draft_lens", torch.int32, dev)
    _need(pen_tokens, "pen_tokens", torch.int32, dev)
    _need(pen_counts, "pen_counts", torch.int32, dev, pen_tokens.numel())
    _need(pen_offsets, "pen_offsets", torch.int64, dev, lanes + 1)
    for t, name in ((presence, "presence"), (frequency, "frequency")):
        if t is not None:
            _need(t, name, torch.float32, dev, lanes)
    if lane_status is not None:
        _need(lane_status, "lane_status", torch.int32, dev, lanes)
    rc = lib.spec_apply_penalties(_ptr(target), _DTYPES[target.dtype], target.stride(0), target.shape[1], lanes,
                                  _ptr(row_offsets), _ptr(draft_tokens), _ptr(draft_lens), _ptr(pen_tokens),
                                  _ptr(pen_counts), _ptr(pen_offsets), _ptr(presence), _ptr(frequency),
                                  _ptr(lane_status), _stream(stream))
    if rc != SPEC_OK:
        raise SpecError(rc, "spec_apply_penalties")


# ---------------------------------------------------------------------------
# Log probabilities of given tokens (include/spec_logprobs.h)
# ---------------------------------------------------------------------------
SPEC_LOGPROBS_MAX_TOP = 20


class _Layout:
    """Packs a ctypes structure's fields, in order, into bytes in one step (filling a
    structure of thirty fields takes longer than a small kernel runs)."""

    _CODES = {ctypes.c_void_p: "Q", ctypes.c_int: "i", ctypes.c_int32: "i", ctypes.c_int64: "q", ctypes.c_uint64: "Q",
              ctypes.c_float: "f"}

    def __init__(self, cls):
        self.pack = struct.Struct("=" + self._format(cls)).pack

    @classmethod
    def _format(cls, kind):
        fmt, at = "", 0
        for name, field in kind._fields_:
            here = getattr(kind, name).offset
            inner = cls._format(field) if issubclass(field, ctypes.Structure) else cls._CODES[field]
            fmt += "x" * (here - at) + inner
            at = here + ctypes.sizeof(field)
        return fmt + "x" * (ctypes.sizeof(kind) - at)


_LOGPROBS_LAYOUT = _Layout(_LogprobsArgs)
_LINEAR_LAYOUT = _Layout(_LinearArgs)
_CACHE_ROWS_LAYOUT = _Layout(_CacheRowsArgs)
_PAGED_ATTENTION_LAYOUT = _Layout(_PagedAttentionArgs)


def _raw_stream(stream, index):
    return torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream


def _at(t, name, dtype, index, numel):
    """Address of a tensor that _need accepts, 0 for None.  (Comparing a device's number
    takes a third of comparing devices; these calls' checks are most of a small call.)"""
    if t is None:
        return 0
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index and t.is_contiguous()
            and t.numel() >= numel):
        _need(t, name, dtype, torch.device("cuda", index), numel)
    return t.data_ptr()


def spec_token_logprobs(logits, tokens, logprobs, entropy=None, top_ids=None, top_logprobs=None, temperatures=None,
                        row_status=None, rows=None, stream=None):
    """Log probability of each row's token (see spec_token_logprobs in
    include/spec_logprobs.h).

    logits: [rows, V] bf16 or float32 CUDA tensor with unit inner stride; tokens
    int32 [rows] (negative: the row is not asked for); logprobs, entropy
    float32 [rows]; top_ids int32 and top_logprobs float32 [rows, n], n <=
    SPEC_LOGPROBS_MAX_TOP; temperatures float32 [rows] (<= 0: unscaled);
    row_status int32 [rows].  ``rows`` defaults to logits.shape[0].
    """
    lib = _lib or load_library()
    code = _DTYPES.get(logits.dtype)
    shape, strides = logits.shape, logits.stride()
    if code is None or len(shape) != 2 or (strides[1] != 1 and shape[1] > 1):
        raise ValueError("logits must be a 2-D bf16/float32 tensor with unit inner stride")
    if not logits.is_cuda:
        raise ValueError("logits must be on a CUDA device")
    dev = logits.get_device()
    have, V = shape
    n = have if rows is None else int(rows)
    if n > have:
        raise ValueError("rows exceeds the rows of logits")
    if tokens is None or logprobs is None:
        raise ValueError("tokens and logprobs are required")
    top = ids = alts = 0
    if top_ids is not None and top_logprobs is not None:
        if top_ids.dim() != 2 or top_ids.shape != top_logprobs.shape:
            raise ValueError("top_ids and top_logprobs must be [rows, n]")
        top = top_ids.shape[1]
        ids = _at(top_ids, "top_ids", torch.int32, dev, n * top)
        alts = _at(top_logprobs, "top_logprobs", torch.float32, dev, n * top)
    elif top_ids is not top_logprobs:
        raise ValueError("top_ids and top_logprobs go together")
    try:
        args = _LOGPROBS_LAYOUT.pack(
            logits.data_ptr(), code, strides[0] if have > 1 else max(strides[0], V), V, n,
            _at(tokens, "tokens", torch.int32, dev, n), _at(temperatures, "temperatures", torch.float32, dev, n),
            _at(logprobs, "logprobs", torch.float32, dev, n), _at(entropy, "entropy", torch.float32, dev, n), top, ids, alts,
            _at(row_status, "row_status", torch.int32, dev, n))
    except (struct.error, OverflowError) as e:
        raise ValueError(f"spec_token_logprobs: a size does not fit 32 bits ({e})") from None
    rc = lib.spec_token_logprobs(args, _raw_stream(stream, dev))
    if rc != SPEC_OK:
        raise SpecError(rc, "spec_token_logprobs")


# ---------------------------------------------------------------------------
# Linear attention with decay (include/spec_linear.h)
# ---------------------------------------------------------------------------
SPEC_LINEAR_MAX_DIM = 256


def spec_linear_workspace(lanes, v_heads, dk, dv, max_len):
    """Most bytes of scratch memory that spec_linear_prefill can use with up to this many
    lanes and tokens a lane."""
    return int(load_library().spec_linear_workspace(int(lanes), int(v_heads), int(dk), int(dv), int(max_len)))


def new_linear_workspace(lanes, v_heads, dk, dv, max_len, device):
    """A uint8 scratch buffer for spec_linear_prefill with up to this many lanes and tokens a
    lane (kept by the caller; calls that may run at the same time need one each)."""
    return torch.empty(spec_linear_workspace(lanes, v_heads, dk, dv, max_len), dtype=torch.uint8, device=device)


def _states(t, name, index, shape):
    """Address and strides of a state tensor ([.., dk, dv], the last two contiguous)."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.float32 or t.get_device() != index:
        raise ValueError(f"{name} must be a float32 tensor on cuda:{index}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}")
    s = t.stride()
    # (a size of one leaves its stride free, but the kernels read [dk][dv] rows)
    if (s[-1] != 1 and shape[-1] > 1) or (s[-2] != shape[-1] and shape[-2] > 1):
        raise ValueError(f"{name}'s last two dimensions must be contiguous")
    return t.data_ptr(), s


def _linear_call(entry, what, q, k, v, log_decay, row_offsets, out, max_len, scale, lane_status, before, before_name,
                 after, after_name, cols, workspace, stream):
    dtype, dev = q.dtype, q.get_device()
    code = _DTYPES.get(dtype)
    if code is None or not q.is_cuda:
        raise ValueError("q must be a bf16/float32 tensor on a CUDA device")
    if not (k.dtype is v.dtype is out.dtype is dtype and k.get_device() == v.get_device() == out.get_device() == dev):
        raise ValueError(f"k, v and out must be {dtype} tensors on cuda:{dev}, like q")
    qn, vn, qs, ks, vs, os_, gs = q.shape, v.shape, q.stride(), k.stride(), v.stride(), out.stride(), log_decay.stride()
    if k.shape != qn or out.shape != vn:
        raise ValueError("k must have q's shape, and out v's")
    if len(qn) != 3 or len(vn) != 3 or qn[0] != vn[0]:
        raise ValueError("q, k, v and out must be [rows, heads, size]")
    rows, hk, dk = qn
    _, hv, dv = vn
    if (qs[2] != 1 or ks[2] != 1) and dk > 1 or (vs[2] != 1 or os_[2] != 1) and dv > 1:
        raise ValueError("q, k, v and out must have unit inner stride")
    if hk == 0 or hv % hk:
        raise ValueError("v's heads must be a multiple of q's and k's")
    if log_decay.dtype is not torch.float32 or log_decay.get_device() != dev or log_decay.shape != (rows, hv):
        raise ValueError("log_decay must be a float32 [rows, v_heads] tensor (expanded strides allowed)")
    if row_offsets is None:
        raise ValueError("row_offsets is required")
    offsets = _at(row_offsets, "row_offsets", torch.int32, dev, 1)
    lanes = row_offsets.numel() - 1
    in_ptr = out_ptr = in_lane = in_head = out_lane = out_col = out_head = 0
    if before is not None:
        in_ptr, (in_lane, in_head, _, _) = _states(before, before_name, dev, (lanes, hv, dk, dv))
    if after is not None:
        if cols is None:
            out_ptr, (out_lane, out_head, _, _) = _states(after, after_name, dev, (lanes, hv, dk, dv))
        else:
            out_ptr, (out_lane, out_col, out_head, _, _) = _states(after, after_name, dev, (lanes, cols, hv, dk, dv))
    if workspace is None and cols is None and dtype is torch.bfloat16:  # (float32 prompts are never split)
        with torch.cuda.stream(stream):  # (memory of the stream that uses it; None: the current one)
            workspace = new_linear_workspace(lanes, hv, dk, dv, max_len, q.device)
    try:
        args = _LINEAR_LAYOUT.pack(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), qs[0], qs[1], ks[0], ks[1], vs[0], vs[1], os_[0],
            os_[1], log_decay.data_ptr(), gs[0], gs[1], offsets, in_ptr, in_lane, in_head, out_ptr, out_lane,
            out_col, out_head, _at(lane_status, "lane_status", torch.int32, dev, lanes), code, lanes, rows, max_len, hk, hv,
            dk, dv, dk ** -0.5 if scale is None else scale, 0 if workspace is None else workspace.data_ptr(),
            0 if workspace is None else workspace.numel())
    except (struct.error, OverflowError) as e:
        raise ValueError(f"{what}: a size does not fit 32 bits, or scale is no number ({e})") from None
    rc = entry(args, _raw_stream(stream, dev))
    if rc != SPEC_OK:
        raise SpecError(rc, what)


def spec_linear_prefill(q, k, v, log_decay, row_offsets, state_in, out, state_out, max_len, scale=None,
                        lane_status=None, workspace=None, stream=None):
    """Linear attention with decay over whole prompts (see spec_linear_prefill in
    include/spec_linear.h).

    q, k: [rows, k_heads, dk], v, out: [rows, v_heads, dv] of one dtype (bf16 or
    float32), lanes packed one after the other; log_decay: float32 [rows,
    v_heads] (``decay.expand(rows, -1)`` for one decay a head); row_offsets
    int32 [lanes + 1]; state_in (None: zeros) and state_out (None: not wanted;
    may be state_in) float32 [lanes, v_heads, dk, dv]; max_len: an upper bound
    of the lanes' lengths.  ``scale`` defaults to dk ** -0.5.  lane_status
    int32 [lanes] is read and updated: fill it with zeros before the first
    call.  ``workspace`` comes from new_linear_workspace (any size will do, a
    smaller one makes long prompts slower); without one the call takes scratch
    memory from PyTorch's allocator, on the stream that it runs on.
    """
    lib = _lib or load_library()
    if workspace is not None:
        _at(workspace, "workspace", torch.uint8, q.get_device(), 0)
    _linear_call(lib.spec_linear_prefill, "spec_linear_prefill", q, k, v, log_decay, row_offsets, out, int(max_len), scale,
                 lane_status, state_in, "state_in", state_out, "state_out", None, workspace, stream)


def spec_linear_verify(q, k, v, log_decay, row_offsets, live, staged, out, scale=None, lane_status=None, stream=None):
    """Linear attention with decay over a round's columns (see spec_linear_verify in
    include/spec_linear.h): reads ``live`` [lanes, v_heads, dk, dv] (None:
    zeros) and writes the state after column c of lane b to ``staged[b, c]``
    ([lanes, cols, v_heads, dk, dv]), from which spec_commit_state rolls.  For
    single-token decoding ``staged`` may be ``live.unsqueeze(1)``.  The other
    arguments are those of spec_linear_prefill.
    """
    lib = _lib or load_library()
    if not isinstance(staged, torch.Tensor) or staged.dim() != 5:
        raise ValueError("staged must be a [lanes, cols, v_heads, dk, dv] tensor")
    cols = staged.shape[1]
    _linear_call(lib.spec_linear_verify, "spec_linear_verify", q, k, v, log_decay, row_offsets, out, cols, scale,
                 lane_status, live, "live", staged, "staged", cols, None, stream)


# ---------------------------------------------------------------------------
# Paged key/value cache and the attention over it (include/spec_cache.h)
# ---------------------------------------------------------------------------
SPEC_CACHE_MAX_DIM = 256
SPEC_CACHE_LEAST_EXP = -48
SPEC_CACHE_MOST_EXP = 48

_CACHE_TYPES = {torch.bfloat16: 1, torch.float8_e4m3fn: 2, torch.int8: 3}


def _free_strides(shape, strides):
    """Strides of all dimensions but the last; those of a size of one, which are free, as for a
    packed tensor."""
    out, packed = [], shape[-1]
    for n, s in zip(shape[-2::-1], strides[-2::-1]):
        out.append(s if n > 1 else packed)
        packed = max(packed, out[-1] * n)
    return out[::-1]


class PagedCache:
    """Keys and values [pages, page_size, kv_heads, dim] (bf16, float8_e4m3fn or int8; any
    strides, the same for both, with a contiguous last dimension) and, for the 8-bit types,
    their exponents' bytes, uint8 [pages, page_size, kv_heads].  Checked once, when it is made;
    ``k, v, k_exps, v_exps = cache`` gives the tensors back."""

    __slots__ = ("_tensors", "_pools", "_sizes", "_heads", "_code", "_device")

    def __init__(self, k, v, k_exps=None, v_exps=None):
        code = _CACHE_TYPES.get(k.dtype)
        shape, strides, dev = k.shape, k.stride(), k.get_device()
        if code is None or len(shape) != 4:
            raise ValueError("k must be a bf16, float8_e4m3fn or int8 [pages, page_size, kv_heads, dim] tensor")
        if v.dtype is not k.dtype or v.shape != shape or v.stride() != strides or v.get_device() != dev:
            raise ValueError("v must match k's dtype, device, shape and strides")
        if strides[3] != 1:
            raise ValueError("k and v must have unit inner stride")
        ek = ev = 0
        es = (0, 0, 0)
        if code != 1:
            for t, name in ((k_exps, "k_exps"), (v_exps, "v_exps")):
                if not isinstance(t, torch.Tensor) or t.dtype is not torch.uint8 or t.get_device() != dev or t.shape != shape[:3]:
                    raise ValueError(f"{name} must be a uint8 [pages, page_size, kv_heads] tensor on k's device")
            es = k_exps.stride()
            if v_exps.stride() != es:
                raise ValueError("v_exps must have k_exps' strides")
            ek, ev = k_exps.data_ptr(), v_exps.data_ptr()
        elif k_exps is not None or v_exps is not None:
            raise ValueError("a bf16 cache has no exponents")
        self._tensors = (k, v, k_exps, v_exps)
        self._pools = (k.data_ptr(), v.data_ptr(), *_free_strides(shape, strides), ek, ev, *es)
        self._sizes, self._heads, self._code, self._device = shape[:2], shape[2:], code, dev

    k = property(lambda self: self._tensors[0])
    v = property(lambda self: self._tensors[1])
    k_exps = property(lambda self: self._tensors[2])
    v_exps = property(lambda self: self._tensors[3])

    def __iter__(self):
        return iter(self._tensors)


def new_paged_cache(pages, page_size, kv_heads, dim, dtype, device):
    """An empty (zeroed) PagedCache; dtype: torch.bfloat16, torch.float8_e4m3fn or torch.int8."""
    if dtype not in _CACHE_TYPES:
        raise ValueError("dtype must be torch.bfloat16, torch.float8_e4m3fn or torch.int8")
    shape = (pages, page_size, kv_heads, dim)
    # (zeros of one byte are zeros of every type)
    k, v = (torch.zeros(shape[:3] + (dim * dtype.itemsize,), dtype=torch.uint8, device=device).view(dtype) for _ in range(2))
    if dtype is torch.bfloat16:
        return PagedCache(k, v)
    exps = [torch.full(shape[:3], 127 + SPEC_CACHE_LEAST_EXP, dtype=torch.uint8, device=device) for _ in range(2)]
    return PagedCache(k, v, *exps)


def _cache_fields(cache, block_tables, cached_lens, row_offsets, lane_status, rows, max_len, dev):
    """The fields of a spec_paged_cache, in order."""
    if not isinstance(cache, PagedCache) or cache._device != dev:
        raise ValueError(f"cache must be a PagedCache on cuda:{dev}, like the rows")
    if row_offsets is None or cached_lens is None or block_tables is None:
        raise ValueError("block_tables, cached_lens and row_offsets are required")
    offsets = _at(row_offsets, "row_offsets", torch.int32, dev, 1)
    lanes = row_offsets.numel() - 1
    shape = block_tables.shape
    if block_tables.dtype is not torch.int32 or block_tables.get_device() != dev or len(shape) != 2 or shape[0] != lanes:
        raise ValueError(f"block_tables must be an int32 [lanes, width] tensor on cuda:{dev}")
    width, (stride, inner) = shape[1], block_tables.stride()
    if inner != 1 and width > 1 and lanes > 0:
        raise ValueError("block_tables must have unit inner stride")
    if lanes <= 1 and stride < width:  # (a size of one leaves its stride free)
        stride = width
    pages, page_size = cache._sizes
    kv_heads, dim = cache._heads
    return (*cache._pools, block_tables.data_ptr(), stride, _at(cached_lens, "cached_lens", torch.int32, dev, lanes), offsets,
            _at(lane_status, "lane_status", torch.int32, dev, lanes), cache._code, pages, page_size, width, lanes, rows,
            max_len, kv_heads, dim)


def _call(entry, what, args, stream, dev):
    """The library's call on the tensors' device, whichever is the current one."""
    if torch._C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            rc = entry(args, _raw_stream(stream, dev))
    else:
        rc = entry(args, _raw_stream(stream, dev))
    if rc != SPEC_OK:
        raise SpecError(rc, what)


def _cache_rows_call(entry, what, cache, block_tables, cached_lens, row_offsets, k, v, max_len, lane_status, stream):
    dtype, shape, dev = k.dtype, k.shape, k.get_device()
    code = _DTYPES.get(dtype)
    if code is None or not k.is_cuda or len(shape) != 3:
        raise ValueError("k must be a bf16/float32 [rows, kv_heads, dim] tensor on a CUDA device")
    if v.dtype is not dtype or v.shape != shape or v.get_device() != dev:
        raise ValueError("v must match k's dtype, device and shape")
    ks, vs = k.stride(), v.stride()
    if ks[2] != 1 or vs[2] != 1:
        raise ValueError("k and v must have unit inner stride")
    fields = _cache_fields(cache, block_tables, cached_lens, row_offsets, lane_status, shape[0], int(max_len), dev)
    if shape[1:] != cache._heads:
        raise ValueError("k and v must have the cache's heads and head size")
    if shape[0] < 2 or shape[1] < 2:
        ks, vs = _free_strides(shape, ks), _free_strides(shape, vs)
    try:
        args = _CACHE_ROWS_LAYOUT.pack(*fields, k.data_ptr(), v.data_ptr(), ks[0], ks[1], vs[0], vs[1], code)
    except (struct.error, OverflowError) as e:
        raise ValueError(f"{what}: a size does not fit 32 bits ({e})") from None
    _call(entry, what, args, stream, dev)


def spec_cache_write(cache, block_tables, cached_lens, row_offsets, k, v, max_len, lane_status=None, stream=None):
    """The lanes' new keys and values into their slots of the cache (see spec_cache_write in
    include/spec_cache.h).

    cache: a PagedCache; block_tables int32 [lanes, width]: a lane's pages;
    cached_lens int32 [lanes]: the tokens that a lane's cache holds already, behind which
    its rows go; row_offsets int32 [lanes + 1]; k, v: [rows, kv_heads, dim] bf16 or float32,
    lanes packed one after the other, rows and heads at strides of 16 bytes' multiples; max_len: an upper
    bound of the lanes' rows.  lane_status int32 [lanes] is read and updated: fill it
    with zeros before the first call.
    """
    lib = _lib or load_library()
    _cache_rows_call(lib.spec_cache_write, "spec_cache_write", cache, block_tables, cached_lens, row_offsets, k, v, max_len,
                     lane_status, stream)


def spec_cache_read(cache, block_tables, cached_lens, row_offsets, k_out, v_out, max_len, lane_status=None, stream=None):
    """Slots of the cache as the values they stand for (see spec_cache_read in
    include/spec_cache.h): row i of lane b is the token at position ``cached_lens[b] + i``.
    k_out and v_out [rows, kv_heads, dim], bf16 or float32, are written; the other arguments
    are those of spec_cache_write.
    """
    lib = _lib or load_library()
    _cache_rows_call(lib.spec_cache_read, "spec_cache_read", cache, block_tables, cached_lens, row_offsets, k_out, v_out,
                     max_len, lane_status, stream)


def spec_paged_attention_workspace(q_heads, kv_heads, dim, max_len):
    """Most bytes of scratch memory that spec_paged_attention can use with these heads and up
    to max_len columns a lane."""
    return int(load_library().spec_paged_attention_workspace(int(q_heads), int(kv_heads), int(dim), int(max_len)))


def new_paged_attention_workspace(q_heads, kv_heads, dim, max_len, device):
    """A uint8 scratch buffer for spec_paged_attention with these heads and up to max_len columns a
    lane, whatever the lanes and contexts (kept by the caller; calls that may run at the same
    time need one each)."""
    with torch.cuda.device(device):
        size = spec_paged_attention_workspace(q_heads, kv_heads, dim, max_len)
    return torch.empty(size, dtype=torch.uint8, device=device)


def spec_paged_attention(q, cache, block_tables, cached_lens, row_offsets, out, max_len, scale=None, window=0, lse=None,
                         lane_status=None, max_context=0, workspace=None, stream=None):
    """Attention of each lane's columns over its paged cache (see spec_paged_attention in
    include/spec_cache.h): column i of lane b sees positions up to its own,
    ``cached_lens[b] + i``, where spec_cache_write has put its key and value.

    q, out: [rows, q_heads, dim] bf16, lanes packed one after the other, rows and heads at
    strides of multiples of 8 elements; q_heads is a multiple of the cache's heads.  ``scale``
    defaults to dim ** -0.5; ``window`` > 0: the last so many positions, its own
    among them, are seen; lse: float32 [rows, q_heads] with unit inner stride, or None;
    ``max_context``: an upper bound of the lanes' positions (0: what the tables hold).
    ``workspace`` comes from new_paged_attention_workspace (a larger one will do; with a smaller one no
    context is split over thread blocks); without one the call takes scratch memory from
    PyTorch's allocator, on the stream that it runs on.  The other arguments are those of
    spec_cache_write.
    """
    lib = _lib or load_library()
    shape, dev = q.shape, q.get_device()
    if q.dtype is not torch.bfloat16 or not q.is_cuda or len(shape) != 3:
        raise ValueError("q must be a bf16 [rows, q_heads, dim] tensor on a CUDA device")
    if out.dtype is not torch.bfloat16 or out.shape != shape or out.get_device() != dev:
        raise ValueError("out must match q's dtype, device and shape")
    rows, hq, dim = shape
    qs, os_ = q.stride(), out.stride()
    if qs[2] != 1 or os_[2] != 1:
        raise ValueError("q and out must have unit inner stride")
    max_len = int(max_len)
    fields = _cache_fields(cache, block_tables, cached_lens, row_offsets, lane_status, rows, max_len, dev)
    kv = fields[-2]
    if dim != fields[-1] or kv == 0 or hq == 0 or hq % kv:  # (checked again by the library, but for dim)
        raise ValueError("q must have the cache's head size and a multiple of its heads")
    if rows < 2 or hq < 2:
        qs, os_ = _free_strides(shape, qs), _free_strides(shape, os_)
    lse_ptr = lse_row = 0
    if lse is not None:
        if lse.dtype is not torch.float32 or lse.get_device() != dev or lse.shape != (rows, hq) or (lse.stride(1) != 1 and hq > 1):
            raise ValueError(f"lse must be a float32 [rows, q_heads] tensor on cuda:{dev} with unit inner stride")
        lse_ptr, lse_row = lse.data_ptr(), lse.stride(0) if rows > 1 else max(lse.stride(0), hq)
    if workspace is None:
        with torch.cuda.stream(stream):  # (memory of the stream that uses it; None: the current one)
            workspace = new_paged_attention_workspace(hq, kv, dim, max_len, q.device)
    else:
        _at(workspace, "workspace", torch.uint8, dev, 0)
    try:
        args = _PAGED_ATTENTION_LAYOUT.pack(
            *fields, q.data_ptr(), out.data_ptr(), qs[0], qs[1], os_[0], os_[1], lse_ptr, lse_row, hq, int(window),
            int(max_context), dim ** -0.5 if scale is None else scale, workspace.data_ptr(), workspace.numel())
    except (struct.error, OverflowError) as e:
        raise ValueError(f"spec_paged_attention: a size does not fit 32 bits, or scale is no number ({e})") from None
    _call(lib.spec_paged_attention, "spec_paged_attention", args, stream, dev)
