"""Workloads of a paged key/value cache and the attention that reads it.

Three operators, each with listed cases and drawn ones of the same ranges:

  store   new tokens' keys and values quantised into the pages of a cache (8-bit
          values, a power of two for each token and head), and read back as the
          values that later rounds will see
  read    a lane's stretch of the cache read back out of its pages
  attend  attention of a chunk of new tokens (one, a verify round's columns, or a
          prompt's part) over the paged cache that holds them and all before them

``prepare`` makes what a serving program holds before the call, ``run`` makes
one pass (``own`` False: elementary torch operations in 32 bits; True: the
library's calls), ``exact`` states the definitions again in 64 bits and
``work`` counts the bytes and operations that a pass cannot do without.
"""

import math
import random

import torch

own = False

# Cache types: the largest value, and its exponent and fraction as frexp gives them.
FORMATS = {"e4m3": (448.0, 9, 0.875), "int8": (127.0, 7, 0.9921875)}
LEAST, MOST = -48, 48  # exponents of the powers of two that scale a token's head


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # Single-token decoding of one request: one row of eight heads, latency counts.
        dict(name="store_1x1_e4m3", op="store", lanes=1, lo=1, hi=1, before=1000, kv=8, d=128, page=16, cache="e4m3",
             dtype="bf16", pick=1),
        # A round of 64 lanes of one to four columns, fp32 activations.
        dict(name="store_64x4_int8_f32", op="store", lanes=64, lo=1, hi=4, before=4000, kv=8, d=128, page=64,
             cache="int8", dtype="f32", pick=2),
        # A batch of prompts of mixed lengths (one of them empty), pages that end inside them.
        dict(name="store_24x0to3000_e4m3", op="store", lanes=24, lo=0, hi=3000, before=500, kv=8, d=128, page=48,
             cache="e4m3", dtype="bf16", pick=3),
        # One long lane leaves for another machine in fp32.
        dict(name="read_1x40001_int8_f32", op="read", lanes=1, lo=40001, hi=40001, before=0, kv=8, d=128, page=64,
             cache="int8", dtype="f32", pick=4),
        # Stretches of 32 lanes come back for another layout, heads of 64, small pages.
        dict(name="read_32x100to4000_e4m3", op="read", lanes=32, lo=100, hi=4000, before=300, kv=4, d=64, page=16,
             cache="e4m3", dtype="bf16", pick=5),
        # Single-token decoding of one request with a short context: latency counts.
        dict(name="attend_1x1_ctx1500", op="attend", lanes=1, lo=1, hi=1, ctx_lo=1500, ctx_hi=1500, hq=16, kv=8, d=128,
             page=16, cache="bf16", window=0, lse=False, pick=6),
        # Single-token decoding of one request with a very long context.
        dict(name="attend_1x1_ctx131000", op="attend", lanes=1, lo=1, hi=1, ctx_lo=131000, ctx_hi=131000, hq=32, kv=8,
             d=128, page=16, cache="bf16", window=0, lse=False, pick=7),
        # Decoding of 64 lanes with contexts of all lengths, 8-bit integers.
        dict(name="attend_64x1_int8", op="attend", lanes=64, lo=1, hi=1, ctx_lo=0, ctx_hi=8192, hq=32, kv=8, d=128,
             page=64, cache="int8", window=0, lse=False, pick=8),
        # A verify round of 8 lanes x 8 columns, 8-bit floats.
        dict(name="attend_8x8_e4m3", op="attend", lanes=8, lo=8, hi=8, ctx_lo=2000, ctx_hi=16000, hq=32, kv=8, d=128,
             page=64, cache="e4m3", window=0, lse=False, pick=9),
        # A verify round of 64 lanes of one to four columns through a sliding-window layer,
        # heads of 64, pages that end inside every tile.
        dict(name="attend_64x4_window", op="attend", lanes=64, lo=1, hi=4, ctx_lo=0, ctx_hi=6000, hq=32, kv=4, d=64,
             page=24, cache="bf16", window=1000, lse=False, pick=10),
        # A batch of prompts' parts over what the cache holds of them, with the rows' log sums
        # (a later part of the context is merged in by them).
        dict(name="attend_12x0to1500_e4m3", op="attend", lanes=12, lo=0, hi=1500, ctx_lo=0, ctx_hi=3000, hq=16, kv=2,
             d=128, page=32, cache="e4m3", window=0, lse=True, pick=11),
        # The largest: 2,048 tokens of a long prompt behind 30,000 that are cached.
        dict(name="attend_1x2048_ctx30000", op="attend", lanes=1, lo=2048, hi=2048, ctx_lo=30000, ctx_hi=30000, hq=32,
             kv=8, d=128, page=64, cache="bf16", window=0, lse=False, pick=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["store", "read", "attend", "attend"])
    pick = rng.randrange(1, 1 << 30)
    kv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    page = rng.choice([16, 16, 24, 32, 48, 64, 100, 128])
    lanes = _log_int(rng, 1, 64)
    if op != "attend":
        hi = _log_int(rng, 1, 65536 // lanes)
        lo = hi if rng.random() < 0.3 else rng.randint(0, hi)
        return dict(op=op, lanes=lanes, lo=lo, hi=hi, before=_log_int(rng, 1, 4000) - 1, kv=kv, d=d, page=page,
                    cache=rng.choice(["e4m3", "int8"]), dtype=rng.choice(["bf16", "f32"]), pick=pick)
    hq = kv * rng.choice([1, 2, 4, 8])
    if rng.random() < 0.5:  # decoding and verify rounds
        hi = rng.choice([1, 1, 2, 4, 8, 16])
        ctx_hi = _log_int(rng, 1, min(131000, 600000 // lanes))
    else:
        hi = _log_int(rng, 16, 2048)
        ctx_hi = _log_int(rng, 1, 30000)
        # (a padded batch's scores of all heads stay below those of the largest case)
        lanes = min(lanes, max(1, 2048 * 30000 * 32 // (hq * hi * (hi + ctx_hi))))
    lo = hi if rng.random() < 0.5 else rng.randint(0, hi)
    ctx_lo = ctx_hi if rng.random() < 0.3 else rng.randint(0, ctx_hi)
    return dict(op="attend", lanes=lanes, lo=lo, hi=hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi, hq=hq, kv=kv, d=d, page=page,
                cache=rng.choice(["bf16", "bf16", "e4m3", "int8"]),
                window=rng.choice([0, 0, 0, _log_int(rng, 16, 4096)]), lse=rng.random() < 0.3, pick=pick)


def _lens(case):
    """The lanes' new tokens and the tokens before them (part of the case, not of the seed)."""
    rng = random.Random(case["pick"])
    lanes = case["lanes"]
    lens = [rng.randint(case["lo"], case["hi"]) for _ in range(lanes)]
    lens[-1] = case["hi"]
    if lanes > 2 and case["lo"] == 0:
        lens[1] = 0
    if case["op"] == "attend":
        before = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(lanes)]
        before[0] = case["ctx_hi"]
    else:
        before = [rng.randint(0, case["before"]) for _ in range(lanes)]
    return lens, before


def work(case):
    lens, before = _lens(case)
    kv, d = case["kv"], case["d"]
    slot = 2 * kv * d * (2 if case["cache"] == "bf16" else 1) + (0 if case["cache"] == "bf16" else 2 * kv)
    if case["op"] != "attend":
        row = 2 * kv * d * (4 if case["dtype"] == "f32" else 2)
        # store: rows in, slots out, slots in, rows out; each number scaled and rounded
        times = 2 if case["op"] == "store" else 1
        return {"bytes": times * sum(lens) * (row + slot), "flops": times * sum(lens) * 4 * kv * d}
    rows = sum(lens) * case["hq"] * (4 * d + (4 if case["lse"] else 0))
    seen, pairs = 0, 0  # slots that a lane's columns see, and pairs of a column and a slot
    for n, c in zip(lens, before):
        w = case["window"] or n + c
        seen += min(n + c, w + n - 1) if n else 0
        # column i sees min(c + i + 1, w)
        full = max(0, min(n, c + n - w + 1)) if w <= c + n else 0
        part = n - full
        pairs += full * w + part * c + part * (part + 1) // 2
    return {"bytes": rows + seen * slot, "flops": 4 * pairs * case["hq"] * d}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _tokens(n, kv, d, g, dev):
    """Keys or values as projections leave them: tokens of different sizes, some loud channels."""
    x = torch.randn(n, kv, d, generator=g, device=dev)
    x *= torch.exp(0.4 * torch.randn(n, kv, 1, generator=g, device=dev))
    x[..., ::16] *= 4.0
    return x


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 1000003 + case["pick"])
    lens, before = _lens(case)
    lanes, kv, d, page = case["lanes"], case["kv"], case["d"], case["page"]
    totals = [n + c for n, c in zip(lens, before)]
    width = max(1, -(-max(totals) // page))
    owned = [-(-t // page) for t in totals]
    pages = sum(owned) + 3
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    tables = torch.full((lanes, width), -1, dtype=torch.int32)  # (-1: no page, never looked at)
    host, at = order.cpu(), 0
    for b in range(lanes):
        tables[b, :owned[b]] = host[at:at + owned[b]]
        at += owned[b]
    tables = tables.to(dev)
    offsets = torch.tensor([sum(lens[:i]) for i in range(lanes + 1)], dtype=torch.int32, device=dev)
    cached = torch.tensor(before, dtype=torch.int32, device=dev)
    rows = sum(lens)
    st = dict(op=case["op"], kind=case["cache"], tables=tables, offsets=offsets, cached=cached, max_len=max(lens),
              max_context=max(totals), page=page, status=torch.zeros(lanes, dtype=torch.int32, device=dev))
    kind = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}[case["cache"]]
    shape = (pages, page, kv, d)
    st["k_exps"] = st["v_exps"] = None
    for name in ("k", "v"):
        pool = torch.empty(shape, dtype=kind, device=dev)
        exps = None if case["cache"] == "bf16" else torch.empty(shape[:3], dtype=torch.uint8, device=dev)
        for p0 in range(0, pages, max(1, 65536 // page)):
            p1 = min(pages, p0 + max(1, 65536 // page))
            x = _tokens((p1 - p0) * page, kv, d, g, dev)
            if exps is None:
                pool[p0:p1] = x.view(p1 - p0, page, kv, d).to(kind)
            else:
                q, e = _quantise(x, case["cache"])
                pool[p0:p1] = q.view(p1 - p0, page, kv, d)
                exps[p0:p1] = e.view(p1 - p0, page, kv)
        # Slots behind the lanes' last tokens hold what an earlier request left there.
        for b in range(lanes):
            if totals[b] % page:
                pool[tables[b, owned[b] - 1].long(), totals[b] % page:] = 100 if case["cache"] == "int8" else 400.0
        st[name + "_pool"], st[name + "_exps"] = pool, exps
    if case["op"] == "attend":
        hq = case["hq"]
        st["q"] = (2.0 * torch.randn(rows, hq, d, generator=g, device=dev)).to(torch.bfloat16)
        st["out"] = torch.zeros(rows, hq, d, dtype=torch.bfloat16, device=dev)
        st["lse"] = torch.zeros(rows, hq, device=dev) if case["lse"] else None
        st["window"], st["scale"] = case["window"], d ** -0.5
        if own:
            import speculative_decoding_verify_bf16_gb300 as sv
            st["workspace"] = sv.new_paged_attention_workspace(hq, kv, d, st["max_len"], dev)
    else:
        dtype = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        st["k"], st["v"] = (_tokens(rows, kv, d, g, dev).to(dtype) for _ in range(2))
        st["k_out"], st["v_out"] = torch.zeros_like(st["k"]), torch.zeros_like(st["v"])
    if own:
        import speculative_decoding_verify_bf16_gb300 as sv
        st["cache"] = sv.PagedCache(st["k_pool"], st["v_pool"], st["k_exps"], st["v_exps"])
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    if own:
        return _own(state)
    if state["op"] == "attend":
        return _plain_attend(state)
    return _plain_store_read(state)


def _own(s):
    import speculative_decoding_verify_bf16_gb300 as sv
    lanes = (s["cache"], s["tables"], s["cached"], s["offsets"])
    if s["op"] == "attend":
        sv.spec_paged_attention(s["q"], *lanes, s["out"], s["max_len"], scale=s["scale"], window=s["window"], lse=s["lse"],
                                lane_status=s["status"], max_context=s["max_context"], workspace=s["workspace"])
        return {"out": s["out"], "lse": s["lse"], "status": s["status"]}
    if s["op"] == "store":
        sv.spec_cache_write(*lanes, s["k"], s["v"], s["max_len"], lane_status=s["status"])
    sv.spec_cache_read(*lanes, s["k_out"], s["v_out"], s["max_len"], lane_status=s["status"])
    return {"k": s["k_out"], "v": s["v_out"], "status": s["status"]}


def _quantise(x, kind):
    """8-bit values of [n, heads, d] and their exponents' bytes, [n, heads]."""
    top, whole, fraction = FORMATS[kind]
    m, e = torch.frexp(x.float().abs().amax(-1))
    e = e - whole + (m > fraction).to(e.dtype)  # the least e with top * 2^e >= the largest
    e = torch.where(m > 0, e, torch.full_like(e, LEAST)).clamp(LEAST, MOST)
    y = (x.float() * _power(-e)[..., None]).clamp(-top, top)
    y = y.round().to(torch.int8) if kind == "int8" else y.to(torch.float8_e4m3fn)
    return y, (e + 127).to(torch.uint8)


def _power(e):
    """2^e in fp32, exactly (int32, within the range of normal numbers)."""
    return ((e + 127) << 23).view(torch.float32)


def _slots(s):
    """Of each packed row: its page and its place there."""
    off = s["offsets"].long()
    row = torch.arange(s["k"].shape[0], device=off.device)
    lane = (row[:, None] >= off[1:]).sum(1)
    at = s["cached"].long()[lane] + row - off[lane]
    return s["tables"].long()[lane, at // s["page"]], at % s["page"]


def _values(pool, exps):
    """What stored numbers stand for, in fp32."""
    x = pool.float()
    return x if exps is None else x * _power(exps.int() - 127)[..., None]


def _plain_store_read(s):
    page, at = _slots(s)
    out = {}
    for n in ("k", "v"):
        pool, exps = s[n + "_pool"], s[n + "_exps"]
        if s["op"] == "store":
            q, e = _quantise(s[n], s["kind"])
            pool.view(torch.uint8)[page, at] = q.view(torch.uint8)
            exps[page, at] = e
        out[n] = _values(pool.view(torch.uint8)[page, at].view(pool.dtype), exps[page, at]).to(s[n].dtype)
    out["status"] = torch.zeros_like(s["status"])
    return out


def _plain_attend(s):
    off, cached = s["offsets"].long(), s["cached"].long()
    lanes, cols, span = off.numel() - 1, s["max_len"], s["max_context"]
    rows, hq, d = s["q"].shape
    kv = s["k_pool"].shape[2]
    n = off[1:] - off[:-1]
    i, j = torch.arange(cols, device=off.device), torch.arange(span, device=off.device)
    held = j < (cached + n)[:, None]
    page = torch.where(held, s["tables"].long()[:, j // s["page"]], torch.zeros_like(j))

    def gather(pool, exps):  # [lanes, span, kv, d] -> [lanes, kv, span, d]
        x = pool.view(torch.uint8 if exps is not None else pool.dtype)[page, j % s["page"]].view(pool.dtype)
        x = _values(x, None if exps is None else exps[page, j % s["page"]])
        return torch.where(held[:, :, None, None], x, torch.zeros((), device=x.device)).transpose(1, 2)

    real = i < n[:, None]
    q = s["q"].float()[torch.where(real, off[:-1, None] + i, torch.zeros_like(i))] * s["scale"]
    q = q.view(lanes, cols, kv, hq // kv, d).permute(0, 2, 3, 1, 4).reshape(lanes, kv, hq // kv * cols, d)
    scores = (q @ gather(s["k_pool"], s["k_exps"]).transpose(-1, -2)).view(lanes, kv, hq // kv, cols, span)
    last = cached[:, None] + i  # the last position that a column sees
    seen = j <= last[:, :, None]
    if s["window"]:
        seen &= j > last[:, :, None] - s["window"]
    scores.masked_fill_(~seen[:, None, None], float("-inf"))
    m = scores.amax(-1, keepdim=True)
    scores = scores.sub_(m).exp_()
    total = scores.sum(-1, keepdim=True)
    o = scores.view(lanes, kv, hq // kv * cols, span) @ gather(s["v_pool"], s["v_exps"])
    o = o.view(lanes, kv, hq // kv, cols, d) / total
    row = torch.arange(rows, device=off.device)
    lane = (row[:, None] >= off[1:]).sum(1)
    o = o[lane, :, :, row - off[lane]].reshape(rows, hq, d).to(torch.bfloat16)
    lse = None
    if s["lse"] is not None:
        lse = (m + total.log())[..., 0][lane, :, :, row - off[lane]].reshape(rows, hq)
    return {"out": o, "lse": lse, "status": torch.zeros_like(s["status"])}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    status = torch.zeros(case["lanes"], dtype=torch.int32, device=s["status"].device)
    if case["op"] == "store":
        return {n: _rounded(s[n].double(), case["cache"]) for n in ("k", "v")} | {"status": status}
    lens, before = _lens(case)
    lane_values = lambda n, b, count: _stretch(s, n, b, 0, count)  # noqa: E731
    if case["op"] == "read":
        whole = lambda n: torch.cat([_stretch(s, n, b, c, c + m) for b, (m, c) in enumerate(zip(lens, before))])  # noqa: E731
        return {"k": whole("k"), "v": whole("v"), "status": status}
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=status.device)
    lse = None if s["lse"] is None else torch.zeros(s["lse"].shape, dtype=torch.float64, device=status.device)
    per, first = case["hq"] // case["kv"], 0
    for b, (n, c) in enumerate(zip(lens, before)):
        if n == 0:
            continue
        K, V = lane_values("k", b, n + c), lane_values("v", b, n + c)
        distance = torch.arange(c, c + n, device=status.device)[:, None] - torch.arange(c + n, device=status.device)
        hidden = distance < 0
        if case["window"]:
            hidden |= distance >= case["window"]
        for h in range(case["hq"]):
            x = torch.mm(s["q"][first:first + n, h].double(), K[:, h // per].T) / math.sqrt(case["d"])
            x[hidden] = -math.inf
            z = torch.logsumexp(x, 1)
            if lse is not None:
                lse[first:first + n, h] = z
            out[first:first + n, h] = torch.mm((x - z[:, None]).exp(), V[:, h // per])
        first += n
    return {"out": out, "lse": lse, "status": status}


def _stretch(s, n, b, j0, j1):
    """Tokens j0 .. j1 - 1 of lane b in 64 bits, [tokens, heads, d]."""
    j = torch.arange(j0, j1, device=s["status"].device)
    where = s["tables"][b].long()[j // s["page"]] * s["page"] + j % s["page"]
    x = s[n + "_pool"].flatten(0, 1)
    x = x.view(torch.uint8)[where].view(x.dtype) if s[n + "_exps"] is not None else x[where]
    x = x.double()
    return x if s[n + "_exps"] is None else _scaled(x, s[n + "_exps"].flatten(0, 1)[where].long()[..., None] - 127)


def _scaled(x, e):
    """x * 2^e in 64 bits."""
    return x * torch.bitwise_left_shift(e + 1023, 52).view(torch.float64)


def _rounded(x, kind):
    """[n, heads, d] rounded to the 8-bit type under the least power of two that holds the
    largest number."""
    top = FORMATS[kind][0]
    m, e = torch.frexp(x.abs().amax(-1, keepdim=True) / top)
    e = torch.where(m == 0.5, e - 1, e)
    e = torch.where(m == 0, LEAST, e).long().clamp(LEAST, MOST)
    y = _scaled(x, -e)
    if kind == "int8":
        y = torch.round(y)
    else:  # three bits behind the leading one, which is 2^-6 at least
        step = torch.frexp(y.abs().clamp_min(2.0 ** -6))[1].long() - 4
        y = _scaled(torch.round(_scaled(y, -step)), step)
    return _scaled(y, e)
