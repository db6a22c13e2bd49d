"""Workloads of the operators around a verify round of a recurrent target.

Three operators, each with listed cases and drawn ones of the same ranges:

  logprobs  log probabilities of given tokens, with the row's entropy and its
            top alternatives, over logit rows as a verify round brings them
  prefill   linear attention with a decay for each head over whole prompts,
            from and to the lanes' recurrent states
  verify    the same recurrence over one to sixteen columns a lane, with the
            state after every column staged for the commit

``prepare`` makes what a serving program holds before the call, ``run`` makes
one pass (``own`` False: elementary torch operations in 32 bits; True: the
library's calls), ``exact`` states the definitions again in 64 bits and
``work`` counts the bytes and operations that a pass cannot do without.
"""

import math
import random

import torch

own = False

SKIP = -1  # a token slot that holds no committed token: its row is not asked for


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # The smallest round: one lane, three drafts, a toy vocabulary, fp32.
        dict(name="logprobs_4x1024_f32", op="logprobs", rows=4, V=1024, pad=0, dtype="f32", top=5,
             temps=False, skip=0.0, masked=0.0, pick=1),
        # One decoding request with a large vocabulary: a single row, latency counts.
        dict(name="logprobs_1x262144", op="logprobs", rows=1, V=262144, pad=0, dtype="bf16", top=5,
             temps=False, skip=0.0, masked=0.0, pick=2),
        # A round of 8 lanes x 8 columns, every row asked for, the most alternatives.
        dict(name="logprobs_64x151936_top20", op="logprobs", rows=64, V=151936, pad=0, dtype="bf16", top=20,
             temps=True, skip=0.0, masked=0.0, pick=3),
        # fp32 logits at an odd vocabulary and row stride, most of it masked by a grammar.
        dict(name="logprobs_96x100003_f32_masked", op="logprobs", rows=96, V=100003, pad=2, dtype="f32", top=8,
             temps=True, skip=0.0, masked=0.9, pick=4),
        # The ragged 128-lane round: the committed tokens' rows of 576.
        dict(name="logprobs_576x262144_ragged", op="logprobs", rows=576, V=262144, pad=0, dtype="bf16", top=5,
             temps=True, skip=0.4, masked=0.0, pick=5),
        # A short prompt of one request: latency counts.
        dict(name="prefill_1x200", op="prefill", lanes=1, lo=200, hi=200, hk=16, hv=16, d=128, fresh=True,
             resets=0.0, pick=6),
        # A long prompt of one request: few heads, a long axis.
        dict(name="prefill_1x16384", op="prefill", lanes=1, lo=16384, hi=16384, hk=16, hv=16, d=128, fresh=False,
             resets=0.0, pick=7),
        # A batch of prompts of mixed lengths (one of them empty), two value heads to a
        # key head, packed documents whose borders reset the state.
        dict(name="prefill_24x0to3000_grouped", op="prefill", lanes=24, lo=0, hi=3000, hk=8, hv=16, d=128,
             fresh=False, resets=0.002, pick=8),
        # The largest: 64 lanes of 2048 tokens.
        dict(name="prefill_64x2048", op="prefill", lanes=64, lo=2048, hi=2048, hk=16, hv=16, d=128, fresh=True,
             resets=0.0, pick=9),
        # Single-token decoding of one request.
        dict(name="verify_1x1", op="verify", lanes=1, cols=1, full=True, hk=16, hv=16, d=128, dtype="bf16", pick=10),
        # A round of 8 lanes x 8 columns, fp32 activations, grouped heads.
        dict(name="verify_8x8_f32", op="verify", lanes=8, cols=8, full=True, hk=8, hv=16, d=128, dtype="f32", pick=11),
        # One layer of the 64-lane round with commit: up to four columns a lane.
        dict(name="verify_64x4_ragged", op="verify", lanes=64, cols=4, full=False, hk=16, hv=16, d=128, dtype="bf16",
             pick=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["logprobs", "prefill", "verify"])
    pick = rng.randrange(1, 1 << 30)
    if op == "logprobs":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        V = _log_int(rng, 900, 262144)
        rows = _log_int(rng, 1, min(576, max(1, 576 * 262144 // (V * (2 if dtype == "f32" else 1)))))
        return dict(op=op, rows=rows, V=V, pad=rng.choice([0, 0, 1, 3, 8]), dtype=dtype, top=rng.randint(1, 20),
                    temps=rng.random() < 0.5, skip=rng.choice([0.0, 0.0, 0.3]), masked=rng.choice([0.0, 0.0, 0.5, 0.95]),
                    pick=pick)
    if op == "prefill":
        lanes = _log_int(rng, 1, 64)
        hi = _log_int(rng, 20, min(16384, 131072 // lanes))
        lo = hi if rng.random() < 0.3 else rng.randint(0, hi)
        hv = rng.choice([4, 8, 16])
        return dict(op=op, lanes=lanes, lo=lo, hi=hi, hk=hv // rng.choice([1, 2]), hv=hv, d=128,
                    fresh=rng.random() < 0.5, resets=rng.choice([0.0, 0.0, 0.005]), pick=pick)
    lanes = _log_int(rng, 1, 64)
    cols = rng.randint(1, 8 if lanes <= 32 else 4)
    hv = rng.choice([4, 8, 16])
    return dict(op=op, lanes=lanes, cols=cols, full=rng.random() < 0.5, hk=hv // rng.choice([1, 2]), hv=hv, d=128,
                dtype=rng.choice(["bf16", "f32"]), pick=pick)


def _lens(case):
    """The lanes' lengths in tokens (part of the case, not of the seed)."""
    rng = random.Random(case["pick"])
    lanes = case["lanes"]
    if case["op"] == "verify":
        return [case["cols"] if case["full"] else rng.randint(1, case["cols"]) for _ in range(lanes)]
    lens = [rng.randint(case["lo"], case["hi"]) for _ in range(lanes)]
    lens[-1] = case["hi"]
    if lanes > 2 and case["lo"] == 0:
        lens[1] = 0
    return lens


def _asked(case):
    """Which rows of a logprobs case hold a token."""
    rng = random.Random(case["pick"])
    return [rng.random() >= case["skip"] for _ in range(case["rows"])]


def work(case):
    if case["op"] == "logprobs":
        n = sum(_asked(case))
        size = 2 if case["dtype"] == "bf16" else 4
        per_row = 4 + 4 + 4 + 4 + 8 * case["top"] + (4 if case["temps"] else 0)
        # each logit: scaled, exponential, two sums with a product, two comparisons
        return {"bytes": n * case["V"] * size + case["rows"] * per_row, "flops": 7 * n * case["V"]}
    lens = _lens(case)
    tokens, d, hk, hv = sum(lens), case["d"], case["hk"], case["hv"]
    size = 4 if case.get("dtype") == "f32" else 2
    rows = tokens * (2 * hk * d * size + 2 * hv * d * size + 4 * hv)
    state = hv * d * d * 4
    # each token and head: decay, outer product and matrix-vector product
    flops = tokens * hv * (5 * d * d)
    if case["op"] == "prefill":
        return {"bytes": rows + case["lanes"] * state * (1 if case["fresh"] else 2), "flops": flops}
    return {"bytes": rows + state * (case["lanes"] + tokens), "flops": flops}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 1000003 + case["pick"])
    if case["op"] == "logprobs":
        return _prepare_logprobs(case, g, dev)
    return _prepare_linear(case, g, dev)


def _prepare_logprobs(case, g, dev):
    rows, V = case["rows"], case["V"]
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    buf = torch.empty(rows, V + case["pad"], dtype=dtype, device=dev)
    low = torch.finfo(dtype).min
    for r0 in range(0, rows, 64):  # N(0, 2) with one token 8 above, masked tokens at -inf or the type's lowest value
        n = min(64, rows - r0)
        x = torch.randn(n, V, generator=g, device=dev) * 2.0
        hot = torch.randint(0, V, (n, 1), generator=g, device=dev)
        x.scatter_add_(1, hot, torch.full((n, 1), 8.0, device=dev))
        if case["masked"]:
            gone = torch.rand(n, V, generator=g, device=dev) < case["masked"]
            gone.scatter_(1, hot, False)
            fill = torch.where(torch.arange(n, device=dev) % 2 == 0, float("-inf"), low)[:, None]
            x = torch.where(gone, fill, x)
        buf[r0:r0 + n, :V] = x.to(dtype)
    buf[:, V:] = 1e4  # row padding that must never be read
    logits = buf[:, :V]
    best = torch.cat([logits[r0:r0 + 64].float().argmax(1) for r0 in range(0, rows, 64)])
    other = torch.randint(0, V, (rows,), generator=g, device=dev)
    # Most rows ask for their likeliest token (a grammar's always do), the rest for any.
    likely = torch.rand(rows, generator=g, device=dev) < (1.0 if case["masked"] else 0.8)
    tokens = torch.where(likely, best, other).to(torch.int32)
    tokens = torch.where(torch.tensor(_asked(case), device=dev), tokens, torch.full_like(tokens, SKIP))
    temps = None
    if case["temps"]:  # half the rows greedy (0: as they are), half at U[0.3, 1.2]
        temps = 0.3 + 0.9 * torch.rand(rows, generator=g, device=dev)
        temps[::2] = 0.0
    f32, i32 = dict(dtype=torch.float32, device=dev), dict(dtype=torch.int32, device=dev)
    return dict(op="logprobs", logits=logits, tokens=tokens, temps=temps, top=case["top"],
                logprobs=torch.empty(rows, **f32), entropy=torch.empty(rows, **f32),
                top_ids=torch.empty(rows, case["top"], **i32), top_logprobs=torch.empty(rows, case["top"], **f32),
                row_status=torch.empty(rows, **i32))


def _prepare_linear(case, g, dev):
    lens = _lens(case)
    lanes, tokens, hk, hv, d = case["lanes"], sum(lens), case["hk"], case["hv"], case["d"]
    dtype = torch.float32 if case.get("dtype") == "f32" else torch.bfloat16

    def unit(h):
        x = torch.randn(tokens, h, d, generator=g, device=dev)
        return (x / x.norm(dim=-1, keepdim=True)).to(dtype)

    q, k = unit(hk), unit(hk)
    v = torch.randn(tokens, hv, d, generator=g, device=dev).to(dtype)
    # A rate for each head from slow to fast, times a gate for each token.
    rate = torch.logspace(-3, 0, hv, device=dev)
    decay = -rate * torch.nn.functional.softplus(torch.randn(tokens, hv, generator=g, device=dev))
    if case.get("resets"):
        border = torch.rand(tokens, 1, generator=g, device=dev) < case["resets"]
        decay = torch.where(border, float("-inf"), decay)
    offsets = torch.tensor([sum(lens[:i]) for i in range(lanes + 1)], dtype=torch.int32, device=dev)
    st = dict(op=case["op"], q=q, k=k, v=v, log_decay=decay.contiguous(), offsets=offsets, scale=d ** -0.5,
              max_len=max(lens), out=torch.zeros(tokens, hv, d, dtype=dtype, device=dev),
              status=torch.zeros(lanes, dtype=torch.int32, device=dev))
    state = None
    if not case.get("fresh"):
        state = torch.randn(lanes, hv, d, d, generator=g, device=dev) * 0.3
    st["state"] = state
    if case["op"] == "prefill":
        st["state_out"] = torch.zeros(lanes, hv, d, d, device=dev)
    else:
        st["staged"] = torch.zeros(lanes, case["cols"], hv, d, d, device=dev)
        st["cols"], st["full"] = case["cols"], all(n == case["cols"] for n in lens)
    if own and case["op"] == "prefill":
        import speculative_decoding_verify_bf16_gb300 as sv
        st["workspace"] = sv.new_linear_workspace(lanes, hv, d, d, max(lens), dev)
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    op = state["op"]
    if own:
        import speculative_decoding_verify_bf16_gb300 as sv
        if op == "logprobs":
            sv.spec_token_logprobs(state["logits"], state["tokens"], state["logprobs"], entropy=state["entropy"],
                                   top_ids=state["top_ids"], top_logprobs=state["top_logprobs"],
                                   temperatures=state["temps"], row_status=state["row_status"])
            return {n: state[n] for n in ("logprobs", "entropy", "top_ids", "top_logprobs", "row_status")}
        if op == "prefill":
            sv.spec_linear_prefill(state["q"], state["k"], state["v"], state["log_decay"], state["offsets"],
                                   state["state"], state["out"], state["state_out"], state["max_len"],
                                   scale=state["scale"], lane_status=state["status"], workspace=state["workspace"])
            return {"out": state["out"], "state": state["state_out"], "status": state["status"]}
        sv.spec_linear_verify(state["q"], state["k"], state["v"], state["log_decay"], state["offsets"], state["state"],
                              state["staged"], state["out"], scale=state["scale"], lane_status=state["status"])
        return {"out": state["out"], "staged": state["staged"], "status": state["status"]}
    if op == "logprobs":
        return _plain_logprobs(state)
    if op == "prefill":
        return _plain_prefill(state)
    return _plain_verify(state)


def _plain_logprobs(s):
    x = s["logits"].float()
    rows, V = x.shape
    tok = s["tokens"].long()
    asked = tok >= 0
    x = x + 0.0  # -0 counts as +0
    # Distinct integer keys whose order is (value, then lower index first).
    bits = x.view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    keys = order * (1 << 32) + ((1 << 32) - 1 - torch.arange(V, device=x.device))
    top = torch.topk(keys, s["top"], dim=1).values
    ids = (1 << 32) - 1 - (top & ((1 << 32) - 1))
    if s["temps"] is not None:
        x = x / torch.where(s["temps"] > 0, s["temps"], torch.ones_like(s["temps"]))[:, None]
    z = x - x.max(dim=1, keepdim=True).values
    e = z.exp()
    total = e.sum(1)
    lse = total.log()
    entropy = lse - torch.where(e > 0, e * z, torch.zeros_like(z)).sum(1) / total
    logp = z.gather(1, tok.clamp_min(0)[:, None])[:, 0] - lse
    top_logp = z.gather(1, ids) - lse[:, None]
    zero = torch.zeros_like(logp)
    return {"logprobs": torch.where(asked, logp, zero), "entropy": torch.where(asked, entropy, zero),
            "top_ids": torch.where(asked[:, None], ids, torch.full_like(ids, SKIP)).to(torch.int32),
            "top_logprobs": torch.where(asked[:, None], top_logp, zero[:, None]),
            "row_status": torch.zeros(rows, dtype=torch.int32, device=x.device)}


def _plain_prefill(s):
    C = 64
    off = s["offsets"].long()
    lanes, hv, d = off.numel() - 1, s["v"].shape[1], s["v"].shape[2]
    n = -(-s["max_len"] // C)
    rep = hv // s["k"].shape[1]
    pos = torch.arange(n * C, device=off.device)
    valid = pos < (off[1:] - off[:-1])[:, None]
    idx = torch.where(valid, off[:-1, None] + pos, torch.zeros_like(pos))

    def lay(x):  # packed [tokens, heads, d] -> [lanes, heads, chunks, C, d]
        y = torch.where(valid[:, :, None, None], x.float()[idx], torch.zeros((), device=x.device))
        if y.shape[2] != hv:
            y = y.repeat_interleave(rep, dim=2)
        return y.permute(0, 2, 1, 3).reshape(lanes, hv, n, C, d)

    q, k, v = lay(s["q"]) * s["scale"], lay(s["k"]), lay(s["v"])
    g = torch.where(valid[:, :, None], s["log_decay"][idx], torch.zeros((), device=off.device))
    g = g.permute(0, 2, 1).reshape(lanes, hv, n, C)
    lower = torch.ones(C, C, dtype=torch.bool, device=off.device).tril()
    strict = lower.tril(-1)
    # between[i, j] = sum of g over j < l <= i
    between = torch.where(strict, g[..., :, None], torch.zeros((), device=off.device)).cumsum(-2)
    weight = torch.where(lower, between.exp(), torch.zeros((), device=off.device))
    out = (q @ k.transpose(-1, -2) * weight) @ v
    from_start = g.cumsum(-1).exp()[..., None]
    to_end = weight[..., -1, :, None]
    S = s["state"]
    if S is None:
        S = torch.zeros(lanes, hv, d, d, device=off.device)
    for c in range(n):
        out[:, :, c] += (q[:, :, c] * from_start[:, :, c]) @ S
        S = S * from_start[:, :, c, -1:] + (k[:, :, c] * to_end[:, :, c]).transpose(-1, -2) @ v[:, :, c]
    row = torch.arange(s["v"].shape[0], device=off.device)
    lane = (row[:, None] >= off[1:]).sum(1)
    out = out.reshape(lanes, hv, n * C, d)[lane, :, row - off[lane]]
    return {"out": out.to(s["out"].dtype), "state": S, "status": torch.zeros(lanes, dtype=torch.int32, device=off.device)}


def _plain_verify(s):
    off = s["offsets"].long()
    lens = off[1:] - off[:-1]
    hv = s["v"].shape[1]
    rep = hv // s["k"].shape[1]
    last = s["v"].shape[0] - 1
    S, staged, out = s["state"], s["staged"], s["out"]
    outs = []
    for j in range(s["cols"]):
        row = (off[:-1] + j).clamp_max(last)
        q, k, v = s["q"][row].float(), s["k"][row].float(), s["v"][row].float()
        if rep > 1:
            q, k = q.repeat_interleave(rep, dim=1), k.repeat_interleave(rep, dim=1)
        S = S * s["log_decay"][row].exp()[:, :, None, None] + k[..., :, None] * v[..., None, :]
        outs.append((q[..., :, None] * S).sum(-2) * s["scale"])
        if s["full"]:
            staged[:, j] = S
        else:
            staged[:, j] = torch.where((j < lens)[:, None, None, None], S, staged[:, j])
    r = torch.arange(last + 1, device=off.device)
    lane = (r[:, None] >= off[1:]).sum(1)
    out.copy_(torch.stack(outs, 1)[lane, r - off[lane]])
    return {"out": out, "staged": staged, "status": torch.zeros_like(s["status"])}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "logprobs":
        return _exact_logprobs(s)
    return _exact_linear(s, case)


def _exact_logprobs(s):
    parts = []
    for r0 in range(0, s["logits"].shape[0], 64):
        x = s["logits"][r0:r0 + 64].double()
        tok = s["tokens"][r0:r0 + 64].long()
        ordered, ids = torch.sort(x, dim=1, descending=True, stable=True)
        ordered, ids = ordered[:, :s["top"]], ids[:, :s["top"]]
        T = torch.ones(x.shape[0], dtype=torch.float64, device=x.device)
        if s["temps"] is not None:
            t = s["temps"][r0:r0 + 64].double()
            T = torch.where(t > 0, t, T)
        logp = torch.log_softmax(x / T[:, None], dim=1)
        H = -torch.xlogy(logp.exp(), logp.exp()).sum(1)
        skip = tok < 0
        given = logp.gather(1, tok.clamp_min(0)[:, None])[:, 0].masked_fill(skip, 0.0)
        alt = logp.gather(1, ids).masked_fill(skip[:, None], 0.0)
        parts.append((given, H.masked_fill(skip, 0.0), ids.masked_fill(skip[:, None], SKIP).to(torch.int32), alt))
    given, H, ids, alt = (torch.cat(p) for p in zip(*parts))
    return {"logprobs": given, "entropy": H, "top_ids": ids, "top_logprobs": alt,
            "row_status": torch.zeros_like(ids[:, 0])}


def _exact_linear(s, case):
    """The recurrence itself, a token of every lane at a time."""
    lens = _lens(case)
    first = [sum(lens[:i]) for i in range(len(lens))]
    hv, d = s["v"].shape[1], s["v"].shape[2]
    group = torch.arange(hv, device=s["v"].device) // (hv // s["k"].shape[1])
    S = torch.zeros(len(lens), hv, d, d, dtype=torch.float64, device=s["v"].device)
    if s["state"] is not None:
        S += s["state"]
    out = torch.zeros(s["v"].shape, dtype=torch.float64, device=S.device)
    staged = s["staged"].double() if case["op"] == "verify" else None
    alive = None
    for t in range(max(lens)):
        now = [b for b, n in enumerate(lens) if n > t]
        if now != alive:
            alive = now
            lane = torch.tensor(now, device=S.device)
            base = torch.tensor([first[b] for b in now], device=S.device)
            part = S if len(now) == len(lens) else None
        rows = base + t
        q, k, v = (s[n][rows].double() for n in "qkv")
        a = s["log_decay"][rows].double().exp()[:, :, None, None]
        x = part if part is not None else S[lane]
        x = torch.einsum("bhi,bhj->bhij", k[:, group], v).add_(x * a)
        out[rows] = torch.einsum("bhi,bhij->bhj", q[:, group], x) * s["scale"]
        if part is not None:
            S = part = x
        else:
            S[lane] = x
        if staged is not None:
            staged[lane, t] = x
    status = torch.zeros(len(lens), dtype=torch.int32, device=S.device)
    if case["op"] == "verify":
        return {"out": out, "staged": staged, "status": status}
    return {"out": out, "state": S, "status": status}
