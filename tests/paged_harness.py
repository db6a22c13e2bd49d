"""Shared by the tests of the paged cache: caches with lanes in shuffled pages, and the
attention's check against the float64 oracle.

Bounds of an output, with u = 2^-24 and mag the output's sum with |v| for v:

* a score is a sum of dim products in fp32, each addition cut off rather than rounded: within
  2 (dim + 2) u of the sum of magnitudes (peak), then scaled and taken from the maximum, three
  roundings of a number up to peak * log2(e); 2^x adds 2^-22 and its argument's error.  A weight is so within
  E = (2 (dim + 2) + 16) u peak + 2^-20 of itself, numerator and denominator both: 2 E mag.
* a weight is rounded once to enter the second product: 2^-8 of itself in bf16, 2^-11 in fp16 (8-bit
  caches), there also 2^-25 at least of the largest w_j 2^e_j.  The sum over n positions adds 2 n u.
* the output's own rounding: 2^-8 of its value.
"""

import numpy as np
import torch

import speculative_decoding_verify_bf16_gb300 as sv
from oracle import paged

DEV = "cuda"
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def offsets_of(lens):
    return torch.tensor(np.cumsum([0] + list(lens)), dtype=torch.int32, device=DEV)


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device=DEV)


class Lanes:
    """Lanes of `before` cached and `lens` new tokens in shuffled pages of a cache whose other
    slots hold NaN (the 8-bit types' largest number with the exponent byte 255)."""

    def __init__(self, lens, before, kind="bf16", kv=2, d=128, page=16, seed=0, layout="slots", spare=3, extra_width=2,
                 k_scale=1.0, v_scale=1.0):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.g, self.lens, self.before, self.kind, self.kv, self.d, self.page = g, list(lens), list(before), kind, kv, d, page
        totals = [n + c for n, c in zip(lens, before)]
        need = [-(-t // page) for t in totals]
        pages = sum(need) + spare
        dtype = TYPES[kind]
        if layout == "heads":  # [pages, heads, slots, d]
            k, v = (torch.zeros(pages, kv, page, d * dtype.itemsize, dtype=torch.uint8, device=DEV).view(dtype).transpose(1, 2)
                    for _ in range(2))
        elif layout == "joined":  # keys and values of a page side by side
            both = torch.zeros(pages, page, 2, kv, d * dtype.itemsize, dtype=torch.uint8, device=DEV).view(dtype)
            k, v = both[:, :, 0], both[:, :, 1]
        else:
            k, v = (torch.zeros(pages, page, kv, d * dtype.itemsize, dtype=torch.uint8, device=DEV).view(dtype) for _ in range(2))
        ek = ev = None
        if kind == "bf16":
            k.fill_(float("nan")), v.fill_(float("nan"))
        else:
            fill = 0x7E if kind == "e4m3" else 127
            k.view(torch.uint8).fill_(fill), v.view(torch.uint8).fill_(fill)
            if layout == "heads":
                ek, ev = (torch.full((pages, kv, page), 255, dtype=torch.uint8, device=DEV).transpose(1, 2) for _ in range(2))
            else:
                ek, ev = (torch.full((pages, page, kv), 255, dtype=torch.uint8, device=DEV) for _ in range(2))
        self.cache = sv.PagedCache(k, v, ek, ev)
        order = torch.randperm(pages, generator=g, device=DEV).cpu().numpy()
        width = max(need + [0]) + extra_width
        tables = np.full((len(lens), width), -7, np.int32)
        at = 0
        for b, n in enumerate(need):
            tables[b, :n] = order[at:at + n]
            at += n
        self.host_tables = tables
        self.tables = torch.tensor(tables, device=DEV)
        self.cached, self.offsets = i32(before), offsets_of(lens)
        self.max_len = max(lens) if len(lens) else 0
        # every position of every lane, keys and values as they will be stored
        self.k, self.v = [], []  # float64 [total, kv, d] a lane
        for b, t in enumerate(totals):
            for name, to, scale in (("k", self.k, k_scale), ("v", self.v, v_scale)):
                x = torch.randn(t, kv, d, generator=g, device=DEV) * scale
                x *= torch.exp(0.5 * torch.randn(t, kv, 1, generator=g, device=DEV))
                to.append(self.put(name, b, 0, x.to(torch.bfloat16)))

    def put(self, name, b, first, x):
        """x [n, kv, d] into lane b's slots from position `first`, by the oracle's rounding; the
        values that it then holds."""
        page, slot = paged.lane_slots(self.host_tables[b], self.page, first, x.shape[0])
        page, slot = torch.tensor(page, device=DEV).long(), torch.tensor(slot, device=DEV).long()
        pool = getattr(self.cache, name)
        if self.kind == "bf16":
            pool[page, slot] = x.to(torch.bfloat16)
            return x.to(torch.bfloat16).double().cpu().numpy()
        y, byte = paged.quantise(x.double().cpu().numpy(), self.kind)
        z = torch.tensor(np.nan_to_num(y), device=DEV).float().to(TYPES[self.kind])
        pool.view(torch.uint8)[page, slot] = z.view(torch.uint8)
        getattr(self.cache, name + "_exps")[page, slot] = torch.tensor(byte, device=DEV).to(torch.uint8)
        return paged.values(y, byte)

    def queries(self, hq, scale=1.0):
        return (torch.randn(sum(self.lens), hq, self.d, generator=self.g, device=DEV) * scale).to(torch.bfloat16)

    def where(self):
        return self.cache, self.tables, self.cached, self.offsets


def attend(L, q, window=0, scale=None, workspace=None, lse=True, status=None, out=None, stream=None, max_context=0):
    rows, hq = q.shape[:2]
    out = torch.full_like(q, 7.0) if out is None else out
    z = torch.full((rows, hq), 7.0, device=DEV) if lse else None
    status = torch.zeros(len(L.lens), dtype=torch.int32, device=DEV) if status is None else status
    sv.spec_paged_attention(q, *L.where(), out, L.max_len, scale=scale, window=window, lse=z, lane_status=status,
                            max_context=max_context, workspace=workspace, stream=stream)
    return out, z, status


def check_lane(L, b, q, out, lse, window=0, scale=None):
    """Lane b's outputs against the oracle; the squared errors and values for a mean."""
    first, n = sum(L.lens[:b]), L.lens[b]
    scale = L.d ** -0.5 if scale is None else scale
    got = out[first:first + n].double().cpu().numpy()
    want, z, mag, peak = paged.attention(q[first:first + n].double().cpu().numpy(), L.k[b], L.v[b], L.before[b], scale, window)
    count = L.before[b] + n
    E = (2 * (L.d + 2) + 16) * U * peak + 2.0 ** -20 + 2 * count * U
    half = 2.0 ** -8 if L.kind == "bf16" else 2.0 ** -11
    bound = (half + 2 * E[..., None]) * mag + 2.0 ** -8 * np.abs(want)
    if L.kind != "bf16":  # weights too small for fp16's normal numbers
        bound += count * 2.0 ** -25 * 2 * np.abs(L.v[b]).max()
    assert (np.abs(got - want) <= bound + 1e-30).all(), (b, np.max(np.abs(got - want) / (bound + 1e-30)))
    if lse is not None:
        g = lse[first:first + n].double().cpu().numpy()
        assert (np.abs(g - z) <= E + 2.0 ** -22 * (np.abs(z) + peak)).all(), (b, np.max(np.abs(g - z)))
    return ((got - want) ** 2).sum(), (want ** 2).sum()


def check(lens, before, hq=4, window=0, scale=None, q_scale=1.0, workspace=None, **kw):
    L = Lanes(lens, before, **kw)
    q = L.queries(hq, q_scale)
    out, lse, status = attend(L, q, window, scale, workspace)
    torch.cuda.synchronize()
    assert status.tolist() == [0] * len(lens)
    sums = np.array([check_lane(L, b, q, out, lse, window, scale) for b in range(len(lens)) if lens[b]]).reshape(-1, 2).sum(0)
    if q.numel() >= 4096:  # roundings are independent: 2^-8 / sqrt(7) of the values each, at most two of them
        assert sums[0] <= (2.0 ** -8 if L.kind == "bf16" else 2.0 ** -9) ** 2 * sums[1]
    return L, q, out, lse
