"""The attention's check over 8-bit caches where small weights count.

A weight enters the second product as the fp16 number nearest to 2^(x_j + e_j - M), e_j the exponent of position j's
value.  Rounding leaves 2^-11 of it or, where fp16's numbers are 2^-24 apart, 2^-25.  M is 7 less than a
maximum of x_j + e_j at most, so a position's value y_j 2^e_j misses (w_j being the row's weights, their sum 1)

    2^-11 w_j |y_j| 2^e_j  or  2^-32 |y_j| max_i w_i 2^e_i.

The other terms are paged_harness's.
"""

import numpy as np

from oracle import paged
from paged_harness import U


def exponents(L, b):
    """e of lane b's values, [positions, heads]."""
    page, slot = paged.lane_slots(L.host_tables[b], L.page, 0, L.k[b].shape[0])
    return L.cache.v_exps.cpu().numpy()[page, slot].astype(np.int64) - 127


def check_lane(L, b, q, out, lse, window=0, scale=None, floor=2.0 ** -32):
    """Lane b's outputs against the oracle, whatever the sizes of its values."""
    first, n = sum(L.lens[:b]), L.lens[b]
    scale = L.d ** -0.5 if scale is None else scale
    got = out[first:first + n].double().cpu().numpy()
    qs = q[first:first + n].double().cpu().numpy()
    want, z, mag, peak = paged.attention(qs, L.k[b], L.v[b], L.before[b], scale, window)
    count, per = L.before[b] + n, q.shape[1] // L.kv
    E = (2 * (L.d + 2) + 16) * U * peak + 2.0 ** -20 + 2 * count * U
    bound = (2.0 ** -11 + 2 * E[..., None]) * mag + 2.0 ** -8 * np.abs(want)
    power = 2.0 ** exponents(L, b)
    for i in range(n):
        end = L.before[b] + i + 1
        start = max(0, end - window) if window else 0
        for h in range(q.shape[1]):
            w = np.exp(scale * (L.k[b][start:end, h // per] @ qs[i, h]) - z[i, h])
            e = power[start:end, h // per]
            y = np.abs(L.v[b][start:end, h // per]) / e[:, None]
            bound[i, h] += floor * (w * e).max() * y.sum(0)
    assert (np.abs(got - want) <= bound + 1e-30).all(), (b, np.max(np.abs(got - want) / (bound + 1e-30)))
    if lse is not None:
        g = lse[first:first + n].double().cpu().numpy()
        assert (np.abs(g - z) <= E + 2.0 ** -22 * (np.abs(z) + peak)).all(), (b, np.max(np.abs(g - z)))
