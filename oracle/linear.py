"""Linear attention with a decay for each head, token after token in float64.

S_t = exp(g_t) S_(t-1) + k_t v_t^T and o_t = scale * S_t^T q_t, head h reading
key head h // (v_heads / k_heads).
"""

import numpy as np


def linear_attention(q, k, v, log_decay, offsets, state=None, scale=1.0):
    """q, k [rows, k_heads, dk]; v [rows, v_heads, dv]; log_decay [rows, v_heads];
    offsets [lanes + 1]; state [lanes, v_heads, dk, dv] or None (zeros).

    Returns out [rows, v_heads, dv], the final states, the list of each lane's
    snapshots [count, v_heads, dk, dv], and the magnitudes (out_mag,
    state_mag): the same sums with every term replaced by its absolute value,
    from which error bounds follow."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    g = np.asarray(log_decay, np.float64)
    lanes, hv, dv, dk = len(offsets) - 1, v.shape[1], v.shape[2], k.shape[2]
    rep = hv // k.shape[1]
    group = np.arange(hv) // rep
    S0 = np.zeros((lanes, hv, dk, dv)) if state is None else np.asarray(state, np.float64)
    out = np.zeros(v.shape)
    out_mag = np.zeros(v.shape)
    final, final_mag, snaps = S0.copy(), np.abs(S0), []
    for b in range(lanes):
        S, A = S0[b].copy(), np.abs(S0[b])
        mine = []
        for t in range(int(offsets[b]), int(offsets[b + 1])):
            a = np.exp(g[t])[:, None, None]
            kt, qt = k[t][group], q[t][group]
            S = a * S + kt[:, :, None] * v[t][:, None, :]
            A = a * A + np.abs(kt[:, :, None] * v[t][:, None, :])
            out[t] = scale * np.einsum("hi,hij->hj", qt, S)
            out_mag[t] = abs(scale) * np.einsum("hi,hij->hj", np.abs(qt), A)
            mine.append(S)
        final[b], final_mag[b] = S, A
        snaps.append(np.stack(mine) if mine else np.zeros((0, hv, dk, dv)))
    return out, final, snaps, out_mag, final_mag
