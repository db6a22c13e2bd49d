"""Log probabilities of given tokens in float64, with entropy and alternatives."""

import numpy as np

from .verify import STATUS_NONFINITE, STATUS_OK, STATUS_TOKEN_RANGE


def token_logprobs(logits, tokens, temperatures=None, top=0):
    """Per row: (status, log p(token), entropy, ids [top], log p of the ids).

    A negative token asks for nothing (zeros and ids -1); a failed row gives
    NaN and ids -1; ids past the vocabulary are -1 at -inf."""
    x = np.asarray(logits, np.float64)
    rows, V = x.shape
    status = np.full(rows, STATUS_OK, np.int32)
    lp, ent = np.zeros(rows), np.zeros(rows)
    ids, alt = np.full((rows, top), -1, np.int32), np.zeros((rows, top))
    for r in range(rows):
        tok = int(tokens[r])
        if tok < 0:
            continue
        if tok >= V:
            status[r] = STATUS_TOKEN_RANGE
        elif np.isnan(x[r]).any() or (x[r] == np.inf).any() or (x[r] == -np.inf).all():
            status[r] = STATUS_NONFINITE
        if status[r] != STATUS_OK:
            lp[r] = ent[r] = np.nan
            alt[r] = np.nan
            continue
        T = 1.0 if temperatures is None or not temperatures[r] > 0 else float(temperatures[r])
        z = x[r] / T
        z = z - z.max()
        e = np.exp(z)
        logp = z - np.log(e.sum())
        p = e / e.sum()
        lp[r] = logp[tok]
        ent[r] = -np.sum(p[p > 0] * logp[p > 0])
        order = np.argsort(-x[r], kind="stable")[:top]
        ids[r, :len(order)], alt[r, :len(order)] = order, logp[order]
        alt[r, len(order):] = -np.inf
    return status, lp, ent, ids, alt
