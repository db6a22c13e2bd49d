"""Pins of the oracle's linear attention and log probabilities (no GPU needed)."""

import numpy as np
import pytest
from scipy.special import log_softmax
from scipy.stats import entropy as scipy_entropy

from oracle.linear import linear_attention
from oracle.logprobs import token_logprobs


def test_logprobs_match_scipy():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(6, 50)) * 3
    x[2, 5:30] = -np.inf
    T = np.array([0.0, 0.7, 1.3, -1.0, 0.2, 1.0])
    tok = rng.integers(0, 5, 6)
    status, lp, ent, ids, alt = token_logprobs(x, tok, T, top=4)
    assert (status == 0).all()
    for r in range(6):
        z = x[r] / (T[r] if T[r] > 0 else 1.0)
        ref = log_softmax(z)
        np.testing.assert_allclose(lp[r], ref[tok[r]], rtol=1e-12)
        np.testing.assert_allclose(ent[r], scipy_entropy(np.exp(ref)), rtol=1e-12)
        np.testing.assert_allclose(alt[r], np.sort(ref)[::-1][:4], rtol=1e-12)
        np.testing.assert_allclose(ref[ids[r]], alt[r], rtol=1e-12)


def test_logprobs_ties_skips_and_failures():
    x = np.zeros((6, 4))
    x[2, 1] = np.nan
    x[3] = -np.inf
    x[4, 0] = np.inf
    status, lp, ent, ids, alt = token_logprobs(x, [0, -1, 0, 0, 0, 4], None, top=6)
    assert status.tolist() == [0, 0, 4, 4, 4, 5]
    assert ids[0].tolist() == [0, 1, 2, 3, -1, -1] and (alt[0, 4:] == -np.inf).all()
    np.testing.assert_allclose(lp[0], -np.log(4))
    np.testing.assert_allclose(ent[0], np.log(4))
    assert lp[1] == 0 and (ids[1:] == -1).all() and np.isnan(lp[2:]).all()


@pytest.mark.parametrize("rep", [1, 2])
def test_linear_attention_equals_the_decay_matrix_form(rep):
    """o_i = scale (e^{G_i} q_i S_0 + sum_{j <= i} e^{G_i - G_j} (q_i . k_j) v_j)."""
    rng = np.random.default_rng(2)
    n, hk, dk, dv = 9, 2, 5, 4
    hv = hk * rep
    q, k = rng.normal(size=(2, n, hk, dk))
    v, g = rng.normal(size=(n, hv, dv)), -rng.random((n, hv))
    S0 = rng.normal(size=(2, hv, dk, dv))
    out, final, snaps, _, _ = linear_attention(q, k, v, g, [0, 0, n], S0, 0.5)
    np.testing.assert_array_equal(final[0], S0[0])  # an empty lane
    for h in range(hv):
        G = np.cumsum(g[:, h])
        L = np.tril(np.exp(G[:, None] - G[None, :]))
        want = 0.5 * (np.exp(G)[:, None] * (q[:, h // rep] @ S0[1, h]) + (q[:, h // rep] @ k[:, h // rep].T * L) @ v[:, h])
        np.testing.assert_allclose(out[:, h], want, rtol=1e-10, atol=1e-12)
    np.testing.assert_array_equal(snaps[1][-1], final[1])


def test_linear_attention_reset_forgets():
    rng = np.random.default_rng(3)
    q, k, v = rng.normal(size=(3, 4, 1, 3))
    g = np.zeros((4, 1))
    g[2] = -np.inf
    full = linear_attention(q, k, v, g, [0, 4])
    tail = linear_attention(q[2:], k[2:], v[2:], np.zeros((2, 1)), [0, 2])
    np.testing.assert_array_equal(full[0][2:], tail[0])
    np.testing.assert_array_equal(full[1], tail[1])
