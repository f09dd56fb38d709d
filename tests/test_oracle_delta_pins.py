"""Pins of the delta-rule oracle (CPU): closed forms that it must meet."""
import numpy as np
import pytest

from oracle import delta_oracle as DO
from oracle import ttt_oracle as O


def _inputs(seed, B=1, Hk=2, Hv=4, N=24, dk=8, dv=6):
    r = np.random.default_rng(seed)
    q, k = r.standard_normal((2, B, Hk, N, dk))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    v = r.standard_normal((B, Hv, N, dv))
    return q, k, v, -r.random((B, Hv, N)), r.random((B, Hv, N))


def test_orthonormal_keys_without_decay_are_linear_attention():
    """Keys that are orthonormal never meet an earlier write: with g = 0 the
    rule is token-causal linear attention with eta = beta."""
    r = np.random.default_rng(0)
    N = dk = 8
    k = np.linalg.qr(r.standard_normal((dk, dk)))[0][None, None]
    q = r.standard_normal((1, 1, N, dk))
    v = r.standard_normal((1, 1, N, 5))
    b = r.random((1, 1, N))
    o, S = DO.delta_rule(q, k, v, np.zeros((1, 1, N)), b, scale=1.0)
    ro, rS = O.linattn_chunked_forward(q, k, v, b, None, 1, 1)
    assert np.allclose(o, ro, atol=1e-12) and np.allclose(S, rS, atol=1e-12)


def test_beta_one_stores_the_value():
    """With beta = 1 and unit keys the state returns v for the key just written."""
    q, k, v, g, _ = _inputs(1)
    q = k
    o, _ = DO.delta_rule(q, k, v, g, np.ones_like(g), scale=1.0)
    assert np.allclose(o, v, atol=1e-12)


def test_chunk_form_equals_the_recurrence():
    """(1 + A)^-1 form of one chunk: A_ij = beta_i e^(G_i - G_j) k_i . k_j."""
    q, k, v, g, b = _inputs(2, Hk=1, Hv=1)
    r = np.random.default_rng(3)
    S0 = r.standard_normal((1, 1, 6, 8))
    o, S = DO.delta_rule(q, k, v, g, b, S0, scale=1.0)
    K, Q, V, G, bb, M = k[0, 0], q[0, 0], v[0, 0], np.cumsum(g[0, 0]), b[0, 0], S0[0, 0]
    D = np.tril(np.exp(np.minimum(G[:, None] - G[None], 0)))
    A = np.tril(bb[:, None] * D * (K @ K.T), -1)
    X = np.linalg.solve(np.eye(len(G)) + A, bb[:, None] * (V - np.exp(G)[:, None] * (K @ M.T)))
    assert np.allclose(o[0, 0], np.exp(G)[:, None] * (Q @ M.T) + (D * (Q @ K.T)) @ X, atol=1e-10)
    assert np.allclose(S[0, 0], np.exp(G[-1]) * M + X.T @ (np.exp(G[-1] - G)[:, None] * K),
                       atol=1e-10)


def test_packed_sequences_equal_single_ones():
    q, k, v, g, b = _inputs(4)
    S0 = np.random.default_rng(5).standard_normal((3, 4, 6, 8))
    o, S = DO.delta_rule(q, k, v, g, b, S0, starts=[2, 9, 9, 20])
    for s, (a, e) in enumerate(((2, 9), (9, 9), (9, 20))):
        cut = [x[:, :, a:e] for x in (q, k, v, g, b)]
        ro, rS = DO.delta_rule(*cut, S0[s:s + 1])
        assert np.array_equal(o[:, :, a:e], ro) and np.array_equal(S[s], rS[0])
    assert np.isnan(o[:, :, :2]).all() and np.isnan(o[:, :, 20:]).all()


@pytest.mark.parametrize("group", [12, 4])
def test_norm_rows_have_unit_mean_square(group):
    y = np.random.default_rng(6).standard_normal((5, 12)) * 7
    r, h = DO.block_norm(y, group=group, eps=0.0, w_next=np.ones(12))
    assert np.allclose((r.reshape(5, -1, group) ** 2).mean(-1), 1)
    assert np.allclose((h ** 2).mean(-1), 1)
