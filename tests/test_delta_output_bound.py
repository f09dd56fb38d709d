"""A bound on bf16 outputs of the delta rule that sees a dropped low part.

With r the exact outputs, x the kernel's before the last rounding and bf16() the
rounding to the nearest bf16 number, |bf16(x) - x| <= |bf16(r) - x|, so
    |bf16(x) - r| <= |bf16(x) - x| + |x - r| <= |bf16(r) - r| + 2 |x - r|.
The chunk form's x is off by the state's own error (3.9e-5, the bound of the
states) and by the pairs of bf16 numbers that the outputs alone use: S, D o QK^T
and X, 2^-17 each, and the low parts' product, 2^-18.  Here, on the CPU: outputs
made with pairs keep to the bound, and ones made with any of the three rounded
to a single bf16 number do not.
"""
import numpy as np
import pytest
import torch

from oracle import delta_oracle as DO

STATE = 3.9e-5
UNROUNDED = STATE + 3 * 2.0 ** -17 + 2.0 ** -18


def bf16(x):
    return torch.from_numpy(np.array(x, dtype=np.float64)).to(torch.bfloat16).double().numpy()


def pair(x):
    hi = bf16(x)
    return hi + bf16(x - hi)


def output_bound(ref):
    """Largest |o - ref| / |ref| of bf16 outputs o."""
    return float(np.linalg.norm(bf16(ref) - ref) / np.linalg.norm(ref)) + 2 * UNROUNDED


def chunk_outputs(q, k, v, g, b, S0, keep):
    """One chunk of the rule: O = scale (e^G Q S^T + (D o Q K^T) X) with `keep`
    applied to S, P = D o Q K^T and X."""
    G = np.cumsum(g)
    D = np.tril(np.exp(np.minimum(G[:, None] - G[None], 0)))
    A = np.tril(b[:, None] * D * (k @ k.T), -1)
    X = np.linalg.solve(np.eye(len(G)) + A, b[:, None] * (v - np.exp(G)[:, None] * (k @ S0.T)))
    P = D * (q @ k.T)
    o = np.exp(G)[:, None] * (q @ keep["S"](S0).T) + keep["P"](P) @ keep["X"](X)
    return o * q.shape[1] ** -0.5


def inputs(seed, N=64, d=128):
    r = np.random.default_rng(seed)
    q, k = (x / np.linalg.norm(x, axis=1, keepdims=True) for x in r.standard_normal((2, N, d)))
    return (bf16(q), bf16(k), bf16(r.standard_normal((N, d))), -0.1 * r.random(N), r.random(N),
            0.3 * r.standard_normal((d, d)))


@pytest.mark.parametrize("seed", range(3))
@pytest.mark.parametrize("single", ["", "S", "P", "X"])
def test_the_bound_sees_each_low_part(single, seed):
    q, k, v, g, b, S0 = inputs(seed)
    ref, _ = DO.delta_rule(*[x[None, None] for x in (q, k, v, g, b)], S0[None, None])
    keep = {n: bf16 if n == single else pair for n in "SPX"}
    o = bf16(chunk_outputs(q, k, v, g, b, S0, keep))
    err = np.linalg.norm(o - ref[0, 0]) / np.linalg.norm(ref)
    assert (err > output_bound(ref)) == bool(single)
