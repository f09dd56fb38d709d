"""The gated delta rule behind strongly forgetting tokens.

Tokens that clear the state (g of -inf, -80, -37) stand right before tokens that
hardly forget: the decays between the latter must not suffer from the large sums
of the former.  One token of a chunk writes behind the strong ones, all others
have beta = 0, so that a final state is one outer product times one decay and
its relative error is that decay's, plus the pairs' roundings: STATE_BF16 of
the neighbouring tests bounds both (a decay in fp32 adds 2^-21 = 5e-7 at most,
16 additions of numbers below 2 and the exponential).
"""
import numpy as np
import pytest
import torch

from tests.gpu_util import f64, lib, rel_l2
from tests.test_gpu_delta_rule import DEV, STATE_BF16, STATE_F32, check, inputs, oracle, run

pytestmark = pytest.mark.gpu


def strong(seed, n, value, weak, block, Hv=16, N=128, dtype=torch.bfloat16):
    """In every chunk of 64 tokens: `n` tokens of g = value at the start of block
    `block` of 16 tokens, one written token behind them."""
    q, k, v, g, b = inputs(seed, 1, 1, Hv, N, 128, 128, dtype, weak)
    b.zero_()
    for c in range(0, N, 64):
        at = c + 16 * block
        g[..., at:at + n] = value
        b[..., at + n] = 1.0
    return q, k, v, g, b


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("block", [0, 3])
@pytest.mark.parametrize("value", [-float("inf"), -80.0, -37.3])
@pytest.mark.parametrize("n", [6, 8, 12])
def test_decays_behind_strong_tokens(n, value, block, dtype):
    cla = lib()
    t = strong(70, n, value, 0.05, block, dtype=dtype)
    got, ref = run(cla, t), oracle(t)
    tol = STATE_BF16 if dtype == torch.bfloat16 else STATE_F32
    worst = max(rel_l2(f64(got[1])[0, h], ref[1][0, h]) for h in range(16))
    assert worst <= tol
    check(cla, got, ref, dtype)


@pytest.mark.parametrize("n", [6, 10])
def test_corrections_behind_strong_tokens(n):
    """Two writes of one key behind the strong tokens: the second one's
    correction holds the decay between them."""
    cla = lib()
    q, k, v, g, b = strong(71, n, -float("inf"), 0.05, 2)
    for c in range(0, 128, 64):
        at = c + 32 + n
        k[:, :, at + 4] = k[:, :, at]
        b[..., at + 4] = 0.5
    t = (q, k, v, g, b)
    got, ref = run(cla, t), oracle(t)
    assert max(rel_l2(f64(got[1])[0, h], ref[1][0, h]) for h in range(16)) <= STATE_BF16
    check(cla, got, ref, torch.bfloat16)


def test_a_strong_token_now_and_then():
    """Decays from a token's whole range, mixed: uniform in [-16, 0], some of
    -inf, writes everywhere."""
    cla = lib()
    q, k, v, g, b = inputs(72, 1, 2, 4, 640, 64, 64, torch.bfloat16)
    gen = torch.Generator().manual_seed(73)
    g.copy_(-16 * torch.rand(g.shape, generator=gen) ** 4)
    g[torch.rand(g.shape, generator=gen) < 0.1] = -float("inf")
    t = (q, k, v, g, b)
    got, ref = run(cla, t), oracle(t)
    assert all(np.isfinite(f64(x)).all() for x in got)
    assert max(rel_l2(f64(got[1])[0, h], ref[1][0, h]) for h in range(4)) <= STATE_BF16
    check(cla, got, ref, torch.bfloat16)
