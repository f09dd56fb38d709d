"""Packed sequences around bounds that descend: sequences that share no token
with another one, in front of more overlapping ones than the token axis holds,
are computed; whatever does not fit is empty."""
import pytest
import torch

from oracle import delta_oracle as DO
from tests.gpu_util import f64, lib, rel_l2
from tests.test_delta_output_bound import output_bound
from tests.test_gpu_delta_rule import STATE_BF16, STATE_F32, OUT, TTT_ERR_ARG, inputs, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("again", [3, 140])   # with 280 sequences the plan takes turns
def test_a_sequence_in_front_of_overlapping_ones(again, dtype):
    cla = lib()
    N, first = 600, 70
    starts = [0, first] + [N, first] * again + [N]
    n = len(starts) - 1
    t = inputs(97, 1, 1, 2, N, 128, 128, dtype)
    S0 = torch.randn(n, 2, 128, 128, generator=torch.Generator().manual_seed(98)) * 0.3
    o, S = run(cla, t, S0, starts)
    assert cla.device_status() == TTT_ERR_ARG
    ref = DO.delta_rule(*[f64(x)[:, :, :first] for x in t], f64(S0[:1]))
    bf16 = dtype == torch.bfloat16
    assert rel_l2(f64(o)[:, :, :first], ref[0]) <= (output_bound(ref[0]) if bf16 else OUT[dtype])
    assert rel_l2(f64(S[:1]), ref[1]) <= (STATE_BF16 if bf16 else STATE_F32)
    for s in range(2, n, 2):   # the descending ones
        assert torch.equal(S[s].cpu(), S0[s])
    if bf16:
        # of the others, the first that the token axis has room for, and none behind them
        whole = DO.delta_rule(*[f64(x)[:, :, first:] for x in t], f64(S0[1:2]))[1]
        assert rel_l2(f64(S[1:2]), whole) <= STATE_BF16
