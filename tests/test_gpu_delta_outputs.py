"""bf16 outputs of the chunk form held to output_bound (see
test_delta_output_bound.py), which a dropped low part of any pair exceeds, and
outputs whose rows cannot be stored 16 bytes at a time."""
import numpy as np
import pytest
import torch

from tests.gpu_util import assert_status_ok, f64, lib, rel_l2
from tests.test_delta_output_bound import output_bound
from tests.test_gpu_delta_rule import DEV, STATE_BF16, inputs, oracle, run

pytestmark = pytest.mark.gpu

BF = torch.bfloat16

CASES = [
    # B, Hk, Hv, N, dk, dv, decay
    (2, 2, 4, 300, 128, 128, 0.1),     # whole sequences
    (1, 1, 2, 200, 64, 64, 0.02),      # kernels of half the columns
    (1, 2, 2, 333, 96, 72, 0.1),       # columns and rows behind d_k and d_v
    (1, 1, 2, 260, 128, 256, 0.02),    # two tiles
    (1, 2, 4, 2000, 128, 128, 0.01),   # segments, joined by 16 rows
    (1, 4, 16, 1400, 64, 128, 0.01),   # segments, joined by tiles or 32 rows
]


def check(cla, got, ref):
    assert_status_ok(cla)
    o, ro = f64(got[0]), ref[0]
    held = ~np.isnan(ro)
    assert rel_l2(o[held], ro[held]) <= output_bound(ro[held])
    assert rel_l2(f64(got[1]), ref[1]) <= STATE_BF16


@pytest.mark.parametrize("case", CASES, ids=str)
def test_outputs_are_rounded_once(case):
    cla = lib()
    *size, decay = case
    B, Hk, Hv, N, dk, dv = size
    t = inputs(80, *size, BF, decay)
    S0 = torch.randn(B, Hv, dv, dk, generator=torch.Generator().manual_seed(81)) * 0.3
    check(cla, run(cla, t, S0), oracle(t, S0))


def test_outputs_of_packed_sequences_are_rounded_once():
    cla = lib()
    starts = [2, 700, 700, 701, 1130, 3000]
    t = inputs(82, 1, 1, 2, 3003, 128, 128, BF, 0.02)
    S0 = torch.randn(5, 2, 128, 128, generator=torch.Generator().manual_seed(83)) * 0.3
    check(cla, run(cla, t, S0, starts), oracle(t, S0, starts))


@pytest.mark.parametrize("lead,tail", [(1, 0), (8, 3), (0, 4)])
@pytest.mark.parametrize("dv", [128, 72])
def test_outputs_in_rows_of_odd_strides(dv, lead, tail):
    """q, k and v as the tensor cores take them, rows of out at odd offsets or
    distances: the same numbers, and nothing around them is touched."""
    cla = lib()
    N = 150
    t = inputs(84, 1, 1, 2, N, 128, dv, BF, 0.1)
    cla.profile_start()
    want = run(cla, t)
    kinds = {e["name"] for e in cla.profile_stop()}
    room = torch.full((1, 2, N + 1, lead + dv + tail), 7.0, dtype=BF, device=DEV)
    cla.profile_start()
    got = run(cla, t, out=room[:, :, :N, lead:lead + dv])
    assert {e["name"] for e in cla.profile_stop()} == kinds and "delta.chunk" in kinds
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert (room[:, :, N:] == 7.0).all() and (room[..., :lead] == 7.0).all()
    assert (room[..., lead + dv:] == 7.0).all()
    check(cla, got, oracle(t))
