"""Bounded waits of the delta rule's chunk form that run out, without a fault.

The test hook keeps something from the first CTA of one kernel (see
ttt_selftest_withhold_delta): its waits give up after 1 ms, what it has issued is
waited for, and the call ends.  The host reads TTT_ERR_TIMEOUT, the other heads
have their usual bits, and the next call has all of them.
"""
import pytest
import torch

from tests.gpu_util import assert_status_ok, lib
from tests.test_gpu_delta_rule import DEV, inputs

pytestmark = pytest.mark.gpu

TTT_ERR_TIMEOUT = -7

CASES = [
    # kernel held back, (B, Hk, Hv, N, dk, dv), packed bounds
    (1, (1, 2, 4, 500, 128, 128), None),
    (1, (1, 2, 4, 2000, 128, 128), None),
    (4, (1, 3, 3, 600, 128, 128), None),
    (4, (1, 2, 2, 190, 64, 64), None),
    (2, (1, 2, 4, 2000, 128, 128), None),
    (2, (1, 20, 20, 3000, 64, 256), None),
    (3, (1, 2, 4, 2000, 128, 128), None),     # joined by 16 rows
    (3, (1, 20, 20, 3000, 64, 256), None),    # by tiles
    (4, (1, 20, 20, 3000, 64, 256), None),
    (2, (1, 1, 2, 3000, 128, 128), [0, 60, 2990, 3000]),
    (4, (1, 1, 2, 3000, 128, 128), [0, 60, 2990, 3000]),
]


@pytest.mark.parametrize("kernel,size,starts", CASES, ids=str)
def test_a_wait_that_runs_out_ends_the_call(kernel, size, starts):
    cla = lib()
    _, Hk, Hv, N, dk, dv = size
    t = [x.to(DEV) for x in inputs(95, *size, torch.bfloat16, 0.05)]
    s = None if starts is None else torch.tensor(starts, dtype=torch.int32, device=DEV)
    room = torch.full((1, Hv, N + 2, dv), 7.0, dtype=torch.bfloat16, device=DEV)
    out = room[:, :, 1:-1]
    n_seq = 1 if starts is None else len(starts) - 1
    states = torch.full((n_seq + 2, Hv, dv, dk), 7.0, device=DEV)
    cla.profile_start()
    want = cla.delta_rule_chunked_forward(*t, seq_starts=s)
    torch.cuda.synchronize()
    kinds = {e["name"] for e in cla.profile_stop()}
    assert {1: "delta.prep", 2: "delta.carry", 3: "delta.join", 4: "delta.chunk"}[kernel] in kinds
    assert_status_ok(cla)
    cla.set_wait_limit_ns(1_000_000)
    cla.selftest_withhold_delta(kernel)
    try:
        cla.delta_rule_chunked_forward(*t, seq_starts=s, out=out, S_final=states[1:-1])
        status = cla.device_status()
    finally:
        cla.selftest_withhold_delta(0)
        cla.set_wait_limit_ns(200_000_000)
    assert status == TTT_ERR_TIMEOUT
    assert cla.device_status() == 0          # read and cleared
    assert (room[:, :, 0] == 7.0).all() and (room[:, :, -1] == 7.0).all()
    assert (states[0] == 7.0).all() and (states[-1] == 7.0).all()
    if starts is None:
        first = Hv // Hk   # the first key head's
        assert torch.equal(out[:, first:], want[0][:, first:])
        assert torch.equal(states[1, first:], want[1][0, first:])
    got = cla.delta_rule_chunked_forward(*t, seq_starts=s)
    torch.cuda.synchronize()
    assert_status_ok(cla)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
