"""Delta-rule calls right behind one another, on two streams at once.

Each kernel of a call begins while the one before it still runs, and the calls'
kernels hold tensor memory of different sizes: dense and packed calls, whole and
in segments, joined by rows and by tiles, in alternation and without a
synchronisation between them, give the bits that each gives alone.
"""
import pytest
import torch

from tests.gpu_util import assert_status_ok, lib
from tests.test_gpu_delta_rule import DEV, inputs

pytestmark = pytest.mark.gpu

CALLS = [
    # B, Hk, Hv, N, dk, dv, packed bounds
    (1, 2, 4, 2000, 128, 128, None),              # segments, 16 rows a join
    (1, 4, 32, 1000, 64, 64, None),               # whole
    (1, 20, 20, 3000, 64, 256, None),             # segments, joined by tiles
    (1, 1, 2, 1500, 128, 128, [0, 40, 1300, 1500]),
    (3, 2, 16, 90, 128, 72, None),                # many short ones
    (1, 4, 4, 30, 128, 128, None),                # token by token
]


def test_calls_behind_one_another_on_two_streams():
    cla = lib()
    sets = []
    for i, (*size, starts) in enumerate(CALLS):
        t = [x.to(DEV) for x in inputs(90 + i, *size, torch.bfloat16, 0.05)]
        s = None if starts is None else torch.tensor(starts, dtype=torch.int32, device=DEV)
        torch.cuda.synchronize()
        want = cla.delta_rule_chunked_forward(*t, seq_starts=s)
        torch.cuda.synchronize()
        sets.append((t, s, want))
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for turn in range(12):
        for i in range(len(sets)):
            for j, st in enumerate(streams):
                n = (i * (1 + 4 * j) + turn) % len(sets)   # 1 and 5: each call meets each
                t, s, _ = sets[n]
                got.append((n, cla.delta_rule_chunked_forward(*t, seq_starts=s, stream=st)))
    torch.cuda.synchronize()
    assert_status_ok(cla)
    for n, (o, S) in got:
        assert torch.equal(o, sets[n][2][0]) and torch.equal(S, sets[n][2][1])
