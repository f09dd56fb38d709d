"""Window attention at the last positions that 31 bits hold."""
import pytest
import torch

from tests import test_gpu_mixers as M
from tests.gpu_util import assert_status_ok, lib

pytestmark = pytest.mark.gpu

DEV, TYPES = M.DEV, M.TYPES


@TYPES
@pytest.mark.parametrize("d", [64, 200])
@pytest.mark.parametrize("window, sinks", [(1000, 4), (70, 0), (40, 90)], ids=str)
def test_far_positions_are_as_near_ones(window, sinks, d, dtype):
    """Prompts that end at position 2^31 - 2, and single tokens there, against texts some laps
    of the ring long whose next token has the same place."""
    cla = lib()
    N, B = 300, 3
    pasts = [2 ** 31 - 1 - N, 2 ** 31 - 1 - N - window // 2, 2 ** 31 - 1 - N - window + 1]
    near = [sinks + 4 * window + (p - sinks) % window for p in pasts]
    t = [x.to(DEV) for x in M.qkv(1, B, 4, 2, N, d, dtype)]
    one = [x[:, :, 7] for x in t]
    cache = [x.to(DEV) for x in M.caches(2, B, 2, window + sinks, d, dtype)]
    res = []
    for past in (pasts, near):
        c = [x.clone() for x in cache]
        o = cla.window_attention_forward(*t, window, sinks, cache_k=c[0], cache_v=c[1],
                                         past=M.ints(past))
        s = cla.window_attention_step(*one, *c, M.ints([p + N - 1 for p in past]), window, sinks)
        res.append((o, s, *c))
    torch.cuda.synchronize()
    assert_status_ok(cla)
    for a, b in zip(*res):
        assert torch.equal(a, b)
