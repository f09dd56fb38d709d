"""What window attention's prompts report about sequences that hold no token."""
import pytest
import torch

from tests import test_gpu_mixers as M
from tests.gpu_util import lib

pytestmark = pytest.mark.gpu

DEV = M.DEV


@M.TYPES
def test_a_negative_past_of_an_empty_sequence(dtype):
    """Is reported as any other; a sequence without a slot has no past to be looked at."""
    cla = lib()
    t = [x.to(DEV) for x in M.qkv(1, 1, 2, 1, 40, 64, dtype)]
    for past, slots, status in (([3, -1, 5], [0, 1, 2], M.TTT_ERR_ARG),
                                ([3, -1, 5], [0, -1, 2], 0), ([3, 1, 5], [0, 1, 2], 0)):
        cache = [x.to(DEV) for x in M.caches(2, 3, 1, 12, 64, dtype)]
        before = [x.clone() for x in cache]
        cla.window_attention_forward(*t, 10, 2, cache_k=cache[0], cache_v=cache[1],
                                     slots=M.ints(slots), past=M.ints(past),
                                     seq_starts=M.ints([0, 25, 25, 40]))
        assert cla.device_status() == status
        for x, y in zip(cache, before):
            assert torch.equal(x[1], y[1]) and not torch.equal(x[0], y[0])
