"""The fixed-state mixers at sizes on both sides of what their launches choose by:
segments of the scan, rows and pieces of a thread, warps and splits of a row."""
import numpy as np
import pytest
import torch

from oracle import mixers_oracle as MO
from tests import test_gpu_mixers as M
from tests.gpu_util import f64, lib

pytestmark = pytest.mark.gpu

TYPES = M.TYPES


@TYPES
@pytest.mark.parametrize("N", [95, 96, 97, 111, 129, 255, 256, 257, 300])
def test_scan_segments(N, dtype):
    """Segments of 16 tokens and up; cut between sequences, inside one, and behind an
    empty one."""
    cla = lib()
    t = M.scan_inputs(60, 1, N, 40, 16, 1, dtype)
    r = M.gen(61)
    M.scan(cla, t, state=r(1, 40, 16))
    starts = [3, 16, 16, 50, N - 17, N - 2]
    M.scan(cla, t, state=r(5, 40, 16), starts=starts)


@TYPES
@pytest.mark.parametrize("N", [250, 256, 290])
def test_scan_two_segments(N, dtype):
    """Channels that leave room for two segments."""
    M.scan(lib(), M.scan_inputs(62, 4, N, 1100, 16, 1, dtype), state=M.gen(63)(4, 1100, 16))


@TYPES
@pytest.mark.parametrize("size", [
    (40, 4096, 16, 1), (41, 4090, 12, 1), (40, 4090, 13, 2), (20, 2048, 64, 1), (5, 200, 50, 1),
    (6, 1024, 128, 2), (3, 100, 99, 1), (4, 1000, 20, 1), (90, 4096, 4, 1), (91, 4096, 3, 1),
    (61, 4096, 8, 2), (60, 4095, 7, 1), (60, 2048, 32, 1)], ids=str)
def test_scan_step_rows(size, dtype):
    M.test_scan_step(size, dtype)


@TYPES
@pytest.mark.parametrize("size", [(128, 4096, 4), (129, 4092, 2), (130, 4096, 8), (131, 4096, 5),
                                  (60, 2052, 3), (200, 2052, 7), (200, 2050, 6), (64, 2051, 4)],
                         ids=str)
def test_conv_step_rows(size, dtype):
    M.test_conv_step(size, dtype)


@TYPES
@pytest.mark.parametrize("size", [(80, 16, 8, 128, 60, 4), (80, 16, 8, 64, 200, 0),
                                  (5, 32, 8, 128, 900, 4), (1, 24, 2, 112, 515, 1)], ids=str)
def test_attention_step_rows(size, dtype):
    M.test_attention_step(size, dtype)


def bad_slots(n, pool):
    """Slots of n rows: one twice in neighbouring rows, one twice far apart, one outside
    the pool, idle ones; and the rows that keep theirs."""
    slots = [(7 * b) % pool for b in range(n)]
    slots[5] = slots[4]
    slots[n - 1] = slots[0]
    slots[9] = pool
    slots[12] = -1
    return slots, [b for b in range(n) if b not in (5, n - 1, 9, 12)]


@TYPES
def test_scan_step_bad_slots(dtype):
    """Rows of one thread among them."""
    cla = lib()
    n, ch, S, pool = 41, 4096, 16, 53
    x, dt, A, Bm, Cm, D, bias, z = M.scan_inputs(64, 1, n, ch, S, 1, dtype)
    state = M.gen(65)(pool, ch, S)
    slots, good = bad_slots(n, pool)
    st = state.to(M.DEV)
    got = cla.selective_scan_step(x[0].to(M.DEV), dt[0].to(M.DEV), A.to(M.DEV), Bm[0].to(M.DEV),
                                  Cm[0].to(M.DEV), st, D=D.to(M.DEV), dt_bias=bias.to(M.DEV),
                                  z=z[0].to(M.DEV), slots=M.ints(slots))
    torch.cuda.synchronize()
    assert cla.device_status() == M.TTT_ERR_ARG
    at = [slots[b] for b in good]
    t = [f64(y[0, good])[:, None] for y in (x, dt)] + [f64(A)] + [f64(y[0, good])[:, None]
                                                                 for y in (Bm, Cm)]
    ro, rh, eo, eh = MO.selective_scan(*t, f64(D), f64(bias), f64(z[0, good])[:, None], True,
                                       f64(state[at]))
    M.within(got[good], ro[:, 0], eo[:, 0], dtype)
    M.within(st[at], rh, eh, M.F32)
    assert (got[[b for b in range(n) if b not in good]] == 0).all()
    rest = [i for i in range(pool) if i not in at]
    assert torch.equal(st[rest].cpu(), state[rest])


@TYPES
def test_conv_step_bad_slots(dtype):
    cla = lib()
    n, D, W, pool = 160, 4096, 4, 171
    r = M.gen(66)
    x, w, state = r(n, D).to(dtype), r(D, W), r(pool, W - 1, D).to(dtype)
    slots, good = bad_slots(n, pool)
    st = state.to(M.DEV)
    got = cla.short_conv_step(x.to(M.DEV), w.to(M.DEV), st, None, False, M.ints(slots))
    torch.cuda.synchronize()
    assert cla.device_status() == M.TTT_ERR_ARG
    at = [slots[b] for b in good]
    ro, rs, eo = MO.short_conv(f64(x[good])[:, None], f64(w), None, False, f64(state[at]))
    M.within(got[good], ro[:, 0], eo[:, 0], dtype)
    assert np.array_equal(f64(st[at]), rs)
    assert (got[[b for b in range(n) if b not in good]] == 0).all()
    rest = [i for i in range(pool) if i not in at]
    assert torch.equal(st[rest].cpu(), state[rest])


@TYPES
@pytest.mark.parametrize("window, sinks", [(300, 5), (64, 0), (129, 70)], ids=str)
def test_attention_ring_tiles(window, sinks, dtype):
    """Sequences longer than the window behind pasts that end anywhere in the ring: which of
    the cache's tiles a query tile leaves out."""
    places = window + sinks
    pasts = [1, max(1, sinks), sinks + 1, places - 1, places, places + 1, places + 70,
             2 * window + sinks, 5 * places + 33, 0]
    lengths = [90, 400, 1, 333, 260, 128, 257, 500, 64, 77]
    starts = [0] + np.cumsum(lengths).tolist()
    t = M.qkv(67, 1, 4, 2, starts[-1], 64, dtype)
    r = M.gen(68)
    caches = [r(len(pasts), 2, places, 64).to(dtype) for _ in range(2)]
    for x in caches:   # what holds nothing yet
        for s, past in enumerate(pasts):
            x[s, :, min(past, places):] = float("nan")
    cla, slots = lib(), list(range(len(pasts)))
    dev, oracle = [x.to(M.DEV) for x in caches], [f64(x) for x in caches]
    got = cla.window_attention_forward(*[x.to(M.DEV) for x in t], window, sinks, cache_k=dev[0],
                                       cache_v=dev[1], slots=M.ints(slots), past=M.ints(pasts),
                                       seq_starts=M.ints(starts))
    torch.cuda.synchronize()
    assert cla.device_status() == 0
    ref, bound = MO.window_attention(*[f64(x) for x in t], window, sinks, None, oracle, slots, pasts,
                                     starts, M.rounding(dtype, 64))
    M.within(got, ref, bound, dtype)
    for x, y in zip(dev, oracle):   # places that still hold nothing are NaN on both sides
        assert np.array_equal(f64(x), y, equal_nan=True)
