"""The selective scan over texts that are cut into segments, at the ends of fp32's range:
states that are NaN or infinite, decays that underflow over a segment, and growth that
passes the largest number.

The oracle goes token by token.  Finite numbers are held to its bound; NaN and infinities
have to lie where the oracle has them.
"""
import numpy as np
import pytest
import torch

from oracle import mixers_oracle as MO
from tests import test_gpu_mixers as M
from tests.gpu_util import assert_status_ok, f64, lib

pytestmark = pytest.mark.gpu

TYPES = M.TYPES
NAN, INF = float("nan"), float("inf")


def inputs(seed, N, ch, S, dtype, steps):
    """Steps (the softplus of dt, without a bias) of about `steps`; A of -8 to -1."""
    r = M.gen(seed)
    x, z = r(1, N, ch).to(dtype), r(1, N, ch).to(dtype)
    dt = (np.log(np.expm1(steps)) + 0.1 * r(1, N, ch)).to(dtype)
    A = -(1 + 7 * torch.rand(ch, S, generator=torch.Generator().manual_seed(seed)))
    return [x, dt, A, r(1, N, 1, S).to(dtype), r(1, N, 1, S).to(dtype), r(ch), torch.zeros(ch), z]


def alike(got, ref, bound, dtype):
    got = f64(got)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    inf = np.isinf(ref)
    assert np.array_equal(np.isinf(got), inf) and np.array_equal(got[inf], ref[inf])
    held = np.isfinite(ref)
    got, ref, bound = got[held], ref[held], bound[held]
    off = np.abs(got - ref) - (bound + M.HALF[dtype] * (np.abs(ref) + bound))
    assert off.size == 0 or off.max() <= 1e-38, off.max()


def scan(t, state=None, softplus=True, starts=None):
    """The call against the oracle; (out, states)."""
    cla = lib()
    dev = [y.to(M.DEV) for y in t]
    o, h = cla.selective_scan_forward(*dev, softplus,
                                      state=None if state is None else state.to(M.DEV),
                                      seq_starts=M.ints(starts))
    torch.cuda.synchronize()
    assert_status_ok(cla)
    with np.errstate(all="ignore"):
        ro, rh, eo, eh = MO.selective_scan(*[f64(y) for y in t], softplus,
                                           None if state is None else f64(state), starts)
    alike(o, ro, eo, t[0].dtype)
    alike(h, rh, eh, M.F32)
    return o, h


# both kinds of thread: one channel of a few lanes, and four channels
SHAPES = pytest.mark.parametrize("N, ch, S", [(300, 40, 16), (2600, 1024, 16)], ids=str)


@TYPES
@SHAPES
@pytest.mark.parametrize("what", [NAN, INF])
@pytest.mark.parametrize("where", ["x", "dt", "state"])
def test_what_is_not_finite_stays(where, what, N, ch, S, dtype):
    """A token's decay is e^-16 at the least, a segment's below 2^-126: what is not finite in an
    early token's input or step, or in the state before the text, is still so at its end."""
    t = inputs(80, N, ch, S, dtype, 2.0)
    state = M.gen(81)(1, ch, S)
    some = list(range(0, ch, 7))
    if where == "state":
        state[:, some, 3] = what
    else:
        t[0 if where == "x" else 1][:, 17, some] = what
    o, h = scan(t, state)
    bad = ~np.isfinite(f64(h))[0]
    if where == "state":
        assert bad[some, 3].all() and bad.sum() == len(some)
    else:
        assert bad[some].all() and bad.sum() == len(some) * S
    assert not np.isfinite(f64(o)[0, 20:, some]).any()


@TYPES
def test_segments_do_not_change_what_is_not_finite(dtype):
    """The same text in one call, and in calls that are too short for segments."""
    cla = lib()
    N, ch, S = 720, 64, 16
    t = inputs(82, N, ch, S, dtype, 2.0)
    t[0][:, 30, 5] = NAN
    t[0][:, 100, 9] = INF
    t[3][:, 500, :, 2] = NAN
    o, h = scan(t)
    dev = [y.to(M.DEV) for y in t]
    part, st = [], None
    for a in range(0, N, 90):
        cut = [y[:, a:a + 90] if y.dim() > 2 else y for y in dev]
        y, st = cla.selective_scan_forward(*cut, True, state=st)
        part.append(y)
    y = torch.cat(part, 1)
    torch.cuda.synchronize()
    for a, b in ((o, y), (h, st)):
        a, b = f64(a), f64(b)
        assert np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(np.isinf(a), np.isinf(b))


@TYPES
def test_a_new_sequence_drops_what_is_not_finite(dtype):
    """Sequences that begin inside a segment, at its start, and behind tokens of none."""
    N, ch, S = 300, 40, 16
    starts = [0, 40, 96, 96, 250]
    t = inputs(83, N, ch, S, dtype, 2.0)
    t[0][:, 3, ::3] = NAN
    t[0][:, 100, ::5] = INF
    state = M.gen(84)(4, ch, S)
    state[2, 1, 1] = INF   # an empty sequence's
    cla = lib()
    dev = [y.to(M.DEV) for y in t]
    o, h = cla.selective_scan_forward(*dev, state=state.to(M.DEV), seq_starts=M.ints(starts))
    torch.cuda.synchronize()
    assert_status_ok(cla)
    with np.errstate(all="ignore"):
        ro, rh, eo, eh = MO.selective_scan(*[f64(y) for y in t], True, f64(state), starts)
    alike(o[:, :250], ro[:, :250], eo[:, :250], dtype)
    alike(h, rh, eh, M.F32)


@TYPES
@SHAPES
@pytest.mark.parametrize("negative", [False, True], ids=["A", "steps"])
def test_growth_behind_zero_inputs(negative, N, ch, S, dtype):
    """Growth of e^6 a token, from positive A or from negative steps: states are zero as long as
    the inputs are (segments whose growth no number holds), then grow by e^2 a token."""
    t = inputs(85, N, ch, S, dtype, 2.0)
    t[2] = torch.ones(ch, S) if not negative else -torch.ones(ch, S)
    t[1] = torch.full((1, N, ch), -6.0 if negative else 6.0).to(dtype)
    t[1][:, N - 20:] /= 3.0
    t[0][:, :N - 20] = 0.0
    _, h = scan(t, softplus=False)
    assert h.abs().max() > 1e14


GROWN = pytest.mark.parametrize("at, n", [(32, 16), (37, 16), (16, 32), (80, 16)], ids=str)


@GROWN
@pytest.mark.parametrize("N, ch", [(96, 40), (300, 33)], ids=str)
def test_small_states_that_grow_and_large_ones_that_shrink(N, ch, at, n):
    """e^96 within a segment or two, up from 1e-30 and down from 1e30: neither factor is an
    fp32 number, what it leads to is."""
    S = 16
    t = inputs(86, N, ch, S, M.F32, 2.0)
    t[0][:] = 0.0
    t[1][:] = 0.0
    t[1][:, at:at + n] = 96.0 / n
    t[2] = torch.ones(ch, S)
    t[2][1::2] = -1.0
    state = M.gen(87)(1, ch, S)
    state[:, 0::2] *= 1e-30
    state[:, 1::2] *= 1e30
    _, h = scan(t, state, softplus=False)
    h = h.abs().cpu()
    assert h[:, 0::2].max() > 1e11 and 1e-13 < h[:, 1::2].max() < 1e-10


def test_growth_past_the_largest_number():
    """Is infinite, with its sign, and stays so; zero stays zero beside it."""
    cla = lib()
    N, ch, S = 300, 40, 16
    t = inputs(88, N, ch, S, M.F32, 2.0)
    t[0][:] = 0.0
    t[1][:] = 1.0
    t[2] = torch.ones(ch, S)
    t[2][1] = 40.0         # e^640 in sixteen tokens
    state = M.gen(89)(1, ch, S)
    state[:, 2] = 0.0
    o, h = cla.selective_scan_forward(*[y.to(M.DEV) for y in t[:5]], dt_softplus=False,
                                      state=state.to(M.DEV))
    torch.cuda.synchronize()
    want = torch.where(state == 0, state, torch.sign(state) * INF)
    assert torch.equal(h.cpu(), want)
    assert (o[:, :, 2] == 0).all()
