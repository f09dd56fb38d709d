"""Window attention, the selective scan and the short convolution on the GPU
against the fp64 oracle.

Every element is held to the oracle's own bound for a computation in fp32 plus
the rounding of the output: half a step, 2^-8 of the value for bf16 and 2^-24
for fp32.  Where the attention's weights are rounded to bf16 for the product
with v, they add 2^-8 of the weighted absolute values.
"""
import numpy as np
import pytest
import torch

from oracle import mixers_oracle as MO
from tests.gpu_util import assert_status_ok, f64, lib

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TTT_ERR_ARG = -8
BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
TYPES = pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])


def within(got, ref, bound, dtype):
    """Rows that are NaN in the oracle belong to no sequence."""
    got = f64(got)
    held = ~np.isnan(ref)
    assert np.isfinite(got[held]).all()
    off = np.abs(got - ref)[held] - (bound + HALF[dtype] * (np.abs(ref) + bound))[held]
    assert off.size == 0 or off.max() <= 1e-38, off.max()


def gen(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s: torch.randn(s, generator=g)


def ints(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------- attention


def qkv(seed, B, Hq, Hk, N, d, dtype):
    r = gen(seed)
    return r(B, Hq, N, d).to(dtype), r(B, Hk, N, d).to(dtype), r(B, Hk, N, d).to(dtype)


def rounding(dtype, d):
    """Of the weights, where the tensor cores may take the call."""
    return 2.0 ** -8 if dtype == BF16 and d <= 128 and d % 8 == 0 else 0.0


def attn(cla, t, window, sinks, dtype, caches=None, slots=None, past=None, starts=None, out=None,
         **kw):
    """The call on the GPU against the oracle, caches among the results."""
    dev = [x.to(DEV) if x.device.type == "cpu" else x for x in t]
    cd = [None, None] if caches is None else [c.to(DEV) for c in caches]
    co = None if caches is None else [f64(c) for c in caches]
    got = cla.window_attention_forward(*dev, window, sinks, cache_k=cd[0], cache_v=cd[1],
                                       slots=ints(slots), past=ints(past), seq_starts=ints(starts),
                                       out=out, **kw)
    torch.cuda.synchronize()
    assert_status_ok(cla)
    ref, bound = MO.window_attention(*[f64(x) for x in t], window, sinks, kw.get("scale"), co, slots,
                                     past, starts, rounding(dtype, t[0].shape[-1]))
    within(got, ref, bound, dtype)
    if caches is not None:
        assert np.array_equal(f64(cd[0]), co[0]) and np.array_equal(f64(cd[1]), co[1])
    return got, cd


def caches(seed, n, Hk, places, d, dtype):
    r = gen(seed)
    return [r(n, Hk, places, d).to(dtype), r(n, Hk, places, d).to(dtype)]


SIZES = [
    # B, Hq, Hk, N, d, window, sinks
    (1, 1, 1, 1, 64, 1, 0),
    (1, 2, 1, 5, 64, 3, 1),
    (2, 2, 2, 64, 64, 16, 0),
    (1, 4, 2, 129, 128, 40, 4),
    (1, 3, 1, 300, 128, 128, 4),
    (1, 2, 2, 257, 128, 1000, 0),
    (1, 1, 1, 260, 64, 100, 140),
    (1, 1, 1, 400, 128, 1, 2),
    (1, 2, 1, 131, 96, 50, 3),
    (1, 2, 1, 70, 80, 300, 300),
    (1, 1, 1, 67, 40, 20, 0),
    (1, 1, 1, 90, 33, 20, 5),
    (1, 1, 1, 70, 192, 20, 5),
    (1, 1, 1, 70, 256, 30, 0),
    (1, 1, 1, 600, 32, 256, 0),
]


@TYPES
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_attention_sizes(size, dtype):
    cla = lib()
    B, Hq, Hk, N, d, window, sinks = size
    t = qkv(1, B, Hq, Hk, N, d, dtype)
    attn(cla, t, window, sinks, dtype)
    attn(cla, t, window, sinks, dtype, caches(2, B + 2, Hk, window + sinks, d, dtype),
         slots=[B + 1 - b for b in range(B)])


@TYPES
@pytest.mark.parametrize("d", [128, 72])
def test_attention_of_many_blocks(d, dtype):
    """More blocks than the card takes at once, the last of them short."""
    cla = lib()
    attn(cla, qkv(14, 2, 16, 1, 1300, d, dtype), 70, 5, dtype)


@TYPES
@pytest.mark.parametrize("window,sinks", [(40, 4), (130, 0), (1, 1), (16, 200)])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_goes_on_from_a_cache(window, sinks, d, dtype):
    """Pasts in front of, inside and behind the sinks and the first window; an
    empty past; a sequence without a slot."""
    cla = lib()
    places = window + sinks
    past = [0, 1, max(1, sinks), places - 1, places, places + 7, 5 * places + 3, 9]
    n = len(past)
    slots = [7, 3, 4, 0, 8, 1, 2, -1]
    t = qkv(3, n, 2, 1, 70, d, dtype)
    attn(cla, t, window, sinks, dtype, caches(4, n + 1, 1, places, d, dtype), slots, past)


PACKS = [[0, 1, 1, 65, 129, 129, 200], [0, 0, 0, 64], [3, 70, 71, 150], [0, 200],
         list(range(0, 208, 4))]


@TYPES
@pytest.mark.parametrize("starts", PACKS, ids=lambda x: str(x)[:24])
@pytest.mark.parametrize("with_past", [False, True])
def test_attention_packed(starts, with_past, dtype):
    """Lengths of zero and one, rows before and behind the sequences left as they
    were; token-major tensors."""
    cla = lib()
    N, d, window, sinks = 208, 64, 24, 3
    n = len(starts) - 1
    t = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in qkv(5, 1, 2, 1, N, d, dtype)]
    past = [(7 * s * s) % 83 for s in range(n)] if with_past else None
    out = torch.full((1, N, 2, d), 7.0, dtype=dtype, device=DEV).transpose(1, 2)
    got, _ = attn(cla, t, window, sinks, dtype, caches(6, n + 1, 1, window + sinks, d, dtype),
                  [n - s for s in range(n)], past, starts, out=out)
    rows = np.ones(N, dtype=bool)
    rows[starts[0]:starts[-1]] = False
    assert (f64(got)[:, :, rows] == 7.0).all()


@TYPES
def test_attention_values_out_of_sight_do_not_leak(dtype):
    """NaN and infinity in the keys and values that a query does not see: other
    sequences', later tokens', ones behind the window, places that hold nothing,
    and tokens of no sequence."""
    cla = lib()
    starts, window, sinks, d = [5, 75, 139], 20, 2, 64
    t = qkv(7, 1, 2, 1, 150, d, dtype)
    ref, bound = MO.window_attention(*[f64(x) for x in t], window, sinks, starts=starts,
                                     weight_rounding=rounding(dtype, d))
    bad = [x.clone() for x in t]
    for x in bad:
        x[:, :, :5] = float("nan")
        x[:, :, 139:] = float("inf")
    bad[1][:, :, 40] = float("nan")    # seen by 40 .. 59
    bad[2][:, :, 100] = float("inf")   # seen by 100 .. 119
    got = cla.window_attention_forward(*[x.to(DEV) for x in bad], window, sinks,
                                       seq_starts=ints(starts))
    torch.cuda.synchronize()
    for lo, hi in ((5, 40), (60, 100), (120, 139)):
        within(got[:, :, lo:hi], ref[:, :, lo:hi], bound[:, :, lo:hi], dtype)
    assert torch.isnan(got[:, :, 40:60]).all()
    assert torch.isinf(got[:, :, 100:120]).all()
    # a cache whose unused places hold NaN
    c = caches(8, 1, 1, window + sinks, d, dtype)
    for x in c:
        x[:, :, 9:] = float("nan")
    attn(cla, [x[:, :, :90] for x in t], window, sinks, dtype, c, past=[9])


@TYPES
def test_attention_extreme_scores(dtype):
    """Scores far apart, keys of length zero, and a scale of zero and below."""
    cla = lib()
    q, k, v = qkv(9, 1, 2, 1, 150, 64, dtype)
    k[:, :, 10] *= 30
    k[:, :, 20:30] = 0
    q[:, :, 50] *= 20
    for scale in (None, 0.0, -0.1, 1.0):
        attn(cla, (q, k, v), 33, 2, dtype, scale=scale)


@TYPES
def test_attention_strides(dtype):
    """q, k and v as parts of one projection, repeated heads, an output with room
    between its rows, and addresses that are no multiple of 16 bytes."""
    cla = lib()
    N, d = 140, 64
    r = gen(10)
    qkv_ = r(2, N, (4 + 2 + 2) * d).to(dtype).to(DEV)
    q = qkv_[..., :4 * d].view(2, N, 4, d).transpose(1, 2)
    k = qkv_[..., 4 * d:6 * d].view(2, N, 2, d).transpose(1, 2)
    v = qkv_[..., 6 * d:].view(2, N, 2, d).transpose(1, 2)
    out = torch.zeros(2, 4, N, d + 8, device=DEV, dtype=dtype)[..., :d]
    attn(cla, (q, k, v), 30, 3, dtype, out=out)
    one = v[:, :1].expand(2, 2, N, d)
    attn(cla, (q, k, one), 30, 3, dtype)
    room = r(2, 4, N, d + 1).to(dtype).to(DEV)
    attn(cla, (room[..., 1:], k, v), 30, 3, dtype)


STEP_SIZES = [
    # B, Hq, Hk, d, window, sinks
    (1, 1, 1, 64, 1, 0),
    (3, 4, 2, 64, 16, 2),
    (2, 12, 4, 128, 700, 4),
    (2, 8, 1, 128, 1100, 0),
    (1, 6, 2, 96, 50, 0),
    (2, 2, 2, 40, 33, 1),
    (1, 3, 1, 33, 20, 5),
    (1, 2, 1, 200, 300, 0),
    (1, 5, 1, 256, 100, 4),
]


@TYPES
@pytest.mark.parametrize("size", STEP_SIZES, ids=str)
def test_attention_step(size, dtype):
    """Positions from the first on to far ones, rows on other slots than their
    own, an idle row; the caches afterwards."""
    cla = lib()
    B, Hq, Hk, d, window, sinks = size
    places = window + sinks
    r = gen(11)
    for first in (0, sinks, places - 1, places, 100 * places + 7):
        n = B + 1
        q, k, v = r(n, Hq, d).to(dtype), r(n, Hk, d).to(dtype), r(n, Hk, d).to(dtype)
        c = [r(n + 1, Hk, places, d).to(dtype) for _ in range(2)]
        for x in c:   # places that hold nothing yet
            x[:, :, min(places, first + n):] = float("nan")
        slots = [n - b for b in range(n)]
        slots[n // 2] = -1
        pos = [first + b for b in range(n)]
        for b in range(n):   # what this row's slot holds ends at its position
            if slots[b] >= 0:
                for x in c:
                    x[slots[b], :, min(places, pos[b] + 1):] = float("nan")
        cd = [x.to(DEV) for x in c]
        co = [f64(x) for x in c]
        got = cla.window_attention_step(q.to(DEV), k.to(DEV), v.to(DEV), *cd, ints(pos), window, sinks,
                                        slots=ints(slots))
        torch.cuda.synchronize()
        assert_status_ok(cla)
        ref, bound = MO.window_attention_step(f64(q), f64(k), f64(v), co, pos, window, sinks,
                                              slots=slots)
        within(got, ref, bound, dtype)
        for a, b in zip(cd, co):
            assert np.array_equal(f64(a), b, equal_nan=True)


def test_attention_step_bad_rows():
    """Slots outside the pool, used twice and negative positions: idle rows, and
    the status says so; the others are computed."""
    cla = lib()
    r = gen(12)
    q, k, v = (r(4, 2, 64).to(DEV) for _ in range(3))
    for slots, pos, good in (([0, 5, 2, 1], [3, 3, 3, 3], (0, 2, 3)),
                             ([2, 1, 2, 0], [3, 3, 3, 3], (0, 1, 3)),
                             ([0, 1, 2, 3], [3, -1, 3, 3], (0, 2, 3))):
        c = [torch.randn(4, 2, 10, 64, device=DEV) for _ in range(2)]
        co = [f64(x) for x in c]
        got = cla.window_attention_step(q, k, v, *c, ints(pos), 8, 2, slots=ints(slots))
        torch.cuda.synchronize()
        assert cla.device_status() == TTT_ERR_ARG
        keep = [slots[b] if b in good else -1 for b in range(4)]
        ref, bound = MO.window_attention_step(f64(q), f64(k), f64(v), co, pos, 8, 2, slots=keep)
        within(got, ref, bound, F32)
        for a, b in zip(c, co):
            assert np.array_equal(f64(a), b)


def test_attention_bad_slots_and_pasts():
    """A slot outside the pool has no cache, a shared one is written for its first
    sequence, a negative past is none; each is reported."""
    cla = lib()
    t = [x.to(DEV) for x in qkv(13, 3, 1, 1, 20, 64, F32)]
    for slots, past, want_slots, want_past in (
            ([0, 9, 1], [5, 5, 5], [0, -1, 1], [5, 0, 5]),
            ([0, 1, 2], [5, -3, 5], [0, 1, 2], [5, 0, 5])):
        c = [torch.randn(4, 1, 12, 64, device=DEV) for _ in range(2)]
        co = [f64(x) for x in c]
        got = cla.window_attention_forward(*t, 10, 2, cache_k=c[0], cache_v=c[1], slots=ints(slots),
                                           past=ints(past))
        torch.cuda.synchronize()
        assert cla.device_status() == TTT_ERR_ARG
        ref, bound = MO.window_attention(*[f64(x) for x in t], 10, 2, None, co, want_slots, want_past)
        within(got, ref, bound, F32)
        for a, b in zip(c, co):
            assert np.array_equal(f64(a), b)
    c = [torch.zeros(2, 1, 12, 64, device=DEV) for _ in range(2)]
    cla.window_attention_forward(*t, 10, 2, cache_k=c[0], cache_v=c[1], slots=ints([1, 0, 1]))
    torch.cuda.synchronize()
    assert cla.device_status() == TTT_ERR_ARG
    assert torch.equal(c[0][1, 0, 2 + (19 - 2) % 10], t[1][0, 0, 19])


# ---------------------------------------------------------------- scan


def scan_inputs(seed, nb, N, ch, S, G, dtype):
    r = gen(seed)
    x, dt, z = (r(nb, N, ch).to(dtype) for _ in range(3))
    B, C = r(nb, N, G, S).to(dtype), r(nb, N, G, S).to(dtype)
    A = -torch.exp(r(ch, S) * 0.5) * (1 + torch.arange(S) % 5)
    return x, dt, A, B, C, r(ch), r(ch) - 2, z


def scan(cla, t, state=None, starts=None, out=None, gate=True, softplus=True, **kw):
    x, dt, A, B, C, D, bias, z = t
    dev = [y.to(DEV) for y in t]
    o, h = cla.selective_scan_forward(
        *dev[:5], D=dev[5], dt_bias=dev[6], z=dev[7] if gate else None, dt_softplus=softplus,
        state=None if state is None else state.to(DEV), seq_starts=ints(starts), out=out, **kw)
    torch.cuda.synchronize()
    assert_status_ok(cla)
    ro, rh, eo, eh = MO.selective_scan(f64(x), f64(dt), f64(A), f64(B), f64(C), f64(D), f64(bias),
                                       f64(z) if gate else None, softplus,
                                       None if state is None else f64(state), starts)
    within(o, ro, eo, x.dtype)
    within(h, rh, eh, F32)
    return o, h


SCAN_SIZES = [
    # nb, N, channels, S, G
    (1, 1, 1, 1, 1),
    (1, 37, 64, 16, 1),
    (2, 65, 100, 16, 1),
    (1, 130, 72, 8, 2),
    (1, 20, 33, 5, 3),
    (1, 40, 16, 32, 1),
    (1, 50, 24, 64, 2),
    (1, 17, 8, 100, 1),
    (1, 17, 8, 128, 1),
    (2, 700, 1536, 16, 1),
    (1, 1500, 1502, 12, 1),
    (1, 1300, 1720, 8, 4),
    (1, 700, 3200, 20, 2),
]


@TYPES
@pytest.mark.parametrize("size", SCAN_SIZES, ids=str)
def test_scan_sizes(size, dtype):
    cla = lib()
    nb, N, ch, S, G = size
    t = scan_inputs(20, nb, N, ch, S, G, dtype)
    scan(cla, t, torch.randn(nb, ch, S, generator=torch.Generator().manual_seed(21)))
    if N * ch < 100000:
        scan(cla, t, gate=False)
        # steps as they come are not negative: else the states grow without bound
        scan(cla, [y.abs() if i in (1, 6) else y for i, y in enumerate(t)], softplus=False)


SCAN_PACKS = [[0, 1, 1, 65, 129, 129, 200], [0, 0, 0, 64], [3, 70, 71, 150], [0, 200]]


@TYPES
@pytest.mark.parametrize("starts", SCAN_PACKS, ids=str)
def test_scan_packed(starts, dtype):
    cla = lib()
    N, ch, S, n = 208, 96, 16, len(starts) - 1
    t = scan_inputs(22, 1, N, ch, S, 1, dtype)
    state = torch.randn(n, ch, S, generator=torch.Generator().manual_seed(23))
    out = torch.full((1, N, ch), 7.0, dtype=dtype, device=DEV)
    o, h = scan(cla, t, state, starts, out=out)
    rows = np.ones(N, dtype=bool)
    rows[starts[0]:starts[-1]] = False
    assert (f64(o)[:, rows] == 7.0).all()
    for s in range(n):
        if starts[s] == starts[s + 1]:
            assert torch.equal(h[s].cpu(), state[s])


@TYPES
def test_scan_packed_over_segments(dtype):
    """Sequences that begin and end inside, at and between the segments that a long
    call is cut into."""
    cla = lib()
    N, ch, S = 2600, 1024, 16
    starts = [7, 7, 64, 128, 129, 129, 700, 1344, 2400, 2401, 2590]
    n = len(starts) - 1
    t = scan_inputs(24, 1, N, ch, S, 1, dtype)
    state = torch.randn(n, ch, S, generator=torch.Generator().manual_seed(25))
    scan(cla, t, state, starts)
    scan(cla, t, None, starts)


@TYPES
def test_scan_values_of_other_sequences_do_not_leak(dtype):
    cla = lib()
    N, ch, S = 2600, 1024, 16
    starts = [5, 1000, 1700, 2400]
    t = scan_inputs(26, 1, N, ch, S, 1, dtype)
    ro, rh, eo, eh = MO.selective_scan(*[f64(y) for y in t], True, None, starts)
    for i in (0, 1, 3, 4, 7):
        t[i][:, :5] = float("nan")
        t[i][:, 1000:1700] = float("inf")
        t[i][:, 2400:] = float("nan")
    x, dt, A, B, C, D, bias, z = [y.to(DEV) for y in t]
    o, h = cla.selective_scan_forward(x, dt, A, B, C, D, bias, z, seq_starts=ints(starts))
    torch.cuda.synchronize()
    for s in (0, 2):
        a, e = starts[s], starts[s + 1]
        within(o[:, a:e], ro[:, a:e], eo[:, a:e], dtype)
        within(h[s], rh[s], eh[s], F32)


def test_scan_strides():
    """x and z as halves of one projection, B and C behind dt in another, rows of
    the output with room between them, addresses at odd elements."""
    cla = lib()
    for N, ch in ((45, 64), (1100, 2048)):
        r = gen(27)
        xz = r(2, N, 2 * ch).bfloat16()
        low = r(2, N, 7 + 2 * 16).bfloat16()
        dt = r(2, N, ch + 1).bfloat16()
        _, _, A, _, _, D, bias, _ = scan_inputs(28, 2, N, ch, 16, 1, BF16)
        t = [xz[..., :ch], dt[..., 1:], A, low[..., 7:23].unflatten(2, (1, 16)),
             low[..., 23:].unflatten(2, (1, 16)), D, bias, xz[..., ch:]]
        ro, rh, eo, eh = MO.selective_scan(*[f64(y) for y in t], True)
        dxz, dlow, ddt = xz.to(DEV), low.to(DEV), dt.to(DEV)
        out = torch.zeros(2, N, ch + 5, device=DEV, dtype=BF16)[..., :ch]
        o, h = cla.selective_scan_forward(
            dxz[..., :ch], ddt[..., 1:], A.to(DEV), dlow[..., 7:23].unflatten(2, (1, 16)),
            dlow[..., 23:].unflatten(2, (1, 16)), D.to(DEV), bias.to(DEV), dxz[..., ch:], out=out)
        torch.cuda.synchronize()
        within(o, ro, eo, BF16)
        within(h, rh, eh, F32)


def test_scan_extreme_steps():
    """Steps of zero, tiny and huge ones, decays that underflow, positive A."""
    cla = lib()
    t = list(scan_inputs(29, 1, 90, 32, 16, 1, F32))
    t[1][:, 10:20] = -60.0
    t[1][:, 20:25] = -200.0
    t[1][:, 30] = 80.0
    t[2][:4] = 0.0
    t[2][4:6] = 0.01
    scan(cla, t)


@TYPES
@pytest.mark.parametrize("size", [(1, 1, 1, 1), (3, 64, 16, 1), (5, 100, 16, 2), (2, 33, 5, 3),
                                  (2, 40, 32, 1), (2, 24, 64, 1), (2, 9, 128, 1), (130, 128, 16, 1)],
                         ids=str)
def test_scan_step(size, dtype):
    cla = lib()
    B, ch, S, G = size
    n = B + 1
    x, dt, A, Bm, Cm, D, bias, z = scan_inputs(30, 1, n, ch, S, G, dtype)
    pool = torch.randn(n + 2, ch, S, generator=torch.Generator().manual_seed(31))
    slots = [n - b for b in range(n)]
    slots[n // 2] = -1
    st = pool.to(DEV)
    got = cla.selective_scan_step(x[0].to(DEV), dt[0].to(DEV), A.to(DEV), Bm[0].to(DEV), Cm[0].to(DEV),
                                  st, D=D.to(DEV), dt_bias=bias.to(DEV), z=z[0].to(DEV),
                                  slots=ints(slots))
    torch.cuda.synchronize()
    assert_status_ok(cla)
    live = [b for b in range(n) if slots[b] >= 0]
    at = [slots[b] for b in live]
    t = [f64(y[0, live])[:, None] for y in (x, dt)] + [f64(A)] + [f64(y[0, live])[:, None]
                                                                 for y in (Bm, Cm)]
    ro, rh, eo, eh = MO.selective_scan(*t, f64(D), f64(bias), f64(z[0, live])[:, None], True,
                                       f64(pool[at]))
    within(got[live], ro[:, 0], eo[:, 0], dtype)
    within(st[at], rh, eh, F32)
    idle = [b for b in range(n) if slots[b] < 0]
    assert (got[idle] == 0).all()
    rest = [i for i in range(n + 2) if i not in at]
    assert torch.equal(st[rest].cpu(), pool[rest])


# ---------------------------------------------------------------- convolution


def conv(cla, x, w, bias, silu, state=None, starts=None, out=None):
    o, st = cla.short_conv_forward(x.to(DEV), w.to(DEV), None if bias is None else bias.to(DEV), silu,
                                   None if state is None else state.to(DEV), ints(starts), out=out)
    torch.cuda.synchronize()
    assert_status_ok(cla)
    ro, rs, eo = MO.short_conv(f64(x), f64(w), None if bias is None else f64(bias), silu,
                               None if state is None else f64(state), starts)
    within(o, ro, eo, x.dtype)
    assert np.array_equal(f64(st), rs)
    return o, st


@TYPES
@pytest.mark.parametrize("size", [(1, 1, 1, 4), (1, 1, 8, 4), (2, 3, 64, 4), (1, 16, 100, 4),
                                  (2, 33, 72, 2), (1, 50, 40, 3), (1, 37, 24, 5), (1, 40, 17, 6),
                                  (1, 20, 16, 7), (1, 90, 48, 8)], ids=str)
@pytest.mark.parametrize("silu", [False, True])
def test_conv_sizes(size, silu, dtype):
    cla = lib()
    B, N, D, W = size
    r = gen(40)
    x, w, bias, st = r(B, N, D).to(dtype), r(D, W), r(D), r(B, W - 1, D).to(dtype)
    conv(cla, x, w, bias, silu, st)
    conv(cla, x, w, None, silu)


@TYPES
@pytest.mark.parametrize("starts", SCAN_PACKS + [list(range(0, 208, 2))], ids=lambda x: str(x)[:24])
def test_conv_packed(starts, dtype):
    cla = lib()
    r = gen(41)
    N, D, W, n = 208, 40, 4, len(starts) - 1
    x, w, bias, st = r(1, N, D).to(dtype), r(D, W), r(D), r(n, W - 1, D).to(dtype)
    out = torch.full((1, N, D), 7.0, dtype=dtype, device=DEV)
    o, _ = conv(cla, x, w, bias, True, st, starts, out=out)
    rows = np.ones(N, dtype=bool)
    rows[starts[0]:starts[-1]] = False
    assert (f64(o)[:, rows] == 7.0).all()
    conv(cla, x, w, bias, True, None, starts)
    if n == 1:
        return
    # other sequences' values, and those of none
    y = x.clone()
    y[:, :starts[0]] = float("nan")
    y[:, starts[-1]:] = float("inf")
    y[:, starts[1]:starts[2]] = float("nan")
    ro, _, eo = MO.short_conv(f64(x), f64(w), f64(bias), True, f64(st), starts)
    o, _ = cla.short_conv_forward(y.to(DEV), w.to(DEV), bias.to(DEV), True, st.to(DEV), ints(starts))
    torch.cuda.synchronize()
    for a, e in zip(starts[2:-1], starts[3:]):
        within(o[:, a:e], ro[:, a:e], eo[:, a:e], dtype)


@TYPES
def test_conv_strides(dtype):
    cla = lib()
    r = gen(42)
    w, bias = r(48, 4), r(48)
    for at, room in ((0, 96), (48, 96), (1, 50)):
        x = r(2, 70, room).to(dtype)[..., at:at + 48]
        out = torch.zeros(2, 70, 55, device=DEV, dtype=dtype)[..., 3:51]
        conv(cla, x, w, bias, True, None, out=out)


@TYPES
@pytest.mark.parametrize("size", [(1, 1, 2), (3, 64, 4), (2, 1001, 4), (2, 520, 3), (4, 40, 8)],
                         ids=str)
def test_conv_step(size, dtype):
    cla = lib()
    B, D, W = size
    n = B + 1
    r = gen(43)
    x, w, bias, pool = r(n, D).to(dtype), r(D, W), r(D), r(n + 2, W - 1, D).to(dtype)
    slots = [n - b for b in range(n)]
    slots[n // 2] = -1
    st = pool.to(DEV)
    got = cla.short_conv_step(x.to(DEV), w.to(DEV), st, bias.to(DEV), True, ints(slots))
    torch.cuda.synchronize()
    assert_status_ok(cla)
    live = [b for b in range(n) if slots[b] >= 0]
    at = [slots[b] for b in live]
    ro, rs, eo = MO.short_conv(f64(x[live])[:, None], f64(w), f64(bias), True, f64(pool[at]))
    within(got[live], ro[:, 0], eo[:, 0], dtype)
    assert np.array_equal(f64(st[at]), rs)
    assert (got[[b for b in range(n) if slots[b] < 0]] == 0).all()
    rest = [i for i in range(n + 2) if i not in at]
    assert torch.equal(st[rest].cpu(), pool[rest])


# ---------------------------------------------------------------- all of them


def test_bad_bounds_are_reported():
    cla = lib()
    r = gen(50)
    x, w = r(1, 100, 64).to(DEV), r(64, 4).to(DEV)
    t = [y.to(DEV) for y in scan_inputs(51, 1, 100, 64, 16, 1, F32)]
    q = r(1, 2, 100, 64).to(DEV)
    for starts in ([0, 40, 30, 100, 130], [-1, 10, 100, 2 ** 31 - 1, -2 ** 31],
                   [2 ** 31 - 1] * 5, [-5, -4, -3, -2, -1], [0, 100] * 2 + [0]):
        st = ints(starts)
        for call in (lambda: cla.short_conv_forward(x, w, seq_starts=st),
                     lambda: cla.selective_scan_forward(*t[:5], seq_starts=st),
                     lambda: cla.window_attention_forward(q, q, q, 8, 2, seq_starts=st),
                     lambda: cla.window_attention_forward(
                         q, q, q, 8, 2, cache_k=torch.zeros(4, 2, 10, 64, device=DEV),
                         cache_v=torch.zeros(4, 2, 10, 64, device=DEV), past=ints([3, 30, 3, 0]),
                         seq_starts=st)):
            call()
            assert cla.device_status() == TTT_ERR_ARG
            assert cla.device_status() == 0


def layer(seed, d_model, S):
    """Weights of a small hybrid layer: a convolution and a scan next to window
    attention, normed and joined."""
    r = gen(seed)
    return dict(w=r(d_model, 4) / 2, bias=0.1 * r(d_model), A=-torch.exp(0.3 * r(d_model, S)),
                D=r(d_model), dt_bias=r(d_model) - 2, norm=1 + 0.1 * r(d_model))


@TYPES
def test_a_layer_over_prompts_and_tokens(dtype):
    """Two packed prompts in two turns, then single tokens, through convolution, scan,
    window attention and the block's norm, against the oracle over the whole texts."""
    cla = lib()
    H, d, S, window, sinks = 2, 64, 16, 24, 2
    D = H * d
    turns = [[61, 30], [19, 44]]
    steps = 5
    total = [sum(t[s] for t in turns) + steps for s in range(2)]
    L = layer(60, D, S)
    dev = {k: v.to(DEV) for k, v in L.items()}
    r = gen(61)
    text = [dict(x=r(n, D).to(dtype), q=r(n, H, d).to(dtype), k=r(n, H, d).to(dtype),
                 v=r(n, H, d).to(dtype), dt=r(n, D).to(dtype), B=r(n, 1, S).to(dtype),
                 C=r(n, 1, S).to(dtype)) for n in total]
    refs = []
    for t in text:
        u, _, eu = MO.short_conv(f64(t["x"])[None], f64(L["w"]), f64(L["bias"]), True)
        o, e = MO.window_attention(*[f64(t[n]).transpose(1, 0, 2)[None] for n in ("q", "k", "v")],
                                   window, sinks, weight_rounding=rounding(dtype, d))
        refs.append((u, eu, o, e))
    conv_st = torch.zeros(2, 3, D, device=DEV, dtype=dtype)
    scan_st = torch.zeros(2, D, S, device=DEV)
    ck, cv = (torch.full((2, H, window + sinks, d), float("nan"), device=DEV, dtype=dtype)
              for _ in range(2))
    slots = ints([1, 0])
    done = [0, 0]
    scanned = [[], []]
    for t in turns:
        cut = {n: torch.cat([text[s][n][done[s]:done[s] + t[s]] for s in range(2)]).to(DEV)[None]
               for n in text[0]}
        st = ints([0, t[0], t[0] + t[1]])
        u, conv_st = cla.short_conv_forward(cut["x"], dev["w"], dev["bias"], True, conv_st, st)
        y, scan_st = cla.selective_scan_forward(u, cut["dt"], dev["A"], cut["B"], cut["C"], dev["D"],
                                                dev["dt_bias"], state=scan_st, seq_starts=st)
        o = cla.window_attention_forward(*[cut[n].transpose(1, 2) for n in ("q", "k", "v")], window,
                                         sinks, cache_k=ck, cache_v=cv, slots=slots,
                                         past=ints(done), seq_starts=st)
        n, _ = cla.block_norm_forward(y, w=dev["norm"], gate=o.transpose(1, 2).reshape(1, -1, D),
                                      gate_act=cla.GATE_SIGMOID)
        at = 0
        for s in range(2):
            here = slice(at, at + t[s])
            whole = slice(done[s], done[s] + t[s])
            within(u[0, here], refs[s][0][0, whole], refs[s][1][0, whole], dtype)
            within(o[0, :, here], refs[s][2][0, :, whole], refs[s][3][0, :, whole], dtype)
            scanned[s].append((u[0, here], y[0, here]))
            at += t[s]
            done[s] += t[s]
        assert torch.isfinite(n).all()
    conv_pool = conv_st[[1, 0]].contiguous()
    scan_pool = scan_st[[1, 0]].contiguous()
    for i in range(steps):
        cut = {n: torch.stack([text[s][n][done[s]] for s in range(2)]).to(DEV) for n in text[0]}
        u = cla.short_conv_step(cut["x"], dev["w"], conv_pool, dev["bias"], True, slots)
        y = cla.selective_scan_step(u, cut["dt"], dev["A"], cut["B"], cut["C"], scan_pool, dev["D"],
                                    dev["dt_bias"], slots=slots)
        o = cla.window_attention_step(cut["q"], cut["k"], cut["v"], ck, cv, ints(done), window, sinks,
                                      slots=slots)
        for s in range(2):
            within(u[s], refs[s][0][0, done[s]], refs[s][1][0, done[s]], dtype)
            within(o[s], refs[s][2][0, :, done[s]], refs[s][3][0, :, done[s]], dtype)
            scanned[s].append((u[s:s + 1], y[s:s + 1]))
            done[s] += 1
    torch.cuda.synchronize()
    assert_status_ok(cla)
    for s in range(2):   # the scan over the rounded outputs of the convolution
        u, y = (f64(torch.cat(x)) for x in zip(*scanned[s]))
        ro, rh, eo, eh = MO.selective_scan(u[None], *[f64(text[s][n])[None] for n in ("dt",)],
                                           f64(L["A"]), f64(text[s]["B"])[None],
                                           f64(text[s]["C"])[None], f64(L["D"]), f64(L["dt_bias"]))
        within(torch.from_numpy(y), ro[0], eo[0], dtype)
        within(scan_pool[1 - s], rh[0], eh[0], F32)


def test_capture_and_other_streams():
    """Calls captured into graphs and replayed with other inputs and bounds, and two
    streams at once, give what plain calls give."""
    cla = lib()
    r = gen(70)
    q, k, v = (r(1, 4, 300, 128).to(DEV, BF16) for _ in range(3))
    t = [y.to(DEV) for y in scan_inputs(71, 1, 2600, 1024, 16, 1, BF16)]
    w = r(1024, 4).to(DEV)
    st_a, st_b = ints([0, 100, 300]), ints([0, 250, 260])
    sc_a, sc_b = ints([0, 1000, 2600]), ints([0, 5, 2000])
    c0 = [torch.randn(2, 4, 70, 128, device=DEV, dtype=BF16) for _ in range(2)]
    past = ints([33, 100])

    def calls(qq, starts, scan_starts, c):
        return (cla.window_attention_forward(qq, k, v, 66, 4, cache_k=c[0], cache_v=c[1], past=past,
                                             seq_starts=starts),
                *cla.selective_scan_forward(*t[:5], t[5], t[6], t[7], seq_starts=scan_starts),
                *cla.short_conv_forward(t[0], w, None, True, seq_starts=scan_starts),
                cla.window_attention_step(qq[0, :, :2].transpose(0, 1), k[0, :, :2].transpose(0, 1),
                                          v[0, :, :2].transpose(0, 1), c[0], c[1], past, 66, 4))

    q2 = (q * 0.5).contiguous()
    want, seen = [], []
    for qq, a, b in ((q, st_a, sc_a), (q2, st_b, sc_b)):
        c = [x.clone() for x in c0]
        want.append([x.clone() for x in calls(qq, a, b, c)] + c)
    sq, sa, sb, sc = q.clone(), st_a.clone(), sc_a.clone(), [x.clone() for x in c0]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = calls(sq, sa, sb, sc)
    for qq, a, b in ((q, st_a, sc_a), (q2, st_b, sc_b)):
        sq.copy_(qq)
        sa.copy_(a)
        sb.copy_(b)
        for x, y in zip(sc, c0):
            x.copy_(y)
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        seen.append([x.clone() for x in outs] + [x.clone() for x in sc])
    held = [[slice(0, 300), slice(0, 2600)], [slice(0, 260), slice(0, 2000)]]
    for (x, y), (ha, hs) in zip(zip(want, seen), held):
        assert torch.equal(x[0][:, :, ha], y[0][:, :, ha])
        assert torch.equal(x[1][:, hs], y[1][:, hs]) and torch.equal(x[3][:, hs], y[3][:, hs])
        for i in (2, 4, 5, 6, 7):
            assert torch.equal(x[i], y[i])
    streams = [torch.cuda.Stream() for _ in range(2)]
    cs = [[x.clone() for x in c0] for _ in streams]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        got = []
        for s, c, (qq, a, b) in zip(streams, cs, ((q, st_a, sc_a), (q2, st_b, sc_b))):
            with torch.cuda.stream(s):
                for x, y in zip(c, c0):
                    x.copy_(y)
                got.append(calls(qq, a, b, c))
    torch.cuda.synchronize()
    for x, y, (ha, hs) in zip(want, got, held):
        assert torch.equal(x[0][:, :, ha], y[0][:, :, ha])
        assert torch.equal(x[1][:, hs], y[1][:, hs]) and torch.equal(x[5], y[5])
    assert_status_ok(cla)
