"""The gated delta rule on the GPU (whole sequences and single tokens) against
the fp64 oracle.

Tolerances, as relative L2 errors, from the roundings on each path:
  * outputs in bf16 are rounded once, at most half a step, 2^-8 of each value;
    fp32 outputs 2^-24.
  * token by token in fp32: every operation rounds by 2^-24; a state element
    sees about d_k + 4 of them per token in its row's product and they decay
    with it, so 1e-5 (168 * 2^-24) holds without any cancelling of errors.
  * chunks on the tensor cores: each of the four intermediates of a chunk (the
    state, K S^T, (1 + A)^-1 and X) is held as a pair of bf16 numbers, off by at
    most 2^-17, and a product of two pairs leaves out the low parts' product
    (2^-18): 4 * 2^-17 + 2 * 2^-18 = 3.9e-5.
The tests' keys have unit length and beta lies in [0, 1], so that errors of a
state are not enlarged by later tokens.
"""
import numpy as np
import pytest
import torch

from oracle import delta_oracle as DO
from tests.gpu_util import assert_status_ok, f64, lib, rel_l2

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
STATE_F32, STATE_BF16 = 1e-5, 3.9e-5
OUT = {torch.float32: STATE_F32 + 2.0 ** -24, torch.bfloat16: 2.0 ** -8 + STATE_BF16}
TTT_ERR_ARG = -8


def inputs(seed, B, Hk, Hv, N, dk, dv, dtype, decay=0.5, mean=0.0):
    gen = torch.Generator().manual_seed(seed)

    def r(*s):
        return torch.randn(s, generator=gen)

    q = torch.nn.functional.normalize(r(B, Hk, N, dk) + mean, dim=-1).to(dtype)
    k = torch.nn.functional.normalize(r(B, Hk, N, dk) + mean, dim=-1).to(dtype)
    v = r(B, Hv, N, dv).to(dtype)
    g = -decay * torch.nn.functional.softplus(r(B, Hv, N))
    return q, k, v, g, torch.sigmoid(r(B, Hv, N))


def check(cla, got, ref, dtype, state_tol=None):
    o, S = got
    ro, rS = ref
    assert_status_ok(cla)
    tol = state_tol or (STATE_F32 if dtype == torch.float32 else STATE_BF16)
    held = ~np.isnan(ro)
    assert rel_l2(f64(o)[held], ro[held]) <= OUT[dtype]
    assert rel_l2(f64(S), rS) <= tol


def run(cla, t, S0=None, starts=None, **kw):
    dev = [x.to(DEV) for x in t]
    res = cla.delta_rule_chunked_forward(
        *dev, S0=None if S0 is None else S0.to(DEV),
        seq_starts=None if starts is None else torch.tensor(starts, dtype=torch.int32, device=DEV),
        **kw)
    torch.cuda.synchronize()
    return res


def oracle(t, S0=None, starts=None, **kw):
    return DO.delta_rule(*[f64(x) for x in t], None if S0 is None else f64(S0), starts, **kw)


SIZES = [
    # B, Hk, Hv, N, dk, dv
    (1, 1, 1, 1, 128, 128),
    (1, 2, 2, 63, 128, 128),
    (2, 1, 2, 64, 128, 128),
    (1, 2, 4, 65, 128, 128),
    (1, 1, 3, 200, 128, 128),
    (2, 2, 2, 129, 64, 64),
    (1, 1, 1, 190, 96, 72),
    (1, 1, 2, 131, 128, 256),
    (1, 1, 1, 100, 32, 40),
    (1, 1, 1, 70, 256, 64),
    (1, 1, 1, 50, 512, 48),
    (1, 1, 1, 40, 33, 17),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_sizes(size, dtype):
    cla = lib()
    t = inputs(1, *size, dtype)
    B, Hk, Hv, N, dk, dv = size
    S0 = torch.randn(B, Hv, dv, dk, generator=torch.Generator().manual_seed(2)) * 0.3
    check(cla, run(cla, t, S0), oracle(t, S0), dtype)
    check(cla, run(cla, t), oracle(t), dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("decay,mean", [(0.0, 0.0), (0.002, 1.0), (8.0, 0.3), (60.0, 0.0)])
def test_decays_and_correlated_keys(decay, mean, dtype):
    """From no forgetting to forgetting within a token, with keys that share a
    direction (far from orthogonal writes)."""
    cla = lib()
    t = inputs(3, 1, 1, 2, 300, 128, 128, dtype, decay, mean)
    check(cla, run(cla, t), oracle(t), dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_extreme_gates(dtype):
    """beta of 0, 1 and 2, g of 0 and -inf (a token that clears the state), the
    same key written again and again."""
    cla = lib()
    q, k, v, g, b = inputs(4, 1, 1, 1, 192, 64, 64, dtype)
    b[..., 0:20] = 0.0
    b[..., 20:60] = 1.0
    b[..., 60:64] = 2.0
    g[..., 30:50] = 0.0
    g[..., 100] = -float("inf")
    g[..., 128] = -float("inf")
    k[:, :, 140:180] = k[:, :, 140:141]
    t = (q, k, v, g, b)
    check(cla, run(cla, t), oracle(t), dtype)


PACKS = [[0, 1, 1, 65, 129, 129, 200], [0, 0, 0, 64], [3, 70, 71, 150], [0, 200]]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("starts", PACKS, ids=str)
def test_packed_sequences(starts, dtype):
    """Lengths of zero and one, sequences that end inside a chunk, rows before
    and behind the sequences left as they were; token-major inputs."""
    cla = lib()
    N, dk, dv, Hk, Hv = 208, 128, 128, 1, 2
    t = [x.transpose(1, 2).contiguous().transpose(1, 2)
         for x in inputs(5, 1, Hk, Hv, N, dk, dv, dtype)]
    n = len(starts) - 1
    S0 = torch.randn(n, Hv, dv, dk, generator=torch.Generator().manual_seed(6)) * 0.3
    ref = oracle(t, S0, starts)
    out = torch.full((1, N, Hv, dv), 7.0, dtype=dtype, device=DEV).transpose(1, 2)
    got = run(cla, t, S0, starts, out=out)
    check(cla, got, ref, dtype)
    assert (f64(got[0])[np.isnan(ref[0])] == 7.0).all()
    empty = [s for s in range(n) if starts[s] == starts[s + 1]]
    for s in empty:
        assert torch.equal(got[1][s].cpu(), S0[s])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_values_of_other_tokens_do_not_leak(dtype):
    """NaN and infinity in the tokens of other sequences, and of none, reach
    neither outputs nor states."""
    cla = lib()
    starts = [5, 75, 139]
    t = inputs(7, 1, 1, 2, 208, 128, 128, dtype)
    ref = oracle(t, None, starts)
    for x in t:
        x[:, :, :5] = float("nan")
        x[:, :, 139:] = float("inf")
    check(cla, run(cla, t, None, starts), ref, dtype)
    # the second sequence alone is spoilt
    t = inputs(7, 1, 1, 2, 208, 128, 128, dtype)
    t[2][:, :, 75:139] = float("nan")
    o, S = run(cla, t, None, starts)
    assert rel_l2(f64(o)[:, :, 5:75], ref[0][:, :, 5:75]) <= OUT[dtype]
    assert rel_l2(f64(S)[0], ref[1][0]) <= STATE_BF16
    assert torch.isnan(S[1]).any()


def test_bad_bounds_are_reported():
    """Bounds that descend or leave the token axis: those sequences are empty,
    the status says so, the others are computed."""
    cla = lib()
    t = inputs(8, 1, 1, 1, 100, 128, 128, torch.bfloat16)
    S0 = torch.randn(4, 1, 128, 128, generator=torch.Generator().manual_seed(9))
    for starts, good in (([0, 40, 30, 100, 130], {0: (0, 40), 2: (30, 100)}),
                         ([-1, 10, 100, 2 ** 31 - 1, -2 ** 31], {1: (10, 100)})):
        o, S = run(cla, t, S0, starts)
        assert cla.device_status() == TTT_ERR_ARG
        assert cla.device_status() == 0
        for s in range(4):
            if s not in good:
                assert torch.equal(S[s].cpu(), S0[s])
            else:
                a, e = good[s]
                ref = DO.delta_rule(*[f64(x)[:, :, a:e] for x in t], f64(S0[s:s + 1]))
                assert rel_l2(f64(S[s:s + 1]), ref[1]) <= STATE_BF16


def test_overlapping_bounds_stay_inside_the_tensors():
    """Bounds that go back and forth describe more chunks than the token axis
    holds: the descending ones are empty, the call reports and ends, and
    nothing around the outputs and states is touched."""
    cla = lib()
    N, n = 1000, 10
    t = inputs(48, 1, 1, 1, N, 128, 128, torch.bfloat16)
    S0 = torch.randn(n, 1, 128, 128, generator=torch.Generator().manual_seed(49))
    room = torch.full((1, 1, N + 2, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    states = torch.full((n + 2, 1, 128, 128), 4.0, device=DEV)
    run(cla, t, S0, [0, N] * 5 + [0], out=room[:, :, 1:-1], S_final=states[1:-1])
    assert cla.device_status() == TTT_ERR_ARG
    assert (room[:, :, 0] == 3.0).all() and (room[:, :, -1] == 3.0).all()
    assert (states[0] == 4.0).all() and (states[-1] == 4.0).all()
    for s in range(1, n, 2):
        assert torch.equal(states[1 + s].cpu(), S0[s])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_layouts(dtype):
    """Strided views: slices of one projection, a wider head dimension, odd
    offsets (which the wide loads cannot take), g of stride 0 over the batch."""
    cla = lib()
    B, Hk, Hv, N, d = 2, 1, 2, 90, 64
    q, k, v, g, b = inputs(10, B, Hk, Hv, N, d, d, dtype)
    g = g[:1]
    ref = DO.delta_rule(f64(q), f64(k), f64(v), np.broadcast_to(f64(g), (B, Hv, N)), f64(b))
    for lead in (0, 8, 3):
        wide = torch.zeros(B, N, lead + d * (2 * Hk + Hv), dtype=dtype)
        parts = (q.transpose(1, 2).reshape(B, N, -1), k.transpose(1, 2).reshape(B, N, -1),
                 v.transpose(1, 2).reshape(B, N, -1))
        wide[:, :, lead:] = torch.cat(parts, -1)
        w = wide.to(DEV)[:, :, lead:]
        qq = w[..., :d].unflatten(-1, (Hk, d)).transpose(1, 2)
        kk = w[..., d:2 * d].unflatten(-1, (Hk, d)).transpose(1, 2)
        vv = w[..., 2 * d:].unflatten(-1, (Hv, d)).transpose(1, 2)
        res = cla.delta_rule_chunked_forward(qq, kk, vv, g.to(DEV).expand(B, Hv, N), b.to(DEV))
        torch.cuda.synchronize()
        check(cla, res, ref, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_split_calls_carry_the_state(dtype):
    """A prompt in two calls equals one call; the second updates S0 in place."""
    cla = lib()
    t = inputs(11, 1, 2, 2, 333, 128, 128, dtype)
    ref = oracle(t)
    d = [x.to(DEV) for x in t]
    o1, S = cla.delta_rule_chunked_forward(*[x[:, :, :190] for x in d])
    o2, S2 = cla.delta_rule_chunked_forward(*[x[:, :, 190:] for x in d], S0=S, S_final=S)
    torch.cuda.synchronize()
    check(cla, (torch.cat([o1, o2], 2), S2), ref, dtype, 2 * STATE_BF16)


def test_long_sequences_split_over_the_card():
    """Long sequences of few heads, dense and packed with a short one."""
    cla = lib()
    N = 5000
    t = inputs(12, 1, 1, 1, N, 128, 128, torch.bfloat16, 0.02)
    S0 = torch.randn(1, 1, 128, 128, generator=torch.Generator().manual_seed(13)) * 0.3
    check(cla, run(cla, t, S0), oracle(t, S0), torch.bfloat16)
    starts = [0, 3100, 3100, 3170, 5000]
    S0 = torch.randn(4, 1, 128, 128, generator=torch.Generator().manual_seed(14)) * 0.3
    check(cla, run(cla, t, S0, starts), oracle(t, S0, starts), torch.bfloat16)


SPLITS = [
    # B, Hk, Hv, N, dk, dv: four, eight and sixteen heads take the join's three
    # forms; two tiles of d_v, and head sizes below the tile's
    (1, 2, 4, 2000, 128, 128),
    (1, 2, 8, 1500, 128, 128),
    (1, 4, 16, 1400, 64, 128),
    (2, 2, 2, 1300, 128, 256),
    (1, 3, 6, 1290, 96, 72),
    (1, 2, 4, 1500, 64, 64),
    (1, 1, 8, 1300, 40, 136),
    (1, 6, 24, 2500, 128, 64),
    (1, 20, 20, 3000, 64, 256),
]


@pytest.mark.parametrize("size", SPLITS, ids=str)
def test_segments(size):
    """Sequences that are cut into segments: start states and outputs across
    the joins, weak forgetting so that they matter."""
    cla = lib()
    B, Hk, Hv, N, dk, dv = size
    t = inputs(40, *size, torch.bfloat16, 0.01)
    S0 = torch.randn(B, Hv, dv, dk, generator=torch.Generator().manual_seed(41)) * 0.3
    ref = oracle(t, S0)
    run(cla, t, S0)
    cla.profile_start()
    got = run(cla, t, S0)
    kinds = {e["name"] for e in cla.profile_stop()}
    assert {"delta.prep", "delta.carry", "delta.join", "delta.chunk"} <= kinds
    check(cla, got, ref, torch.bfloat16)
    # the states in place, over a call that keeps the card busy on another stream
    S, busy = S0.to(DEV), torch.cuda.Stream()
    dev = [x.to(DEV) for x in t]
    torch.cuda.synchronize()
    other = cla.delta_rule_chunked_forward(*dev, stream=busy)
    o, S = cla.delta_rule_chunked_forward(*dev, S0=S, S_final=S)
    torch.cuda.synchronize()
    assert torch.equal(o, got[0]) and torch.equal(S, got[1]) and other is not None


@pytest.mark.parametrize("dk,dv", [(128, 128), (72, 40)])
def test_states_that_begin_in_the_middle_of_32_bytes(dk, dv):
    """Initial and final states 16 bytes behind an allocation's start."""
    cla = lib()
    t = inputs(46, 1, 1, 2, 200, dk, dv, torch.bfloat16)
    S0 = torch.randn(1, 2, dv, dk, generator=torch.Generator().manual_seed(47)) * 0.3
    n = S0.numel()
    room = torch.full((2, n + 8), 5.0, device=DEV)
    first, last = (r[4:4 + n].view(1, 2, dv, dk) for r in room)
    first.copy_(S0)
    assert first.data_ptr() % 32 == 16
    got = run(cla, t, first, S_final=last)
    check(cla, got, oracle(t, S0), torch.bfloat16)
    assert (room[:, :4] == 5.0).all() and (room[:, 4 + n:] == 5.0).all()


@pytest.mark.parametrize("d", [64, 128])
def test_many_packed_sequences(d):
    """More sequences than the plan's block has threads, one of them long."""
    cla = lib()
    gen = torch.Generator().manual_seed(42)
    lens = torch.randint(0, 40, (300,), generator=gen).tolist()
    lens[77], lens[299] = 1500, 65
    starts = [0] + torch.tensor(lens).cumsum(0).tolist()
    t = inputs(43, 1, 1, 2, starts[-1] + 3, d, d, torch.bfloat16, 0.05)
    S0 = torch.randn(300, 2, d, d, generator=gen) * 0.3
    check(cla, run(cla, t, S0, starts), oracle(t, S0, starts), torch.bfloat16)


@pytest.mark.parametrize("lens", [[2600, 60, 1, 0, 700], [640] * 6, [90] * 40, [64] * 250 + [5000]],
                         ids=["one_long", "equal", "short", "many"])
def test_packed_lengths_that_are_cut_differently(lens):
    """Packed sequences that the plan cuts into long or short segments, or not
    at all, with two value heads per key head."""
    cla = lib()
    starts = [0] + torch.tensor(lens).cumsum(0).tolist()
    t = inputs(50, 1, 2, 4, starts[-1], 64, 128, torch.bfloat16, 0.02)
    S0 = torch.randn(len(lens), 4, 128, 64, generator=torch.Generator().manual_seed(51)) * 0.3
    a = run(cla, t, S0, starts)
    check(cla, a, oracle(t, S0, starts), torch.bfloat16)
    b = run(cla, t, S0, starts)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_captured_packed_call_with_other_lengths():
    """A captured packed call is planned on the device: replayed with other
    bounds it equals a call made with them."""
    cla = lib()
    N = 3000
    t = inputs(54, 1, 1, 2, N, 128, 128, torch.bfloat16, 0.02)
    S0 = torch.randn(4, 2, 128, 128, generator=torch.Generator().manual_seed(55)) * 0.3
    packs = ([0, 700, 1400, 2200, 3000], [0, 10, 10, 2950, 2951], [5, 2900, 2930, 2964, 3000])
    want = [run(cla, t, S0, p) for p in packs]
    dev, S0d = [x.to(DEV) for x in t], S0.to(DEV)
    starts = torch.tensor(packs[0], dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, S = cla.delta_rule_chunked_forward(*dev, S0=S0d, seq_starts=starts)
    for p, (ro, rS) in zip(packs[::-1], want[::-1]):
        starts.copy_(torch.tensor(p, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(S, rS)
        assert torch.equal(o[:, :, p[0]:p[-1]], ro[:, :, p[0]:p[-1]])
    check(cla, want[1], oracle(t, S0, packs[1]), torch.bfloat16)


def test_zero_length_axis_edges_and_one_token_sequences():
    """A packed batch of single tokens, and one in which every sequence is
    empty: outputs untouched, states unchanged."""
    cla = lib()
    t = inputs(44, 1, 2, 2, 9, 128, 128, torch.bfloat16)
    S0 = torch.randn(9, 2, 128, 128, generator=torch.Generator().manual_seed(45))
    check(cla, run(cla, t, S0, list(range(10))), oracle(t, S0, list(range(10))), torch.bfloat16)
    out = torch.full((1, 2, 9, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    o, S = run(cla, t, S0[:4], [5, 5, 5, 5, 5], out=out)
    assert_status_ok(cla)
    assert (o == 3.0).all() and torch.equal(S.cpu(), S0[:4])


def test_same_call_twice_gives_the_same_bits():
    cla = lib()
    t = inputs(15, 2, 1, 2, 1000, 128, 128, torch.bfloat16)
    a, b = run(cla, t), run(cla, t)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_two_streams_and_a_captured_graph():
    """Two calls on streams of their own, and a captured call that is replayed
    on new inputs, equal the plain call."""
    cla = lib()
    sets = [inputs(s, 1, 1, 2, 700, 128, 128, torch.bfloat16) for s in (16, 17)]
    want = [run(cla, t) for t in sets]
    dev = [[x.to(DEV) for x in t] for t in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [cla.delta_rule_chunked_forward(*d, stream=s) for d, s in zip(dev, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    hold = [x.clone() for x in dev[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = cla.delta_rule_chunked_forward(*hold)
    for i in (1, 0):
        for x, y in zip(hold, dev[i]):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(res[0], want[i][0]) and torch.equal(res[1], want[i][1])
    assert_status_ok(cla)


# ---------------------------------------------------------------- single tokens

STEPS = [
    # B, Hk, Hv, dk, dv
    (1, 1, 1, 128, 128), (3, 2, 4, 128, 128), (5, 1, 2, 64, 64), (2, 1, 1, 96, 72),
    (2, 1, 2, 256, 40), (1, 1, 1, 512, 33), (4, 3, 3, 32, 32), (2, 1, 1, 37, 19),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("size", STEPS, ids=str)
def test_step(size, dtype):
    cla = lib()
    B, Hk, Hv, dk, dv = size
    t = inputs(20, B, Hk, Hv, 1, dk, dv, dtype)
    S = torch.randn(B + 2, Hv, dv, dk, generator=torch.Generator().manual_seed(21))
    slots = torch.randperm(B + 2, generator=torch.Generator().manual_seed(22))[:B]
    pool = S.to(DEV)
    o = cla.delta_rule_step(*[x[:, :, 0].to(DEV) for x in t], pool,
                            slots=slots.to(torch.int32).to(DEV))
    torch.cuda.synchronize()
    assert_status_ok(cla)
    ro, rS = oracle(t, S[slots])
    assert rel_l2(f64(o), ro[:, :, 0]) <= OUT[dtype]
    assert rel_l2(f64(pool[slots.to(DEV)]), rS) <= STATE_F32
    rest = [i for i in range(B + 2) if i not in slots.tolist()]
    assert torch.equal(pool[rest].cpu(), S[rest])


def test_step_without_slots_and_with_strided_inputs():
    cla = lib()
    B, Hk, Hv, d = 3, 2, 4, 128
    t = inputs(23, B, Hk, Hv, 1, d, d, torch.bfloat16)
    wide = torch.cat([x[:, :, 0].reshape(B, -1) for x in t[:3]], -1).to(DEV)
    q, k, v = (x.unflatten(-1, (-1, d)) for x in wide.split((Hk * d, Hk * d, Hv * d), -1))
    S = torch.randn(B, Hv, d, d, generator=torch.Generator().manual_seed(24))
    pool = S.to(DEV)
    out = torch.zeros(B, Hv, 2 * d, dtype=torch.bfloat16, device=DEV)
    cla.delta_rule_step(q, k, v, t[3][:, :, 0].to(DEV), t[4][:, :, 0].to(DEV), pool, scale=0.7,
                        out=out[..., d:])
    torch.cuda.synchronize()
    assert_status_ok(cla)
    ro, rS = oracle(t, S, scale=0.7)
    assert rel_l2(f64(out[..., d:]), ro[:, :, 0]) <= OUT[torch.bfloat16]
    assert rel_l2(f64(pool), rS) <= STATE_F32
    assert (out[..., :d] == 0).all()


def test_step_idle_foreign_and_repeated_slots():
    """Idle rows (NaN inputs) give zeros and touch no state; a slot outside the
    pool and the second use of a slot do the same and are reported."""
    cla = lib()
    B, Hv, d = 6, 2, 128
    t = inputs(25, B, 1, Hv, 1, d, d, torch.bfloat16)
    S = torch.randn(4, Hv, d, d, generator=torch.Generator().manual_seed(26))
    for i in (1, 3, 4):
        for x in t:
            x[i] = float("nan")
    for slots, live, bad in (([2, -1, 0, -5, -1, 3], {0: 2, 2: 0, 5: 3}, False),
                             ([2, -1, 0, 4, 2, 1], {0: 2, 2: 0, 5: 1}, True),
                             ([2, -1, 0, 2 ** 31 - 1, -2 ** 31, 1], {0: 2, 2: 0, 5: 1}, True)):
        pool = S.to(DEV)
        o = cla.delta_rule_step(*[x[:, :, 0].to(DEV) for x in t], pool,
                                slots=torch.tensor(slots, dtype=torch.int32, device=DEV))
        assert cla.device_status() == (TTT_ERR_ARG if bad else 0)
        for b in range(B):
            if b in live:
                ro, rS = oracle([x[b:b + 1] for x in t], S[live[b]][None])
                assert rel_l2(f64(o[b]), ro[0, :, 0]) <= OUT[torch.bfloat16]
                assert rel_l2(f64(pool[live[b]]), rS[0]) <= STATE_F32
            else:
                assert (o[b] == 0).all()
        for s in set(range(4)) - set(live.values()):
            assert torch.equal(pool[s].cpu(), S[s])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_prompt_then_tokens(dtype):
    """A served sequence: the prompt in chunks into pool states, then tokens one
    by one, each step replayed from one captured graph; equals the rule over
    the whole sequence."""
    cla = lib()
    B, Hk, Hv, N, d, new = 2, 1, 2, 150, 128, 9
    t = inputs(27, B, Hk, Hv, N + new, d, d, dtype)
    ref = oracle(t)
    dev = [x.to(DEV) for x in t]
    pool = torch.zeros(5, Hv, d, d, device=DEV)
    slots = torch.tensor([3, 1], dtype=torch.int32, device=DEV)
    o, S = cla.delta_rule_chunked_forward(*[x[:, :, :N] for x in dev])
    pool[slots.long()] = S
    hold = [x[:, :, N].clone() for x in dev]
    keep = pool.clone()
    cla.delta_rule_step(*hold, pool, slots=slots)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step = cla.delta_rule_step(*hold, pool, slots=slots)
    pool.copy_(keep)
    outs = [o]
    for i in range(new):
        for x, y in zip(hold, dev):
            x.copy_(y[:, :, N + i])
        graph.replay()
        outs.append(step.clone()[:, :, None])
    torch.cuda.synchronize()
    check(cla, (torch.cat(outs, 2), pool[slots.long()]), ref, dtype, STATE_BF16 + STATE_F32)
