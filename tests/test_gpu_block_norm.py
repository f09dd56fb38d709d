"""The norms around a block on the GPU against the fp64 oracle.

Tolerances: everything is computed in fp32; a mean of D squares summed as a
tree in pieces of at most 128 terms, a reciprocal square root (2 ulp), an exp
(2 ulp) and about ten multiplications are off by less than 64 * 2^-24 = 3.8e-6
of a value; a bf16 result adds half a step, 2^-8 of each value.
"""
import itertools

import pytest
import torch

from oracle import delta_oracle as DO
from tests.gpu_util import f64, lib, rel_l2

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
TOL = {F32: 3.8e-6, BF: 2.0 ** -8 + 3.8e-6}


def make(seed, rows, D, group, io, st, act, residual, scale, nxt):
    gen = torch.Generator().manual_seed(seed)

    def r(*s):
        return torch.randn(s, generator=gen)

    return dict(y=(3 * r(rows, D)).to(io), w=1 + 0.1 * r(group),
                gate=r(rows, D).to(io) if act else None, gate_act=act,
                residual=r(rows, D).to(st) if residual else None,
                scale=r(D) if scale else None, w_next=1 + 0.1 * r(D) if nxt else None)


def want(t, group, eps=1e-6):
    return DO.block_norm(f64(t["y"]), *[None if t[n] is None else f64(t[n])
                                        for n in ("w", "gate")], t["gate_act"],
                         *[None if t[n] is None else f64(t[n])
                           for n in ("residual", "scale", "w_next")], group=group, eps=eps)


def on(t):
    return {k: v.to(DEV) if isinstance(v, torch.Tensor) else v for k, v in t.items()}


def check(got, ref, io, st):
    flat = [None if x is None else f64(x).reshape(ref[0].shape) for x in got]
    assert got[0].dtype == st and rel_l2(flat[0], ref[0]) <= TOL[st]
    if ref[1] is None:
        assert got[1] is None
    else:
        assert got[1].dtype == io and rel_l2(flat[1], ref[1]) <= TOL[io]


@pytest.mark.parametrize("io,st", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)], ids=str)
@pytest.mark.parametrize("rows,D,group", [
    (1, 64, 64), (3, 1536, 1536), (2, 1536, 384), (5, 1024, 128), (4, 1000, 1000), (3, 384, 96),
    (2, 7, 7), (3, 30, 10), (2, 5000, 1000), (1, 16384, 16384), (2, 16384, 64), (1, 16383, 3),
    (2, 1, 1), (300, 48, 16)], ids=str)
def test_sizes(rows, D, group, io, st):
    cla = lib()
    for act, residual, scale, nxt in ((0, True, True, True), (1, False, False, False),
                                      (2, True, False, True)):
        t = make(1, rows, D, group, io, st, act, residual, scale, nxt)
        got = cla.block_norm_forward(**on(t), out_dtype=st)
        torch.cuda.synchronize()
        check(got, want(t, group), io, st)


@pytest.mark.parametrize("io,st", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)], ids=str)
@pytest.mark.parametrize("rows,D,group", [
    (3, 2040, 2040), (400, 1537, 1537), (2, 4095, 4095), (2, 4096, 4096), (700, 4096, 128),
    (2, 6144, 6144), (300, 8192, 8192), (200, 8200, 1640), (2, 6000, 24), (170, 16384, 16384),
    (160, 16383, 16383)], ids=str)
def test_groups_of_many_partial_sums_and_long_rows(rows, D, group, io, st):
    """Groups whose elements halve few times (many partial sums), and the
    forms of rows above 2048, with several rows per block."""
    cla = lib()
    t = make(6, rows, D, group, io, st, 1, True, True, True)
    check(cla.block_norm_forward(**on(t), out_dtype=st), want(t, group), io, st)


def test_every_choice_of_parts():
    cla = lib()
    for act, residual, scale, nxt in itertools.product((0, 1, 2), *[(False, True)] * 3):
        t = make(2, 6, 256, 64, BF, BF, act, residual, scale, nxt)
        check(cla.block_norm_forward(**on(t)), want(t, 64), BF, BF)
    t = make(3, 6, 256, 64, BF, BF, 0, False, False, False)
    t["w"] = None
    check(cla.block_norm_forward(**on(t), group=32), want(t, 32), BF, BF)


def test_zero_rows_large_values_and_large_gates():
    """A row of zeros stays zero before the residual, large values do not
    overflow the sum of squares, gates saturate."""
    cla = lib()
    t = make(4, 4, 512, 128, F32, F32, 2, True, True, True)
    t["y"][0] = 0
    t["y"][1] *= 1e16
    t["y"][2] *= 1e-16
    t["gate"][3, ::2] = 200.0
    t["gate"][3, 1::2] = -200.0
    check(cla.block_norm_forward(**on(t)), want(t, 128), F32, F32)


def test_strided_rows_and_in_place():
    """Rows inside wider rows (aligned and odd offsets), a [B, N, D] view, out
    over the residual, out over y."""
    cla = lib()
    for lead in (0, 8, 3):
        t = make(5, 12, 256, 64, BF, BF, 1, True, True, True)
        ref = want(t, 64)
        d = on(t)
        for n in ("y", "gate", "residual"):
            wide = torch.zeros(12, lead + 256 + 8, dtype=BF, device=DEV)
            wide[:, lead:lead + 256] = d[n]
            d[n] = wide[:, lead:lead + 256].unflatten(0, (3, 4))
        out = torch.full((12, 300), 7.0, dtype=BF, device=DEV)
        got = cla.block_norm_forward(**d, out=out[:, :256])
        check(got, ref, BF, BF)
        assert (out[:, 256:] == 7.0).all()
    d = on(t)
    got = cla.block_norm_forward(**d, out=d["residual"])
    check(got, ref, BF, BF)
    assert got[0].data_ptr() == d["residual"].data_ptr()
    d = on(t)
    check(cla.block_norm_forward(**d, out=d["y"]), ref, BF, BF)


def test_rule_then_norm():
    """The layer's run as it is served: the rule's output, token-major, through
    the heads' norm and gate, then the norms around the block."""
    cla = lib()
    from tests.test_gpu_delta_rule import inputs
    B, H, N, d = 2, 2, 100, 128
    q, k, v, g, b = inputs(30, B, H, H, N, d, d, BF)
    v = v.transpose(1, 2).contiguous().transpose(1, 2)
    o, _ = cla.delta_rule_chunked_forward(*[x.to(DEV) for x in (q, k, v, g, b)])
    y = o.transpose(1, 2).reshape(B, N, H * d)
    assert y.data_ptr() == o.data_ptr()
    t = make(31, B * N, H * d, d, BF, BF, 1, False, False, False)
    m, _ = cla.block_norm_forward(y, w=t["w"].to(DEV), gate=t["gate"].to(DEV).view(B, N, -1),
                                  gate_act=cla.GATE_SILU)
    ro, _ = DO.delta_rule(*[f64(x) for x in (q, k, v, g, b)])
    t["y"] = torch.from_numpy(ro).transpose(1, 2).reshape(B * N, H * d).to(BF)
    ref = want(t, d)
    # the rule's own error of 2^-8 + 3.9e-5 per value passes through the norm once
    assert rel_l2(f64(m).reshape(B * N, -1), ref[0]) <= 2 * (2.0 ** -8 + 4e-5)
    t2 = make(32, B * N, H * d, H * d, BF, F32, 0, True, True, True)
    got = cla.block_norm_forward(m, w=t2["w"].to(DEV), residual=t2["residual"].to(DEV).view(
        B, N, -1), scale=t2["scale"].to(DEV), w_next=t2["w_next"].to(DEV))
    t2["y"] = m.reshape(B * N, -1).cpu()
    check((got[0].reshape(B * N, -1), got[1].reshape(B * N, -1)), want(t2, H * d), BF, F32)


def test_a_captured_layer_between_copies():
    """Rule, token and norm captured behind copies and fills, with copies
    behind them, replayed on new inputs."""
    cla = lib()
    from tests.test_gpu_delta_rule import inputs
    B, H, N, d = 2, 2, 150, 128
    sets = [[x.to(DEV) for x in inputs(s, B, H, H, N + 1, d, d, BF)] for s in (60, 61)]
    hold = [torch.empty_like(x) for x in sets[0]]
    keep = torch.empty(B, H * d, dtype=BF, device=DEV)
    state = torch.empty(B, H, d, d, device=DEV)
    saved = torch.empty_like(state)

    def layer(src):
        for x, y in zip(hold, src):
            x.copy_(y)
        state.zero_()
        o, _ = cla.delta_rule_chunked_forward(*[x[:, :, :N] for x in hold], S0=state, S_final=state)
        o1 = cla.delta_rule_step(*[x[:, :, N] for x in hold], state)
        n, _ = cla.block_norm_forward(o1.view(B, H * d), group=d)
        keep.copy_(n)
        saved.copy_(state)

    want = []
    for s in sets:
        layer(s)
        want.append((keep.clone(), saved.clone()))
    stage = [x.clone() for x in sets[0]]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(stage)
    for i in (1, 0, 1):
        for x, y in zip(stage, sets[i]):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(keep, want[i][0]) and torch.equal(saved, want[i][1])
    ro, rS = DO.delta_rule(*[f64(x) for x in sets[1]])
    assert rel_l2(f64(saved), rS) <= 3.9e-5 + 1e-5
    ref, _ = DO.block_norm(ro[:, :, N].reshape(B, H * d), group=d)
    assert rel_l2(f64(keep), ref) <= 2 * (2.0 ** -8 + 4e-5)
