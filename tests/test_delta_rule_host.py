"""Host-side checks of the delta-rule and norm entry points (no GPU): bad
arguments are refused with the documented codes before the device is touched."""
import itertools
import struct

import pytest
import torch

from tests.test_capi_host import (TTT_ERR_ALIGN, TTT_ERR_ARG, TTT_ERR_CUDA, TTT_ERR_NULL,
                                  TTT_ERR_SHAPE, TTT_ERR_UNSUPPORTED, TTT_ERR_WORKSPACE, cla,
                                  fake)

__all__ = ["cla"]


def rule(cla, B=1, Hk=1, Hv=2, N=64, dk=64, dv=64, n_seq=None, io=1, scale=1.0, packed=False,
         lay=None, nulls=(), ws=None, off=(), S0=True, out=7):
    n_seq = B if n_seq is None else n_seq
    p = [fake(0x100000 * (i + 1) + (2 if i in off else 0)) for i in range(10)]
    p[7] = p[out]
    for i in nulls:
        p[i] = None
    q, k, v, g, b, s0, st, out, sf, wsp = p
    lib = cla.library()
    need = lib.delta_rule_workspace_size(B, Hk, Hv, N, dk, dv, n_seq, io)
    return lib.delta_rule_chunked_forward(
        q, k, v, g, b, s0 if S0 else None, st if packed else None, n_seq, B, Hk, Hv, N, dk, dv,
        io, scale, lay, out, sf, wsp,
        max(need, 256) if ws is None else ws, None)


def layout(cla, **change):
    s = [64 * 64, 64 * 64, 64] * 2 + [2 * 64 * 64, 64 * 64, 64] + [128, 64, 1] * 2 + [
        2 * 64 * 64, 64 * 64, 64]
    for at, x in change.items():
        s[int(at[1:])] = x
    return struct.pack("18q", *s)


def test_rule_refusals(cla):
    for i in (0, 1, 2, 3, 4, 7):
        assert rule(cla, nulls=(i,)) == TTT_ERR_NULL
    for bad in (dict(B=0), dict(N=0), dict(Hk=0), dict(dk=0), dict(dv=-1), dict(Hk=2, Hv=3),
                dict(n_seq=2), dict(B=2, n_seq=2, packed=True), dict(B=2, n_seq=3, packed=True)):
        assert rule(cla, **bad) == TTT_ERR_SHAPE, bad
    assert rule(cla, io=2) == TTT_ERR_ARG
    assert rule(cla, scale=float("nan")) == TTT_ERR_ARG
    assert rule(cla, dk=513) == TTT_ERR_UNSUPPORTED
    assert rule(cla, dv=1025) == TTT_ERR_UNSUPPORTED
    assert rule(cla, n_seq=1 << 20, packed=True) == TTT_ERR_UNSUPPORTED
    assert rule(cla, N=1 << 30) == TTT_ERR_UNSUPPORTED
    assert rule(cla, off=(5,)) == TTT_ERR_ALIGN          # S0
    assert rule(cla, off=(8,)) == TTT_ERR_ALIGN          # S_final
    assert rule(cla, off=(3,)) == TTT_ERR_ALIGN          # g: 4-byte
    assert rule(cla, off=(9,)) == TTT_ERR_ALIGN          # workspace
    assert rule(cla, ws=8) == TTT_ERR_WORKSPACE
    assert rule(cla, nulls=(9,)) == TTT_ERR_WORKSPACE
    assert rule(cla, lay=layout(cla, _2=-64)) == TTT_ERR_ARG
    assert rule(cla, lay=layout(cla, _17=0)) == TTT_ERR_ARG   # out rows on one another
    assert rule(cla, lay=layout(cla, _17=63)) == TTT_ERR_ARG
    assert rule(cla, lay=layout(cla, _16=63 * 64)) == TTT_ERR_ARG
    for i in (0, 1, 2):
        assert rule(cla, out=i) == TTT_ERR_ARG


def test_rule_workspace_size(cla):
    lib = cla.library()
    assert lib.delta_rule_workspace_size(4, 4, 4, 8192, 128, 128, 4, 1) >= 256
    assert lib.delta_rule_workspace_size(4, 4, 6, 8192, 128, 128, 4, 1) == 0
    assert lib.delta_rule_workspace_size(1, 4, 8, 8192, 128, 128, 24, 1) >= 256


def step(cla, B=2, Hk=1, Hv=2, dk=64, dv=64, n_slots=4, slots=True, io=1, scale=1.0, nulls=(),
         off=()):
    p = [fake(0x100000 * (i + 1) + (2 if i in off else 0)) for i in range(8)]
    for i in nulls:
        p[i] = None
    q, k, v, g, b, S, sl, out = p
    return cla.library().delta_rule_step(q, k, v, g, b, S, sl if slots else None, n_slots, B, Hk,
                                         Hv, dk, dv, io, scale, None, out, None)


def test_step_refusals(cla):
    for i in (0, 1, 2, 3, 4, 5, 7):
        assert step(cla, nulls=(i,)) == TTT_ERR_NULL
    for bad in (dict(B=0), dict(n_slots=0), dict(slots=False, n_slots=1), dict(Hk=2, Hv=3)):
        assert step(cla, **bad) == TTT_ERR_SHAPE, bad
    assert step(cla, io=7) == TTT_ERR_ARG
    assert step(cla, scale=float("inf")) == TTT_ERR_ARG
    assert step(cla, dk=1024) == TTT_ERR_UNSUPPORTED
    assert step(cla, B=1 << 20) == TTT_ERR_UNSUPPORTED
    assert step(cla, off=(5,)) == TTT_ERR_ALIGN
    assert step(cla, off=(6,)) == TTT_ERR_ALIGN


def norm(cla, rows=4, D=64, group=64, io=1, st=1, act=0, eps=1e-6, gate=False, nxt=False, h=None,
         strides=None, nulls=(), off=(), over=None):
    p = [fake(0x100000 * (i + 1) + (1 if i in off else 0)) for i in range(8)]
    if over:
        p[over[0]] = p[over[1]]
    for i in nulls:
        p[i] = None
    y, w, z, x, a, wn, out, hh = p
    h = nxt if h is None else h
    return cla.library().block_norm_forward(
        y, w, z if gate else None, x, a, wn if nxt else None, rows, D, group, io, st, act, eps,
        strides, out, hh if h else None, None)


def test_norm_refusals(cla):
    assert norm(cla, nulls=(0,)) == TTT_ERR_NULL
    assert norm(cla, nulls=(6,)) == TTT_ERR_NULL
    assert norm(cla, act=1) == TTT_ERR_NULL              # a gate without its tensor
    assert norm(cla, gate=True) == TTT_ERR_NULL          # and the other way round
    assert norm(cla, nxt=True, h=False) == TTT_ERR_NULL
    assert norm(cla, nxt=False, h=True) == TTT_ERR_NULL
    for bad in (dict(rows=0), dict(D=0), dict(group=0), dict(group=48)):
        assert norm(cla, **bad) == TTT_ERR_SHAPE, bad
    for bad in (dict(io=3), dict(st=-1), dict(act=3), dict(eps=-1.0), dict(eps=float("nan"))):
        assert norm(cla, **bad) == TTT_ERR_ARG, bad
    assert norm(cla, D=32768, group=32768) == TTT_ERR_UNSUPPORTED
    assert norm(cla, off=(0,)) == TTT_ERR_ALIGN
    assert norm(cla, strides=struct.pack("5q", 64, 0, 64, 32, 0)) == TTT_ERR_ARG     # rows of out overlap
    assert norm(cla, strides=struct.pack("5q", -64, 0, 64, 64, 0)) == TTT_ERR_ARG
    # out over another tensor's rows: only over the same ones, of the same type
    assert norm(cla, over=(6, 3), strides=struct.pack("5q", 64, 0, 0, 64, 0)) == TTT_ERR_ARG
    assert norm(cla, over=(6, 0), strides=struct.pack("5q", 128, 0, 64, 64, 0)) == TTT_ERR_ARG
    assert norm(cla, over=(6, 0), st=0) == TTT_ERR_ARG
    for i in (0, 2, 3, 6):
        assert norm(cla, gate=True, act=1, nxt=True, over=(7, i)) == TTT_ERR_ARG


def test_layouts_of_the_outputs(cla):
    """Every order of the axes passes the checks (and gets as far as the
    workspace's, which is the last before the device)."""
    for b, h, n in itertools.permutations(range(3)):
        size = (3, 2, 64)
        order = sorted(zip((b, h, n), range(3)))
        st, at = [0, 0, 0], 64
        for _, ax in order:
            st[ax], at = at, at * size[ax]
        lay = struct.pack("18q", *[64 * 64 * 2, 64 * 64, 64] * 3, *[128, 64, 1] * 2, *st)
        assert rule(cla, B=3, lay=lay, ws=8) == TTT_ERR_WORKSPACE


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
def test_valid_calls_without_device_report_cuda_error(cla):
    assert rule(cla) == TTT_ERR_CUDA
    assert step(cla) == TTT_ERR_CUDA
    assert norm(cla) == TTT_ERR_CUDA


def test_binding_refuses_cpu_tensors_and_bad_shapes(cla):
    q = torch.zeros(1, 1, 8, 64, dtype=torch.bfloat16)
    g = torch.zeros(1, 1, 8)
    with pytest.raises(ValueError):
        cla.delta_rule_chunked_forward(q, q, q, g, g)
    with pytest.raises(ValueError):
        cla.delta_rule_chunked_forward(q, q[:, :, :4], q, g, g)
    with pytest.raises(ValueError):
        cla.delta_rule_chunked_forward(q, q.float(), q, g, g)
    with pytest.raises(ValueError):
        cla.delta_rule_chunked_forward(q, q, q, g, g.double())
    with pytest.raises(ValueError):
        cla.delta_rule_step(q[:, :, 0], q[:, :, 0], q[:, :, 0], g[:, :, 0], g[:, :, 0],
                            torch.zeros(1, 1, 64, 64))
    with pytest.raises(ValueError):
        cla.block_norm_forward(q[0, 0], w=torch.ones(64))
