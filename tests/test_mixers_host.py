"""Host-side checks of the fixed-state mixers' entry points (no GPU): bad
arguments are refused with the documented codes before the device is touched."""
import struct

import pytest
import torch

from tests.test_capi_host import (TTT_ERR_ALIGN, TTT_ERR_ARG, TTT_ERR_CUDA, TTT_ERR_NULL,
                                  TTT_ERR_SHAPE, TTT_ERR_UNSUPPORTED, TTT_ERR_WORKSPACE, cla,
                                  fake)

__all__ = ["cla"]


def pointers(n, off=(), nulls=(), same=()):
    p = [fake(0x100000 * (i + 1) + (2 if i in off else 0)) for i in range(n)]
    for i, j in same:
        p[i] = p[j]
    for i in nulls:
        p[i] = None
    return p


def window(cla, B=2, Hq=4, Hk=2, N=64, d=64, window=16, sinks=2, n_slots=4, n_seq=None, io=1,
           scale=0.125, packed=False, cache=True, slots=True, past=True, lay=None, **kw):
    q, k, v, ck, cv, sl, pa, st, out = pointers(9, **kw)
    return cla.library().window_attention_forward(
        q, k, v, ck if cache else None, cv if cache else None, sl if slots else None, n_slots,
        pa if past else None, st if packed else None, B if n_seq is None else n_seq, B, Hq, Hk, N, d,
        window, sinks, io, scale, lay, out, None)


def test_window_refusals(cla):
    for i in (0, 1, 2, 3, 4, 8):
        assert window(cla, nulls=(i,)) == TTT_ERR_NULL, i
    assert window(cla, cache=False) == TTT_ERR_NULL          # slots and past need the caches
    assert window(cla, cache=False, slots=False) == TTT_ERR_NULL
    for bad in (dict(B=0), dict(N=0), dict(Hq=0), dict(Hk=0), dict(d=0), dict(Hq=3), dict(window=0),
                dict(sinks=-1), dict(n_seq=3), dict(packed=True), dict(n_slots=0),
                dict(slots=False, n_slots=1), dict(B=1, n_seq=0, packed=True)):
        assert window(cla, **bad) == TTT_ERR_SHAPE, bad
    assert window(cla, io=2) == TTT_ERR_ARG
    assert window(cla, scale=float("inf")) == TTT_ERR_ARG
    for bad in (dict(d=257), dict(window=(1 << 30) + 1), dict(sinks=(1 << 30) + 1),
                dict(B=40000), dict(B=1, n_seq=20000, packed=True, n_slots=20000),
                dict(N=(1 << 30) + 1), dict(N=1 << 30)):
        assert window(cla, **bad) == TTT_ERR_UNSUPPORTED, bad
    for i in (3, 4, 5, 6):
        assert window(cla, off=(i,)) == TTT_ERR_ALIGN, i
    assert window(cla, io=0, off=(0,)) == TTT_ERR_ALIGN
    for pair in ((8, 0), (8, 1), (8, 2), (8, 3), (8, 4), (3, 4), (3, 1), (4, 2)):
        assert window(cla, same=(pair,)) == TTT_ERR_ARG, pair
    lay = [4 * 64 * 64, 64 * 64, 64] + [2 * 64 * 64, 64 * 64, 64] * 2 + [4 * 64 * 64, 64 * 64, 64]
    for at, x in ((0, -1), (5, -64), (11, 0), (11, 63), (10, 63 * 64), (9, 64)):
        bad = list(lay)
        bad[at] = x
        assert window(cla, lay=struct.pack("12q", *bad)) == TTT_ERR_ARG, (at, x)
    if not torch.cuda.is_available():
        assert window(cla, lay=struct.pack("12q", *lay)) == TTT_ERR_CUDA


def window_step(cla, B=2, Hq=4, Hk=2, d=64, window=16, sinks=2, n_slots=4, io=1, scale=0.125,
                slots=True, lay=None, **kw):
    q, k, v, ck, cv, pos, sl, out = pointers(8, **kw)
    return cla.library().window_attention_step(q, k, v, ck, cv, pos, sl if slots else None, n_slots, B,
                                               Hq, Hk, d, window, sinks, io, scale, lay, out, None)


def test_window_step_refusals(cla):
    for i in (0, 1, 2, 3, 4, 5, 7):
        assert window_step(cla, nulls=(i,)) == TTT_ERR_NULL, i
    for bad in (dict(B=0), dict(Hq=3), dict(window=0), dict(sinks=-1), dict(n_slots=0),
                dict(slots=False, n_slots=1)):
        assert window_step(cla, **bad) == TTT_ERR_SHAPE, bad
    for bad in (dict(d=257), dict(B=65536, n_slots=65536), dict(Hq=1 << 20, Hk=1)):
        assert window_step(cla, **bad) == TTT_ERR_UNSUPPORTED, bad
    assert window_step(cla, scale=float("nan")) == TTT_ERR_ARG
    for i in (3, 4, 5, 6):
        assert window_step(cla, off=(i,)) == TTT_ERR_ALIGN, i
    for pair in ((7, 0), (7, 3), (7, 4), (3, 4)):
        assert window_step(cla, same=(pair,)) == TTT_ERR_ARG, pair


def scan(cla, B=1, N=64, D=32, S=16, G=2, n_seq=None, io=1, softplus=1, packed=False, ws=None,
         lay=None, **kw):
    x, dt, A, Bm, Cm, Dx, bias, z, s_in, st, out, s_out, wsp = pointers(13, **kw)
    n_seq = B if n_seq is None else n_seq
    lib = cla.library()
    need = lib.selective_scan_workspace_size(B, N, D, S, G, n_seq, io)
    return lib.selective_scan_forward(x, dt, A, Bm, Cm, Dx, bias, z, s_in, st if packed else None,
                                      n_seq, B, N, D, S, G, io, softplus, lay, out, s_out, wsp,
                                      max(need, 256) if ws is None else ws, None)


def test_scan_refusals(cla):
    for i in (0, 1, 2, 3, 4, 10):
        assert scan(cla, nulls=(i,)) == TTT_ERR_NULL, i
    for bad in (dict(B=0), dict(N=0), dict(D=0), dict(S=0), dict(G=0), dict(G=3), dict(n_seq=2),
                dict(B=2, packed=True), dict(B=2, n_seq=3)):
        assert scan(cla, **bad) == TTT_ERR_SHAPE, bad
    assert scan(cla, io=2) == TTT_ERR_ARG
    assert scan(cla, softplus=2) == TTT_ERR_ARG
    for bad in (dict(S=129), dict(D=32770), dict(B=65536), dict(N=1 << 30, B=2),
                dict(n_seq=(1 << 20) + 1, packed=True)):
        assert scan(cla, **bad) == TTT_ERR_UNSUPPORTED, bad
    for i in (2, 5, 6, 8, 11, 12):
        assert scan(cla, off=(i,)) == TTT_ERR_ALIGN, i
    assert scan(cla, ws=8) == TTT_ERR_WORKSPACE
    assert scan(cla, nulls=(12,)) == TTT_ERR_WORKSPACE
    for pair in ((10, 0), (10, 1), (10, 7), (10, 3), (11, 8), (11, 10)):
        assert scan(cla, same=(pair,)) == TTT_ERR_ARG, pair
    lay = [64 * 32, 32] * 3 + [64 * 32, 32] * 2 + [64 * 32, 32]
    for at, x in ((0, -1), (7, -32), (11, 31), (11, 0)):
        bad = list(lay)
        bad[at] = x
        assert scan(cla, lay=struct.pack("12q", *bad)) == TTT_ERR_ARG, (at, x)


def test_scan_workspace_size(cla):
    lib = cla.library()
    assert lib.selective_scan_workspace_size(2, 32768, 1536, 16, 1, 2, 1) >= 256
    assert lib.selective_scan_workspace_size(1, 1, 1, 1, 1, 1, 0) >= 256
    assert lib.selective_scan_workspace_size(2, 64, 32, 16, 3, 2, 1) == 0


def scan_step(cla, B=2, D=32, S=16, G=1, n_slots=4, io=1, softplus=1, slots=True, **kw):
    x, dt, A, Bm, Cm, Dx, bias, z, st, sl, out = pointers(11, **kw)
    return cla.library().selective_scan_step(x, dt, A, Bm, Cm, Dx, bias, z, st,
                                             sl if slots else None, n_slots, B, D, S, G, io, softplus,
                                             None, out, None)


def test_scan_step_refusals(cla):
    for i in (0, 1, 2, 3, 4, 8, 10):
        assert scan_step(cla, nulls=(i,)) == TTT_ERR_NULL, i
    for bad in (dict(B=0), dict(S=0), dict(G=3), dict(n_slots=0), dict(slots=False, n_slots=1)):
        assert scan_step(cla, **bad) == TTT_ERR_SHAPE, bad
    assert scan_step(cla, S=129) == TTT_ERR_UNSUPPORTED
    assert scan_step(cla, softplus=3) == TTT_ERR_ARG
    assert scan_step(cla, off=(8,)) == TTT_ERR_ALIGN
    assert scan_step(cla, same=((10, 8),)) == TTT_ERR_ARG


def conv(cla, B=1, N=64, D=32, W=4, n_seq=None, io=1, silu=1, packed=False, lay=None, **kw):
    x, w, bias, s_in, st, out, s_out = pointers(7, **kw)
    return cla.library().short_conv_forward(x, w, bias, s_in, st if packed else None,
                                            B if n_seq is None else n_seq, B, N, D, W, io, silu, lay,
                                            out, s_out, None)


def test_conv_refusals(cla):
    for i in (0, 1, 5):
        assert conv(cla, nulls=(i,)) == TTT_ERR_NULL, i
    for bad in (dict(B=0), dict(N=0), dict(D=0), dict(W=1), dict(n_seq=2), dict(B=2, packed=True)):
        assert conv(cla, **bad) == TTT_ERR_SHAPE, bad
    for bad in (dict(W=9), dict(D=32769), dict(B=65536)):
        assert conv(cla, **bad) == TTT_ERR_UNSUPPORTED, bad
    assert conv(cla, silu=2) == TTT_ERR_ARG
    assert conv(cla, io=3) == TTT_ERR_ARG
    for i in (1, 2):
        assert conv(cla, off=(i,)) == TTT_ERR_ALIGN, i
    for pair in ((5, 0), (5, 3), (6, 3), (6, 5), (6, 0)):
        assert conv(cla, same=(pair,)) == TTT_ERR_ARG, pair
    assert conv(cla, lay=struct.pack("4q", 64 * 32, 32, 64 * 32, 31)) == TTT_ERR_ARG
    assert conv(cla, lay=struct.pack("4q", 64 * 32, -32, 64 * 32, 32)) == TTT_ERR_ARG


def conv_step(cla, B=2, D=32, W=4, n_slots=4, io=1, silu=1, slots=True, **kw):
    x, w, bias, st, sl, out = pointers(6, **kw)
    return cla.library().short_conv_step(x, w, bias, st, sl if slots else None, n_slots, B, D, W, io,
                                         silu, None, out, None)


def test_conv_step_refusals(cla):
    for i in (0, 1, 3, 5):
        assert conv_step(cla, nulls=(i,)) == TTT_ERR_NULL, i
    for bad in (dict(B=0), dict(W=1), dict(n_slots=0), dict(slots=False, n_slots=1)):
        assert conv_step(cla, **bad) == TTT_ERR_SHAPE, bad
    assert conv_step(cla, W=9) == TTT_ERR_UNSUPPORTED
    for pair in ((5, 0), (5, 3), (3, 0)):
        assert conv_step(cla, same=(pair,)) == TTT_ERR_ARG, pair


def test_bindings_refuse_tensors_of_the_host(cla):
    x = torch.zeros(1, 8, 64)
    w, A, B = torch.zeros(64, 4), torch.zeros(64, 16), torch.zeros(1, 8, 1, 16)
    q, c, i = torch.zeros(1, 2, 8, 64), torch.zeros(1, 2, 8, 64), torch.zeros(1, dtype=torch.int32)
    for call in (lambda: cla.window_attention_forward(q, q, q, 8),
                 lambda: cla.window_attention_step(q[:, :, 0], q[:, :, 0], q[:, :, 0], c, c, i, 8),
                 lambda: cla.selective_scan_forward(x, x, A, B, B),
                 lambda: cla.selective_scan_step(x[0], x[0], A, B[0], B[0], torch.zeros(8, 64, 16)),
                 lambda: cla.short_conv_forward(x, w),
                 lambda: cla.short_conv_step(x[0], w, torch.zeros(8, 3, 64))):
        with pytest.raises(ValueError, match="CUDA device"):
            call()


def test_sizes_past_32_bit_arithmetic(cla):
    """A cache of more than 2^30 places, and a token axis of more than 2^30."""
    half = 1 << 29
    for step in (window, window_step):
        assert step(cla, window=half + 1, sinks=half) == TTT_ERR_UNSUPPORTED
        assert step(cla, window=1 << 30, sinks=1) == TTT_ERR_UNSUPPORTED
        assert step(cla, window=1 << 30, sinks=1 << 30) == TTT_ERR_UNSUPPORTED
        if not torch.cuda.is_available():
            assert step(cla, window=half, sinks=half) == TTT_ERR_CUDA
    no_cache = dict(window=1 << 30, sinks=1 << 30, cache=False, slots=False, past=False)
    if not torch.cuda.is_available():
        assert window(cla, **no_cache) == TTT_ERR_CUDA
    for call in (scan, conv):
        assert call(cla, N=(1 << 30) + 1, B=1) == TTT_ERR_UNSUPPORTED
