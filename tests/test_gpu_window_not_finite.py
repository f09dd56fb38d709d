"""Window attention's prompts over values that are not finite, where the rows that meet them
are made again: no wait of the others runs out meanwhile, and what a row does not see does not
reach it."""
import numpy as np
import pytest
import torch

from tests import test_gpu_mixers as M
from tests.gpu_util import assert_status_ok, lib

pytestmark = pytest.mark.gpu

DEV, BF16 = M.DEV, M.BF16
NAN, INF = float("nan"), float("inf")


def in_64_bits(q, k, v, window, sinks):
    """[Hq, N, d] outputs and sums of weighted absolute values, on the GPU."""
    Hq, N, d = q.shape
    i = torch.arange(N, device=q.device)
    see = (i[None] <= i[:, None]) & ((i[None] < sinks) | (i[:, None] - i[None] < window))
    out, size = [], []
    for h in range(Hq):
        g = h * k.shape[0] // Hq
        s = (q[h].double() @ k[g].double().T) * d ** -0.5
        w = torch.softmax(s.masked_fill(~see, -INF), -1)
        out.append(w @ v[g].double())
        size.append(w @ v[g].double().abs())
    return torch.stack(out), torch.stack(size)


def close(got, ref, size, weights=2.0 ** -8):
    """Weights in bf16, the output's rounding, and 2^-9 for what fp32 loses: scores of d <= 128
    products are off by (d + 6) 2^-24 of their absolute sum (134 x 2^-24 x 0.09 x 200 = 1.5e-4 at
    most), four times that for a weight, and 3 n 2^-24 = 7.4e-4 for sums over n <= 4100 keys."""
    bound = (weights + 2.0 ** -9) * size
    assert ((got.double() - ref).abs() <= bound + 2.0 ** -8 * (ref.abs() + bound)).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("what", [INF, NAN])
def test_a_value_that_all_rows_see_ends_no_wait(what, d):
    """One number of a sink's value under a window of 4096 tokens is not finite: it has its
    column, and waits of 1 ms do not run out while thousands of rows are made again, in blocks
    that have several tiles of queries one after the other."""
    cla = lib()
    g = torch.Generator(device=DEV).manual_seed(1)
    N, window, sinks = 6000, 4096, 4
    q, k, v = (torch.randn(1, h, N, d, generator=g, device=DEV).to(BF16) for h in (16, 2, 2))
    clean = cla.window_attention_forward(q, k, v, window, sinks)
    ref, size = in_64_bits(q[0], k[0], v[0], window, sinks)
    close(clean[0], ref, size)
    bad = v.clone()
    bad[0, 1, 1, 5] = what
    cla.set_wait_limit_ns(1_000_000)
    try:
        got = cla.window_attention_forward(q, k, bad, window, sinks)
        torch.cuda.synchronize()
        assert_status_ok(cla)
    finally:
        cla.set_wait_limit_ns(200_000_000)
    assert torch.equal(got[:, :8], clean[:, :8])
    assert torch.equal(got[:, 8:, 0], clean[:, 8:, 0])      # sees the first token alone
    column = got[:, 8:, 1:, 5]
    assert torch.isnan(column).all() if what != what else (column == INF).all()
    rest = [c for c in range(d) if c != 5]
    close(got[0, 8:, :, rest], ref[8:, :, rest], size[8:, :, rest])
    assert torch.equal(got, cla.window_attention_forward(q, k, bad, window, sinks)) or what != what


@pytest.mark.parametrize("d", [64, 72, 128])
def test_places_and_tokens_of_none_that_hold_nan(d):
    """A long packed batch between tokens of no sequence, on caches as they were allocated:
    every row that shares a key tile with them is made again, next to rows that are not."""
    cla = lib()
    window, sinks = 300, 3
    places = window + sinks
    pasts = [0, 1, 40, places - 1, places, 5 * places + 7]
    lengths = [400, 130, 257, 300, 90, 260]
    starts = [9] + (9 + np.cumsum(lengths)).tolist()
    N = starts[-1] + 50
    t = M.qkv(2, 1, 4, 2, N, d, BF16)
    for x in t:
        x[:, :, :9] = NAN
        x[:, :, starts[-1]:] = NAN
    r = M.gen(3)
    caches = [r(len(pasts), 2, places, d).to(BF16) for _ in range(2)]
    for x in caches:
        for s, past in enumerate(pasts):
            x[s, :, min(past, places):] = NAN
    dev, oracle = [x.to(DEV) for x in caches], [M.f64(x) for x in caches]
    cla.set_wait_limit_ns(1_000_000)
    try:
        out = torch.full((1, 4, N, d), 7.0, dtype=BF16, device=DEV)
        cla.window_attention_forward(*[x.to(DEV) for x in t], window, sinks, cache_k=dev[0],
                                     cache_v=dev[1], past=M.ints(pasts), seq_starts=M.ints(starts),
                                     out=out)
        torch.cuda.synchronize()
        assert_status_ok(cla)
    finally:
        cla.set_wait_limit_ns(200_000_000)
    ref, bound = M.MO.window_attention(*[M.f64(x) for x in t], window, sinks, None, oracle, None, pasts,
                                       starts, M.rounding(BF16, d))
    M.within(out, ref, bound, BF16)
    assert (out[:, :, :9] == 7.0).all() and (out[:, :, starts[-1]:] == 7.0).all()
    for x, y in zip(dev, oracle):
        assert np.array_equal(M.f64(x), y, equal_nan=True)


def test_scores_that_are_not_finite():
    """Queries and keys with NaN and infinities: what such a query, or a query that sees such a
    key, gets is NaN; a key whose score is minus infinity counts nothing."""
    cla = lib()
    N, d, window = 700, 64, 100
    q, k, v = (x.to(DEV) for x in M.qkv(4, 1, 2, 1, N, d, BF16))
    clean = cla.window_attention_forward(q, k, v, window)
    q2, k2 = q.clone(), k.clone()
    q2[:, :, 50] = NAN
    q2[:, 0, 300, 7] = INF
    k2[:, :, 400] = NAN
    k2[:, :, 550] = 0.0
    k2[:, :, 550, 3] = -INF
    q2[:, :, 500:700, 3] = q2[:, :, 500:700, 3].abs() + 1
    ref, size = in_64_bits(q2[0], k2[0], v[0], window, 0)
    got = cla.window_attention_forward(q2, k2, v, window)
    torch.cuda.synchronize()
    assert_status_ok(cla)
    assert torch.equal(torch.isnan(got[0]), torch.isnan(ref))
    gone = torch.isnan(ref).all(-1)
    assert gone[:, 50].all() and gone[0, 300] and not gone[1, 300] and gone[:, 400:500].all()
    assert int(gone.sum()) == 2 * 101 + 1
    held = ~gone
    close(got[0][held], ref[held], size[held])
    same = held.clone()
    same[:, 500:] = False
    assert torch.equal(got[0][same], clean[0][same])


def test_a_replayed_call_without_them():
    """A captured call over NaN, replayed over finite inputs and back."""
    cla = lib()
    g = torch.Generator(device=DEV).manual_seed(5)
    q, k, v = (torch.randn(1, h, 1500, 128, generator=g, device=DEV).to(BF16) for h in (8, 2, 2))
    bad = v.clone()
    bad[:, 0, 700:710] = NAN
    want = [cla.window_attention_forward(q, k, x, 200, 2) for x in (bad, v)]
    held = bad.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = cla.window_attention_forward(q, k, held, 200, 2)
    for x, y in ((bad, want[0]), (v, want[1]), (bad, want[0])):
        held.copy_(x)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(torch.isnan(out), torch.isnan(y))
        assert torch.equal(out.nan_to_num(), y.nan_to_num())
    assert_status_ok(cla)


def test_calls_repeat_themselves():
    """The same call gives the same bits."""
    cla = lib()
    g = torch.Generator(device=DEV).manual_seed(6)
    q, k, v = (torch.randn(1, 8000, h, 128, generator=g, device=DEV).to(BF16).transpose(1, 2)
               for h in (12, 4, 4))
    starts = M.ints([0, 3000, 3001, 7990])
    past = M.ints([5000, 12, 300])
    cache = [torch.randn(3, 4, 1004, 128, generator=g, device=DEV).to(BF16) for _ in range(2)]
    first = None
    for _ in range(20):
        c = [x.clone() for x in cache]
        o = cla.window_attention_forward(q, k, v, 1000, 4, cache_k=c[0], cache_v=c[1], past=past,
                                         seq_starts=starts)[:, :, :7990].clone()
        first = o if first is None else first
        assert torch.equal(o, first)
    torch.cuda.synchronize()
    assert_status_ok(cla)
