"""The fixed-state mixers at their limits: waits that run out, pools and token
axes whose offsets pass 32 bits, more sequences than blocks."""
import pytest
import torch

from tests.gpu_util import assert_status_ok, f64, lib, rel_l2

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16 = torch.bfloat16
TTT_ERR_TIMEOUT = -7


@pytest.mark.parametrize("what", [1, 2])
@pytest.mark.parametrize("d", [64, 128])
def test_a_wait_that_runs_out_ends_the_call(what, d):
    """The test hook keeps a key tile, or weights, from the first block: its waits give
    up, the host reads TTT_ERR_TIMEOUT, the other blocks' outputs have their usual bits,
    nothing around the outputs is touched, and the next call has all of them."""
    cla = lib()
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(1, h, 900, d, generator=g).to(DEV, BF16) for h in (4, 2, 2))
    want = cla.window_attention_forward(q, k, v, 200, 4)
    torch.cuda.synchronize()
    assert_status_ok(cla)
    room = torch.full((1, 4, 902, d), 7.0, dtype=BF16, device=DEV)
    cla.set_wait_limit_ns(1_000_000)
    cla.selftest_withhold_window(what)
    try:
        cla.window_attention_forward(q, k, v, 200, 4, out=room[:, :, 1:-1])
        status = cla.device_status()
    finally:
        cla.selftest_withhold_window(0)
        cla.set_wait_limit_ns(200_000_000)
    assert status == TTT_ERR_TIMEOUT
    assert cla.device_status() == 0   # read and cleared
    assert (room[:, :, 0] == 7.0).all() and (room[:, :, -1] == 7.0).all()
    assert torch.equal(room[:, 1:, 1:-1], want[:, 1:])
    assert torch.equal(room[:, 0, 257:-1], want[:, 0, 256:])
    got = cla.window_attention_forward(q, k, v, 200, 4)
    torch.cuda.synchronize()
    assert_status_ok(cla)
    assert torch.equal(got, want)


def test_slots_far_into_large_pools():
    """The last slots of pools of more than 2^31 elements, against small pools."""
    cla = lib()
    g = torch.Generator().manual_seed(2)
    Hk, d, window, sinks = 8, 128, 2044, 4
    places = window + sinks
    q, k, v = (torch.randn(1, h, 300, d, generator=g).to(DEV, BF16) for h in (16, Hk, Hk))
    small = [torch.randn(1, Hk, places, d, generator=g).to(DEV, BF16) for _ in range(2)]
    slots = (1 << 31) // (Hk * places * d) + 2
    big = [torch.empty(slots, Hk, places, d, device=DEV, dtype=BF16) for _ in range(2)]
    for b, s in zip(big, small):
        b[-1] = s[0]
    past = torch.tensor([5000], dtype=torch.int32, device=DEV)
    last = torch.tensor([slots - 1], dtype=torch.int32, device=DEV)
    res = []
    for c, at in ((small, None), (big, last)):
        o = cla.window_attention_forward(q, k, v, window, sinks, cache_k=c[0], cache_v=c[1], past=past,
                                         slots=at)
        o1 = cla.window_attention_step(q[:, :, 0], k[:, :, 0], v[:, :, 0], *c, past + 300, window,
                                       sinks, at)
        res.append((o, o1))
    for a, b in zip(*res):
        assert torch.equal(a, b)
    for b, s in zip(big, small):
        assert torch.equal(b[-1], s[0])
    del big
    ch, S = 4096, 16
    n = (1 << 31) // (ch * S) + 2
    x, dt = (torch.randn(1, ch, generator=g).to(DEV, BF16) for _ in range(2))
    B = torch.randn(1, 1, S, generator=g).to(DEV, BF16)
    A = -torch.rand(ch, S, generator=g).to(DEV)
    one = torch.randn(1, ch, S, generator=g).to(DEV)
    pool = torch.empty(n, ch, S, device=DEV)
    pool[-1] = one[0]
    last = torch.tensor([n - 1], dtype=torch.int32, device=DEV)
    assert torch.equal(cla.selective_scan_step(x, dt, A, B, B, one),
                       cla.selective_scan_step(x, dt, A, B, B, pool, slots=last))
    assert torch.equal(pool[-1], one[0])
    del pool
    w = torch.randn(ch, 4, generator=g).to(DEV)
    n = (1 << 31) // (3 * ch) + 2
    one = torch.randn(1, 3, ch, generator=g).to(DEV, BF16)
    pool = torch.empty(n, 3, ch, device=DEV, dtype=BF16)
    pool[-1] = one[0]
    last = torch.tensor([n - 1], dtype=torch.int32, device=DEV)
    assert torch.equal(cla.short_conv_step(x, w, one), cla.short_conv_step(x, w, pool, slots=last))
    assert torch.equal(pool[-1], one[0])
    assert_status_ok(cla)


def test_token_axes_of_more_than_2_31_elements():
    """The end of a long text, against calls on its end alone."""
    cla = lib()
    N, D, tail = 1400000, 1536, 3000
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(1, N, D, generator=g, device=DEV, dtype=BF16)
    w = torch.randn(D, 4, generator=g, device=DEV)
    o, st = cla.short_conv_forward(x, w, silu=True)
    o2, st2 = cla.short_conv_forward(x[:, -tail:], w, silu=True, state=x[:, -tail - 3:-tail].contiguous())
    assert torch.equal(o[:, -tail:], o2) and torch.equal(st, st2)
    A = -4.0 * torch.ones(D, 16, device=DEV)   # forgets within a few dozen tokens
    B = torch.randn(1, N, 1, 16, generator=g, device=DEV, dtype=BF16)
    o, h = cla.selective_scan_forward(x, x, A, B, B, dt_bias=torch.ones(D, device=DEV), out=o)
    o2, h2 = cla.selective_scan_forward(x[:, -tail:], x[:, -tail:], A, B[:, -tail:], B[:, -tail:],
                                        dt_bias=torch.ones(D, device=DEV))
    # both within the roundings of a bf16 output, and fp32 sums over a forgotten past
    assert rel_l2(f64(o[:, -1000:]), f64(o2[:, -1000:])) <= 2 * 2.0 ** -8
    assert rel_l2(f64(h), f64(h2)) <= 1e-5
    q = x.view(1, N, 12, 128).transpose(1, 2)
    o = cla.window_attention_forward(q, q[:, :4], q[:, 4:8], 64, out=o.view(1, N, 12, 128).transpose(1, 2))
    o2 = cla.window_attention_forward(q[:, :, -tail:], q[:, :4, -tail:], q[:, 4:8, -tail:], 64)
    assert rel_l2(f64(o[:, :, -1000:]), f64(o2[:, :, -1000:])) <= 2 * 2.0 ** -8
    torch.cuda.synchronize()
    assert_status_ok(cla)


def test_many_sequences_of_one_token():
    """Twenty thousand sequences of one token: each only sees itself."""
    cla = lib()
    n = 20000
    g = torch.Generator(device=DEV).manual_seed(4)
    q, k, v = (torch.randn(1, n, 1, 64, generator=g, device=DEV, dtype=BF16).transpose(1, 2)
               for _ in range(3))
    starts = torch.arange(n + 1, dtype=torch.int32, device=DEV)
    assert torch.equal(cla.window_attention_forward(q, k, v, 100, 2, seq_starts=starts), v)
    x = torch.randn(1, n, 64, generator=g, device=DEV, dtype=BF16)
    w = torch.randn(64, 4, generator=g, device=DEV)
    o, st = cla.short_conv_forward(x, w, seq_starts=starts)
    want = (x.float() * w[:, 3]).to(BF16)
    assert torch.equal(o, want)
    assert torch.equal(st[:, 2], x[0]) and (st[:, :2] == 0).all()
    A = -torch.rand(64, 8, generator=g, device=DEV)
    B = torch.randn(1, n, 1, 8, generator=g, device=DEV, dtype=BF16)
    _, h = cla.selective_scan_forward(x, x, A, B, B, dt_softplus=False, seq_starts=starts)
    want = (x.float() * x.float())[0, :, :, None] * B.float()[0]
    assert rel_l2(f64(h), f64(want)) <= 4 * 2.0 ** -24
    torch.cuda.synchronize()
    assert_status_ok(cla)
