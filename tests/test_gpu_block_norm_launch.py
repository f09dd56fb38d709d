"""Launches of the block norm's form for long unaligned rows, whose shared
memory grows with the row: calls of different lengths must not disturb one
another, neither from two host threads nor in one captured graph.

Tolerances are those of the neighbouring tests of the norms.
"""
import threading

import pytest
import torch

from tests.gpu_util import lib
from tests.test_gpu_block_norm import BF, DEV, F32, check, make, on, want

pytestmark = pytest.mark.gpu

LONG = [(2, 16383, 3), (3, 7001, 7001), (2, 9001, 9001)]   # rows, D, group


def cases():
    return [(make(80 + i, rows, D, group, BF, F32, 1, True, True, True), group)
            for i, (rows, D, group) in enumerate(LONG)]


def test_two_lengths_in_one_captured_graph():
    cla = lib()
    sets = cases()
    dev = [on(t) for t, _ in sets]
    for d in dev:   # a call of each length before
        cla.block_norm_forward(**d, out_dtype=F32)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [cla.block_norm_forward(**d, out_dtype=F32) for d in dev]
    graph.replay()
    torch.cuda.synchronize()
    for g, (t, group) in zip(got, sets):
        check(g, want(t, group), BF, F32)


def test_two_host_threads_with_rows_of_different_length():
    """Threads that call the C entry itself, whose argument checks and launch run
    without the interpreter's lock."""
    cla = lib()
    entry = cla.library().block_norm_forward
    sets = cases()
    dev = [on(t) for t, _ in sets]
    first = [cla.block_norm_forward(**d, out_dtype=F32) for d in dev]
    for g, (t, group) in zip(first, sets):
        check(g, want(t, group), BF, F32)
    torch.cuda.synchronize()
    args, outs, streams = [], [], [torch.cuda.Stream() for _ in dev]
    for d, f, (t, group), st in zip(dev, first, sets, streams):
        out, h = torch.empty_like(f[0]), torch.empty_like(f[1])
        rows, D = d["y"].shape
        outs.append((out, h))
        args.append((d["y"].data_ptr(), d["w"].data_ptr(), d["gate"].data_ptr(),
                     d["residual"].data_ptr(), d["scale"].data_ptr(), d["w_next"].data_ptr(), rows,
                     D, group, cla.TTT_BF16, cla.TTT_F32, cla.GATE_SILU, 1e-6, None,
                     out.data_ptr(), h.data_ptr(), st.cuda_stream))
    codes = [set() for _ in args]

    def work(i):
        torch.cuda.set_device(0)
        for n in range(10000):
            codes[i].add(entry(*args[i]))
            if n % 500 == 499:
                streams[i].synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(args))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == [{0}] * len(args)
    for a, b in zip(outs, first):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
