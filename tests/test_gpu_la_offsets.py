"""The offsets of packed sequences: whatever the caller's tensor is and becomes, a call works on the values that it was
given. Every packed case here is compared with the same call on a plain CPU tensor, bit for bit."""
import itertools
import threading
import time

import pytest
import torch

import layer_reference as ref
from test_gpu_la import TOL, cuda, inputs, run_bwd, run_fwd

pytestmark = pytest.mark.gpu
LENS = [70, 1, 300, 0, 129]
OTHER = torch.tensor([0, 5, 6, 400, 400, 500])


def on_gpu(x, gr):
    return [cuda(x[n]) for n in ("q", "k", "v", "g", "h0")], cuda(gr["dout"]), cuda(gr["dhT"])


def both(gdn, d, cu, dout, dhT):
    return gdn.la_chunk_fwd(*d, cu) + gdn.la_chunk_bwd(*d, cu, dout, dhT)


@pytest.fixture
def case(gdn):
    x, gr = inputs(1, 0, 2, 4, 64, 128, seed=31, lens=LENS)
    d, dout, dhT = on_gpu(x, gr)
    want = both(gdn, d, x["cu"], dout, dhT)
    torch.cuda.synchronize()
    return x["cu"], d, dout, dhT, want


def same(got, want):
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_pinned_and_rewritten_after_the_call(gdn, case, dtype):
    cu, d, dout, dhT, want = case
    pinned = cu.to(dtype).pin_memory()
    torch.cuda._sleep(20_000_000)   # the stream is busy for some 10 ms while the host goes on
    got = both(gdn, d, pinned, dout, dhT)
    pinned.copy_(OTHER)
    same(got, want)


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_captured_and_rewritten_before_the_replay(gdn, case, dtype):
    cu, d, dout, dhT, want = case
    given = cu.to(dtype)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(gdn, d, given, dout, dhT)
    given.copy_(OTHER)
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        same(got, want)


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_on_the_device(gdn, case, dtype):
    cu, d, dout, dhT, want = case
    given = cu.cuda().to(dtype)
    got = both(gdn, d, given, dout, dhT)
    given.copy_(OTHER)
    same(got, want)
    strided = torch.stack([given, given], 1)
    strided[:, 0] = cu.cuda()
    same(both(gdn, d, strided[:, 0], dout, dhT), want)


def test_other_threads_run_while_a_call_waits(gdn, case):
    cu, d, dout, dhT, want = case
    given, ticks, stop = cu.cuda(), [0], threading.Event()

    def count():
        while not stop.is_set():
            ticks[0] += 1
            time.sleep(1e-3)
    torch.cuda.synchronize()
    t = threading.Thread(target=count)
    t.start()
    try:
        torch.cuda._sleep(200_000_000)   # some 100 ms, which the call has to wait for
        before = ticks[0]
        o, hT = gdn.la_chunk_fwd(*d, given)
        during = ticks[0] - before
    finally:
        stop.set()
        t.join()
    assert during >= 10
    same((o, hT), want)


def test_host_tensor_does_not_give_the_lock_away(gdn, case):
    """Beside a thread that never lets go of the interpreter by itself, a call that gave it away would wait for a switch
    (5 ms) each time: 200 calls a second at least. Without, the two threads take turns of 5 ms. (The results are kept:
    torch gives the lock away where a tensor is freed.)"""
    cu, d, *_ = case
    stop, kept = threading.Event(), []

    def busy():
        while not stop.is_set():
            pass
    t = threading.Thread(target=busy)
    t.start()
    try:
        began = time.perf_counter()
        for _ in range(200):
            kept.append(gdn.la_chunk_fwd(*d, cu))
        took = time.perf_counter() - began
    finally:
        stop.set()
        t.join()
    torch.cuda.synchronize()
    assert took < 0.5


def test_device_tensor_is_refused_in_a_capture(gdn, case):
    cu, d, dout, dhT, want = case
    given = cu.cuda()
    with pytest.raises(ValueError, match="captured"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            gdn.la_chunk_fwd(*d, given)
    same(both(gdn, d, cu, dout, dhT), want)


def test_values_that_do_not_fit(gdn, case):
    cu, d, *_ = case
    for bad, match in ((cu.long() + torch.tensor([0, 0, 0, 0, 0, 1 << 32]), "32 bits"), (cu.float(), "whole numbers"),
                       (cu.view(1, -1), "N . 1")):
        with pytest.raises(ValueError, match=match):
            gdn.la_chunk_fwd(*d, bad)


def test_more_sequences_than_a_launch_carries(gdn):
    lens = [n % 3 for n in range(2300)]
    x, gr = inputs(1, 0, 1, 1, 64, 64, seed=32, lens=lens)
    assert x["cu"].tolist() == [0, *itertools.accumulate(lens)]
    o, hT = run_fwd(gdn, x, 1.0)
    got = dict(o=o, hT=hT, **run_bwd(gdn, x, gr, 1.0))
    want = ref.la(*(x[n] for n in ("q", "k", "v", "g", "h0", "cu")), 1.0, gr["dout"], gr["dhT"])
    for n in want:
        assert ref.rel(got[n], want[n]) <= TOL[n], n
