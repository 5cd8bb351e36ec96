"""The layer operators in a program of several Python threads (needs a B200)."""
import threading
import time

import pytest
import torch

import kda_chunked_recurrent_b200 as K

pytestmark = pytest.mark.gpu


def test_other_threads_run_while_a_launch_waits():
    """A stream that is busy for about half a second takes some thousand launches, and the next one
    waits on the host until there is room.  A second thread has to run meanwhile."""
    x = torch.randn(4, 64, device="cuda")
    out = torch.empty_like(x)
    K.rms_norm(x, out=out)
    torch.cuda.synchronize()
    ticks, stop = [], threading.Event()

    def tick():
        while not stop.is_set():
            ticks.append(time.perf_counter())
            time.sleep(0.002)

    other = threading.Thread(target=tick)
    other.start()
    try:
        torch.cuda._sleep(1_000_000_000)
        longest, waited = 0.0, None
        for _ in range(4000):
            a = time.perf_counter()
            K.rms_norm(x, out=out)
            b = time.perf_counter()
            if b - a > longest:
                longest, waited = b - a, (a, b)
    finally:
        stop.set()
        other.join()
    torch.cuda.synchronize()
    if longest < 0.1:
        pytest.skip("the queue took all launches")
    inside = sum(waited[0] < t < waited[1] for t in ticks)
    assert inside > longest / 0.002 / 10, f"{inside} ticks of 2 ms in {longest:.3f} s"


def test_calls_from_several_threads():
    """Each thread with its stream and pool: the results of one after the other."""
    g = torch.Generator().manual_seed(1)
    rows = [torch.randn(40, 96, generator=g).cuda() for _ in range(4)]
    w = torch.randn(96, 4, generator=g).cuda()
    A_log, BC = torch.zeros(96, 16, device="cuda"), torch.randn(40, 2, 1, 16, generator=g).cuda()

    def work(x, into):
        cpool, spool = torch.zeros(1, 3, 96, device="cuda"), torch.zeros(1, 96, 16, device="cuda")
        for t in range(40):
            u = x[None, t:t + 1]
            y = K.conv_decode(K.rms_norm(u[0])[0][None], w, cpool)[0]
            into.append(K.scan_decode(y, u, A_log, BC[None, t:t + 1, 0], BC[None, t:t + 1, 1],
                                      spool)[0])
        into += [cpool, spool]

    want = [[] for _ in rows]
    for x, into in zip(rows, want):
        work(x, into)
    torch.cuda.synchronize()
    got = [[] for _ in rows]

    def run(x, into):
        with torch.cuda.stream(torch.cuda.Stream()):
            work(x, into)
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=run, args=a) for a in zip(rows, got)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(got, want):
        assert len(a) == len(b) and all(torch.equal(u, v) for u, v in zip(a, b))
