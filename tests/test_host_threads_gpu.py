"""C calls of several host threads at once, each on a stream of its own: none may
fail, and results have to be those of a call alone."""
import threading

import pytest
import torch

import mxfp4_routed_expert_route_gb300 as lib
from mxfp4_routed_expert_route_gb300 import _native

pytestmark = pytest.mark.gpu


def run_threads(calls, rounds):
    """calls: (function of a stream's handle that returns a status, its outputs)."""
    want = []
    for f, outs in calls:
        assert f(torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
        for t in outs:
            t.zero_()
    torch.cuda.synchronize()
    start, failed = threading.Barrier(len(calls)), [0] * len(calls)

    def work(i, f):
        stream = torch.cuda.Stream()
        start.wait(60)
        for _ in range(rounds):
            failed[i] += f(stream.cuda_stream) != 0
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(i, f)) for i, (f, _) in enumerate(calls)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert failed == [0] * len(calls)
    for (_, outs), first in zip(calls, want):
        assert all(torch.equal(a, b) for a, b in zip(outs, first))


def router(E):
    g = torch.Generator(device="cuda").manual_seed(E)
    x = torch.randn(1, E, generator=g, device="cuda")
    sel = torch.empty(1, 4, dtype=torch.int32, device="cuda")
    p = torch.empty(1, 4, device="cuda")
    f = _native.load().mxfp4_route_experts

    def call(stream, x=x):                         # keeps the logits
        return f(x.data_ptr(), _native.DTYPE_F32, E, None, 1, E, 4, _native.SCORE_SOFTMAX, 1, 1,
                 2, 1, 1.0, sel.data_ptr(), p.data_ptr(), stream)

    return call, [sel, p]


def test_routers_of_different_widths():
    """More than 768 experts take shared memory that the kernel has to be allowed
    first; a narrower call may not take it back from a wider one."""
    run_threads([router(E) for E in (1024, 776, 1024, 800)], 30000)
