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


def experts(E):
    """An expert linear of 300 pairs, whose lists one block makes with counters in
    shared memory: 128 bytes an expert."""
    g = torch.Generator(device="cuda").manual_seed(E)
    T, K, I, O = 300, 1, 32, 8
    x, xs = lib.quantize_mxfp4(torch.randn(T, I, generator=g, device="cuda"))
    w, ws = lib.quantize_mxfp4(torch.randn(E, O, I, generator=g, device="cuda"))
    sel = torch.randint(0, E, (T, K), generator=g, device="cuda", dtype=torch.int32)
    p = torch.rand(T, K, generator=g, device="cuda")
    ys = torch.randn(T, O, generator=g, device="cuda")
    out = torch.empty_like(ys)
    l = _native.load()
    need = l.mxfp4_expert_linear_quantized_workspace_size(T, E, I, O, K)
    work = torch.empty(need, dtype=torch.uint8, device="cuda")
    tensors = (x, xs, w, ws, sel, p, ys, out)

    def call(stream):
        return l.mxfp4_expert_linear_quantized(*(t.data_ptr() for t in tensors), T, E, I, O, K,
                                               _native.DTYPE_F32, _native.INDEX_I32,
                                               work.data_ptr(), need, stream)

    return call, [out]


def test_expert_linears_of_different_numbers_of_experts():
    run_threads([experts(E) for E in (768, 384, 704, 400)], 10000)
