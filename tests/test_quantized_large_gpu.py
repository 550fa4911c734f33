"""Operators on quantised tokens where offsets pass 32 bits, and a first call that is
captured."""
import math
import os
import subprocess
import sys

import pytest
import torch

import mxfp4_routed_expert_route_gb300 as lib
import quantized_ref as ref
from test_quantized_products_gpu import check, rows

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def some(n, *more):
    g = torch.Generator().manual_seed(n % 1000)
    return torch.cat([torch.randint(0, n, (60,), generator=g), torch.tensor([0, n - 1, *more])]).cuda()


def test_linear_results_past_32_bits():
    T, I, O = 70001, 64, 32769
    x, w = rows(T, I, seed=1), rows(O, I, seed=2)
    got = lib.mxfp4_linear(*x, *w, dtype=BF16)
    t = some(T, (1 << 31) // O, (1 << 31) // O + 1, (1 << 32) // (2 * O))
    vx, vw = ref.values(x[0][t], x[1][t]), ref.values(*w)
    check(got[t], vx @ vw.T, ref.product_bound(vx, vw, I, BF16), BF16)
    assert lib.wait_timeouts() == 0


def test_experts_weights_and_partial_results_past_32_bits():
    """4.3 GB of codes; 2.3e9 float32 results before they are combined."""
    T, K, E, I, O = 40000, 2, 300, 1024, 28800
    g = torch.Generator(device="cuda").manual_seed(3)
    x, w = rows(T, I, seed=4), rows(E, O, I, seed=5)
    assert w[0].numel() > 1 << 32 and T * K * O > 1 << 31
    sel = torch.randint(0, E, (T, K), generator=g, device="cuda")
    p = torch.rand(T, K, generator=g, device="cuda")
    ys = torch.randn(T, O, generator=g, device="cuda").to(BF16)
    got = lib.mxfp4_expert_linear_quantized(*x, *w, sel, p, ys)
    for t in some(T, (1 << 31) // (K * O), (1 << 32) // (4 * K * O))[::4].tolist():
        vx = ref.values(x[0][t:t + 1], x[1][t:t + 1])
        want, terms = ys[t:t + 1].double(), ys[t:t + 1].double().abs()
        bound = torch.zeros_like(want)
        for k in range(K):
            e, q = int(sel[t, k]), p[t, k].double()
            vw = ref.values(w[0][e], w[1][e])
            want, terms = want + q * (vx @ vw.T), terms + q * (vx @ vw.T).abs()
            bound += q * ref.product_bound(vx, vw, I, BF16, more=4)
        check(got[t:t + 1], want, bound + (K + 1) * 2.0 ** -24 * terms, BF16)
    assert lib.wait_timeouts() == 0 and lib.device_errors() == 0


def test_quantize_past_32_bits():
    n, I = 36000, 120000                              # 4.3e9 values
    x = torch.randn(1, I, device="cuda").to(BF16).repeat(n, 1)
    scale = torch.exp2(torch.arange(n, device="cuda") % 60 - 30.0)[:, None]
    x *= scale.to(BF16)
    packed, scales = lib.quantize_mxfp4(x)
    back = lib.dequantize_mxfp4(packed, scales)
    for r in some(n, (1 << 31) // I, (1 << 32) // I)[::5].tolist():
        want_p, want_s = ref.quantize(x[r:r + 1])
        assert torch.equal(packed[r:r + 1].cpu(), want_p) and torch.equal(scales[r:r + 1].cpu(), want_s)
        assert torch.equal(back[r].cpu().double(), ref.values(want_p, want_s)[0])


def test_route_past_32_bits_and_a_bias_that_is_nan():
    wide = torch.empty(70000, 33000, device="cuda", dtype=BF16)    # rows 66 KB apart
    logits = wide[:, 7:71]
    logits.copy_(torch.randn(70000, 64, device="cuda"))
    bias = torch.randn(64, device="cuda") * 0.1
    bias[[3, 40]] = math.nan
    for b in (None, bias):
        sel, p = lib.route_experts(logits, 6, score="sigmoid", bias=b)
        t = some(70000, (1 << 31) // 33000, (1 << 31) // 33000 + 1)
        want_sel, want_p = ref.route(logits[t].cpu(), 6, "sigmoid", None if b is None else b.cpu())
        assert torch.equal(sel[t].cpu(), want_sel)
        torch.testing.assert_close(p[t].double().cpu(), want_p, rtol=ref.WEIGHT_RTOL, atol=0)


FIRST = """
import torch
import mxfp4_routed_expert_route_gb300 as lib
x = torch.randn({T}, 320, device="cuda").to(torch.bfloat16)
w = torch.randint(0, 256, (8, 96, 10, 16), device="cuda", dtype=torch.uint8)
ws = torch.randint(118, 124, (8, 96, 10), device="cuda", dtype=torch.uint8)
logits, ys = torch.randn({T}, 8, device="cuda"), torch.randn({T}, 96, device="cuda")
torch.cuda.synchronize()
def layer():
    sel, p = lib.route_experts(logits, 2)
    q = lib.quantize_mxfp4(x)
    return (sel, p, *q, lib.dequantize_mxfp4(*q), lib.mxfp4_linear(*q, w[0], ws[0]),
            lib.mxfp4_expert_linear_quantized(*q, w, ws, sel, p, ys))
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = layer()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(out, layer()))
assert lib.wait_timeouts() == 0 and lib.device_errors() == 0
"""


@pytest.mark.parametrize("T", [5, 700])
def test_the_first_calls_of_a_process_are_captured(T):
    subprocess.run([sys.executable, "-c", FIRST.format(T=T)], check=True, cwd=ROOT, timeout=120)
