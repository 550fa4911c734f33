"""Argument checks of the operators on quantised tokens (C entry points):
everything here returns before any GPU work, so it runs without a GPU."""
import ctypes

import pytest
import torch

import quantized_ref as ref


@pytest.fixture(scope="module")
def lib():
    from mxfp4_routed_expert_route_gb300 import _native, build
    build.build()
    return _native.load()


def test_constants_match_the_header():
    import os
    import re
    from mxfp4_routed_expert_route_gb300 import _native as n
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "mxfp4el_quantized.h")).read()
    defs = re.findall(r"#define\s+MXFP4EL_(\w+)\s+(-?\d+)", text)
    assert defs
    for name, val in defs:
        assert getattr(n, name) == int(val), name


def test_route_checks(lib):
    from mxfp4_routed_expert_route_gb300 import _native as n

    def f(logits=1 << 24, dtype=0, stride=64, bias=1 << 28, T=4, E=64, K=4, score=0, groups=8,
          top=4, best=2, norm=1, scaling=1.0, sel=1 << 30, p=1 << 31):
        return lib.mxfp4_route_experts(logits, dtype, stride, bias, T, E, K, score, groups, top,
                                       best, norm, scaling, sel, p, None)

    bad, big = n.ERR_INVALID_ARGUMENT, n.ERR_TOO_LARGE
    for code, kw in ((n.ERR_UNSUPPORTED_DTYPE, dict(dtype=2)), (bad, dict(T=-1)), (bad, dict(E=0)),
                     (bad, dict(K=-1)), (bad, dict(score=2)), (bad, dict(groups=0)),
                     (bad, dict(groups=3)), (bad, dict(top=0)), (bad, dict(top=9)),
                     (bad, dict(best=0)), (bad, dict(best=3)), (bad, dict(K=33)),
                     (bad, dict(scaling=float("inf"))), (bad, dict(scaling=float("nan"))),
                     (bad, dict(stride=63)), (bad, dict(logits=None)), (bad, dict(sel=None)),
                     (bad, dict(p=None)), (bad, dict(logits=(1 << 24) + 2)),
                     (bad, dict(bias=(1 << 28) + 2)), (bad, dict(sel=(1 << 30) + 1)),
                     (big, dict(E=2048, stride=2048)), (big, dict(T=1 << 40)),
                     (big, dict(groups=64, top=64)), (big, dict(stride=1 << 60)),
                     (big, dict(groups=1, top=1, K=40)),
                     (n.ERR_ALIAS, dict(sel=(1 << 24) + 16)), (n.ERR_ALIAS, dict(p=(1 << 28) + 8)),
                     (n.ERR_ALIAS, dict(p=(1 << 30) + 8)), (n.OK, dict(T=0)), (n.OK, dict(K=0))):
        assert f(**kw) == code, kw


def test_quantize_checks(lib):
    from mxfp4_routed_expert_route_gb300 import _native as n

    def q(x=1 << 24, dtype=1, stride=64, rows=3, I=64, packed=1 << 28, scales=1 << 30):
        return lib.mxfp4_quantize(x, dtype, stride, rows, I, packed, scales, None)

    def d(packed=1 << 24, scales=1 << 26, rows=3, I=64, out=1 << 28, dtype=1):
        return lib.mxfp4_dequantize(packed, scales, rows, I, out, dtype, None)

    bad, big, alias = n.ERR_INVALID_ARGUMENT, n.ERR_TOO_LARGE, n.ERR_ALIAS
    for code, kw in ((n.ERR_UNSUPPORTED_DTYPE, dict(dtype=5)), (bad, dict(rows=-1)),
                     (bad, dict(I=0)), (bad, dict(I=48)), (bad, dict(stride=63)),
                     (bad, dict(x=None)), (bad, dict(x=(1 << 24) + 1)), (bad, dict(packed=None)),
                     (bad, dict(packed=(1 << 28) + 8)), (bad, dict(scales=None)),
                     (big, dict(I=1 << 40, stride=1 << 40)), (big, dict(rows=1 << 50)),
                     (big, dict(stride=1 << 62)), (alias, dict(packed=(1 << 24) + 128)),
                     (alias, dict(scales=(1 << 24) + 128)), (alias, dict(scales=(1 << 28) + 20)),
                     (n.OK, dict(rows=0))):
        assert q(**kw) == code, kw
    for code, kw in ((n.ERR_UNSUPPORTED_DTYPE, dict(dtype=5)), (bad, dict(rows=-1)),
                     (bad, dict(I=16)), (bad, dict(packed=None)), (bad, dict(scales=None)),
                     (bad, dict(out=None)), (bad, dict(out=(1 << 28) + 2)),
                     (bad, dict(packed=(1 << 24) + 4)), (big, dict(rows=1 << 50)),
                     (alias, dict(out=(1 << 24) + 16)), (alias, dict(out=(1 << 26) - 16)),
                     (n.OK, dict(rows=0))):
        assert d(**kw) == code, kw


def test_the_reference_quantiser():
    """Pinned to values worked out by hand, ties and limits among them."""
    x = torch.zeros(32)
    x[:16] = torch.tensor([6.0, 0.25, 0.26, 0.75, 0.74, 1.25, 1.26, 1.75, 2.5, 2.6, 3.5, 3.4, 5.0,
                           5.1, -0.2, -7.9])
    p, s = ref.quantize(x)
    assert s.tolist() == [127]
    code = [7, 0, 1, 2, 1, 2, 3, 4, 4, 5, 6, 5, 6, 7, 8, 15] + [0] * 16
    assert p.flatten().tolist() == [code[2 * i] + 16 * code[2 * i + 1] for i in range(16)]
    v = ref.values(p, s)
    assert v[:3].tolist() == [6.0, 0.0, 0.5] and v[15] == -6.0
    # the scale follows the exponent alone, and is cut at both ends
    for top, want in ((1.0, 125), (1.99, 125), (2.0 ** -126, 0), (2.0 ** -149, 0), (0.0, 0),
                      (3.0e38, 252)):
        assert ref.quantize(torch.tensor([top] + [0.0] * 31))[1].item() == want
    assert ref.quantize(torch.tensor([math_inf] + [1.0] * 31))[1].item() == 255


math_inf = float("inf")


def test_the_reference_router():
    ids, w = ref.route(torch.tensor([[1.0, 3.0, 3.0, 2.0]]), 3)
    assert ids.tolist() == [[1, 2, 3]]
    assert abs(w.sum().item() - 1) < 1e-12 and w[0, 0] == w[0, 1]
    # a bias steers the choice and leaves the weights alone
    ids, w = ref.route(torch.tensor([[0.0, 0.0, 0.0, 0.0]]), 2, "sigmoid",
                       torch.tensor([0.0, 0.1, 0.0, 0.2]), normalize=False, scaling=2.0)
    assert ids.tolist() == [[3, 1]] and w.tolist() == [[1.0, 1.0]]
    # one group of two: the sum of two choices decides
    ids, _ = ref.route(torch.tensor([[5.0, -9.0, 2.0, 2.0]]), 2, "sigmoid",
                       torch.zeros(4), groups=2, top_groups=1)
    assert ids.tolist() == [[2, 3]]
    ids, _ = ref.route(torch.tensor([[5.0, -9.0, 2.0, 2.0]]), 2, "sigmoid",
                       torch.zeros(4), groups=2, top_groups=1, group_best=1)
    assert ids.tolist() == [[0, 1]]
    # NaN is never selected
    ids, w = ref.route(torch.tensor([[float("nan"), 1.0]]), 2)
    assert ids.tolist() == [[1, -1]] and w.tolist() == [[1.0, 0.0]]


def test_linear_checks(lib):
    from mxfp4_routed_expert_route_gb300 import _native as n
    size = lib.mxfp4_linear_workspace_size
    rejected = ctypes.c_size_t(-1).value
    assert size(0, 64, 8) == 0 and size(4, 64, 0) == 0
    for args in ((4, 48, 8), (-1, 64, 8), (4, 64, -8), (1 << 40, 64, 8), (4, 1 << 40, 8)):
        assert size(*args) == rejected, args
    need = size(4, 7168, 256)
    assert need > 0 and need % 256 == 0            # few tiles: K is split over units

    def f(xp=1 << 24, xs=1 << 26, wp=1 << 28, ws=1 << 30, out=1 << 32, T=4, I=7168, O=256, dtype=1,
          work=1 << 36, nwork=need):
        return lib.mxfp4_linear(xp, xs, wp, ws, out, T, I, O, dtype, work, nwork, None)

    bad, big, alias = n.ERR_INVALID_ARGUMENT, n.ERR_TOO_LARGE, n.ERR_ALIAS
    for code, kw in ((n.ERR_UNSUPPORTED_DTYPE, dict(dtype=3)), (bad, dict(T=-1)), (bad, dict(I=33)),
                     (bad, dict(I=0)), (bad, dict(O=-1)), (bad, dict(xp=None)), (bad, dict(xs=None)),
                     (bad, dict(wp=None)), (bad, dict(ws=None)), (bad, dict(out=None)),
                     (bad, dict(xp=(1 << 24) + 8)), (bad, dict(wp=(1 << 28) + 4)),
                     (bad, dict(out=(1 << 32) + 1)), (big, dict(T=1 << 31)), (big, dict(O=1 << 31)),
                     (big, dict(T=1 << 30, O=1 << 29)), (alias, dict(out=(1 << 28) + 64)),
                     (alias, dict(out=(1 << 26) - 64)), (n.ERR_WORKSPACE, dict(work=None)),
                     (n.ERR_WORKSPACE, dict(nwork=need - 1)),
                     (n.ERR_WORKSPACE, dict(work=(1 << 36) + 64)), (alias, dict(work=1 << 32)),
                     (alias, dict(work=1 << 28)), (n.OK, dict(T=0)), (n.OK, dict(O=0))):
        assert f(**kw) == code, kw


def test_expert_linear_quantized_checks(lib):
    from mxfp4_routed_expert_route_gb300 import _native as n
    size = lib.mxfp4_expert_linear_quantized_workspace_size
    rejected = ctypes.c_size_t(-1).value
    assert size(0, 4, 64, 8, 2) == 0 and size(4, 4, 64, 0, 2) == 0
    for args in ((4, 4, 60, 8, 2), (-1, 4, 64, 8, 2), (1 << 40, 4, 64, 8, 2),
                 (1 << 20, 4, 64, 8, 1 << 20), (4, 1 << 20, 1 << 20, 1 << 20, 2)):
        assert size(*args) == rejected, args
    need = size(6, 4, 64, 70, 2)
    assert need >= 6 * 2 * 70 * 4 and need % 256 == 0

    def f(xp=1 << 24, xs=1 << 26, wp=1 << 28, ws=1 << 30, sel=1 << 31, p=1 << 32, ys=1 << 33,
          out=1 << 34, T=6, E=4, I=64, O=70, K=2, dtype=1, idx=0, work=1 << 36, nwork=need):
        return lib.mxfp4_expert_linear_quantized(xp, xs, wp, ws, sel, p, ys, out, T, E, I, O, K,
                                                 dtype, idx, work, nwork, None)

    bad, big, alias = n.ERR_INVALID_ARGUMENT, n.ERR_TOO_LARGE, n.ERR_ALIAS
    dt, nows = n.ERR_UNSUPPORTED_DTYPE, n.ERR_WORKSPACE
    for code, kw in ((dt, dict(dtype=2)), (dt, dict(idx=2)), (bad, dict(T=-1)), (bad, dict(E=-1)),
                     (bad, dict(I=40)), (bad, dict(O=-2)), (bad, dict(K=-1)), (bad, dict(xp=None)),
                     (bad, dict(xs=None)), (bad, dict(wp=None)), (bad, dict(ws=None)),
                     (bad, dict(sel=None)), (bad, dict(p=None)), (bad, dict(ys=None)),
                     (bad, dict(out=None)), (bad, dict(xp=(1 << 24) + 8)),
                     (bad, dict(wp=(1 << 28) + 8)), (bad, dict(sel=(1 << 31) + 2)),
                     (bad, dict(idx=1, sel=(1 << 31) + 4)), (bad, dict(p=(1 << 32) + 2)),
                     (bad, dict(ys=(1 << 33) + 1)), (bad, dict(out=(1 << 34) + 1)),
                     (big, dict(T=1 << 31)), (big, dict(T=1 << 20, K=1 << 20)),
                     (big, dict(T=5000, E=5000, K=1)), (alias, dict(out=(1 << 33) + 16)),
                     (alias, dict(out=(1 << 24) + 16)), (alias, dict(out=(1 << 28) + 16)),
                     (alias, dict(out=(1 << 32) - 16)), (nows, dict(work=None)),
                     (nows, dict(nwork=need - 1)), (nows, dict(work=(1 << 36) + 128)),
                     (alias, dict(work=1 << 34)), (alias, dict(work=1 << 33)),
                     (n.OK, dict(T=0)), (n.OK, dict(O=0))):
        assert f(**kw) == code, kw
