"""Expert routing and the MXFP4 quantiser against plain 64-bit forms
(quantized_ref.py, with the derivation of the tolerance)."""
import math

import pytest
import torch

import mxfp4_routed_expert_route_gb300 as lib
import quantized_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def normal(*shape, seed=0, by=1.0, dtype=F32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * by).to(dtype)


# ---------------------------------------------------------------- quantiser --
def check_quantized(x, packed, scales):
    want_p, want_s = ref.quantize(x)
    assert torch.equal(scales.cpu(), want_s)
    assert torch.equal(packed.cpu(), want_p)
    for dtype in (F32, BF16):
        got = lib.dequantize_mxfp4(packed, scales, dtype)
        want = ref.values(want_p, want_s).reshape(got.shape)
        assert got.dtype == dtype
        assert torch.equal(torch.nan_to_num(got.double().cpu(), nan=7e300, posinf=math.inf),
                           torch.nan_to_num(want.to(dtype).double(), nan=7e300, posinf=math.inf))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", [(1, 32), (3, 2880), (1021, 96), (5, 7, 64), (2, 0, 32), (0, 64),
                                   (64,), (257, 7168)])
def test_quantize(shape, dtype):
    x = normal(*shape, seed=len(shape), dtype=F32)
    x = (x * torch.exp(4 * normal(*shape[:-1], 1, seed=3))).to(dtype)
    packed, scales = lib.quantize_mxfp4(x)
    I = shape[-1]
    assert packed.shape == shape[:-1] + (I // 32, 16) and scales.shape == shape[:-1] + (I // 32,)
    if x.numel():
        check_quantized(x, packed, scales)
    else:
        assert lib.dequantize_mxfp4(packed, scales).shape == shape


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantize_every_tie_and_border(dtype):
    """Half steps of every code and the values around them, at scales from the
    smallest to the largest, both signs."""
    eps = 2.0 ** -7
    y = torch.tensor([v for t in (0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7, 7.9)
                      for v in (t * (1 - eps), t, t * (1 + eps))])
    rows = []
    for e in (-149, -140, -128, -127, -126, -125, -30, 0, 3, 60, 120, 125):
        for top in (4.0, 6.0, 7.75):
            v = torch.cat([y, -y])[None].double() * 2.0 ** e
            v = torch.nn.functional.pad(v, (0, 10)).view(-1, 14)
            v = torch.cat([v, v.new_full((v.shape[0], 1), top * 2.0 ** e),
                           v.new_zeros(v.shape[0], 17)], 1)
            rows.append(v)
    x = torch.cat(rows).float().to(dtype).cuda()
    x[x.isinf()] = 0
    packed, scales = lib.quantize_mxfp4(x)
    check_quantized(x, packed, scales)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantize_what_is_not_finite(dtype):
    x = normal(6, 96, dtype=dtype)
    x[0, 5], x[1, 40], x[2, 95], x[3, :] = math.nan, math.inf, -math.inf, 0.0
    x[4, :32] = -0.0
    packed, scales = lib.quantize_mxfp4(x)
    assert scales[0].tolist()[0] == 255 and scales[1].tolist()[1] == 255
    check_quantized(x, packed, scales)
    v = lib.dequantize_mxfp4(packed, scales)
    assert v[0, :32].isnan().all() and not v[0, 32:].isnan().any()


def test_every_code_under_every_scale():
    packed = torch.arange(256, dtype=torch.uint8).view(16, 16).repeat(256, 1).view(256, 16, 16)
    scales = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 16)
    for dtype in (F32, BF16):
        got = lib.dequantize_mxfp4(packed.cuda(), scales.cuda(), dtype).double().cpu()
        want = ref.values(packed, scales).to(dtype).double()
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got.nan_to_num(nan=0), want.nan_to_num(nan=0))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("skip,width", [(0, 320), (8, 328), (1, 321), (3, 500)])
def test_quantize_rows_of_a_wider_matrix(skip, width, dtype):
    """Views with any row distance and start, aligned to the element alone."""
    x = normal(19, width, dtype=dtype)[:, skip:skip + 288]
    packed, scales = lib.quantize_mxfp4(x)
    check_quantized(x.contiguous(), packed, scales)
    y = normal(4, 6, width, seed=2, dtype=dtype)[..., skip:skip + 288]
    packed, scales = lib.quantize_mxfp4(y)
    check_quantized(y.contiguous(), packed, scales)


def test_quantize_writes_into_given_tensors_and_nowhere_else():
    x = normal(5, 64, dtype=BF16)
    p = torch.full((7, 2, 16), 99, dtype=torch.uint8, device="cuda")
    s = torch.full((7, 2), 99, dtype=torch.uint8, device="cuda")
    got = lib.quantize_mxfp4(x, p[1:6], s[1:6])
    assert got[0].data_ptr() == p[1].data_ptr()
    check_quantized(x, p[1:6], s[1:6])
    assert (p[[0, 6]] == 99).all() and (s[[0, 6]] == 99).all()


def test_quantize_refusals():
    x = normal(4, 64)
    for bad in (x.cpu(), x.half(), x[:, :48], normal(64, 4).T, x.expand(2, 4, 64)):
        with pytest.raises((ValueError, TypeError)):
            lib.quantize_mxfp4(bad)
    p, s = lib.quantize_mxfp4(x)
    with pytest.raises(ValueError):
        lib.quantize_mxfp4(x, p[:3], s)
    with pytest.raises(ValueError):
        lib.quantize_mxfp4(x, p, s.int())
    for args in ((p, s[:3]), (p[..., :8], s), (p.cpu(), s), (p, s.cpu()), (p.transpose(0, 1), s.T)):
        with pytest.raises((ValueError, TypeError)):
            lib.dequantize_mxfp4(*args)
    with pytest.raises(TypeError):
        lib.dequantize_mxfp4(p, s, torch.float16)
    with pytest.raises(TypeError):
        lib.dequantize_mxfp4(p.char(), s)


# ------------------------------------------------------------------- router --
def check_routed(logits, K, sel, p, **kw):
    bias = kw.pop("bias", None)
    want_sel, want_p = ref.route(logits.cpu(), K, bias=None if bias is None else bias.cpu(), **kw)
    assert sel.dtype == torch.int32 and p.dtype == F32
    assert torch.equal(sel.cpu(), want_sel)
    # Under 2^-126 / 2^-24 a float32 weight loses bits of its own.
    torch.testing.assert_close(p.cpu().double(), want_p, rtol=ref.WEIGHT_RTOL, atol=2.0 ** -120)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,E,K,groups,top,best", [
    (1, 1, 1, 1, 1, 2), (8, 32, 4, 1, 1, 2), (33, 5, 5, 1, 1, 1), (7, 384, 8, 1, 1, 2),
    (300, 128, 4, 1, 1, 2), (65, 256, 8, 8, 4, 2), (65, 256, 8, 8, 4, 1), (20, 58, 6, 2, 1, 2),
    (9, 160, 6, 8, 3, 1), (5, 1024, 32, 32, 32, 2), (3, 1024, 32, 1, 1, 2), (17, 96, 13, 32, 7, 2),
    (11, 33, 32, 1, 1, 2), (4, 31, 1, 31, 1, 2), (6, 511, 16, 7, 3, 2)])
def test_route(T, E, K, groups, top, best, dtype, score):
    logits = normal(T, E, seed=T + E, by=1.5, dtype=dtype)
    kw = dict(score=score, groups=groups, top_groups=top, group_best=best)
    for bias in (None, normal(E, seed=E, by=0.1)):
        for more in (dict(), dict(normalize=False, scaling=2.5)):
            sel, p = lib.route_experts(logits, K, bias=bias, **kw, **more)
            check_routed(logits, K, sel, p, bias=bias, **kw, **more)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top", [(1, 1), (4, 2)])
def test_route_decides_next_to_the_border(score, groups, top):
    """Choices that differ by less than float32 shows, and ones that do not
    differ: the order is float64's, equal ones go to the lower index."""
    g = torch.Generator().manual_seed(5)
    T, E, K = 400, 64, 8
    logits = torch.randn(T, 8, generator=g)[:, torch.randint(0, 8, (E,), generator=g)]
    logits = logits + torch.randint(-2, 3, (T, E), generator=g) * 2.0 ** -21 * logits.abs()
    bias = torch.randn(4, generator=g)[torch.randint(0, 4, (E,), generator=g)] * 0.1
    bias = bias + torch.randint(-1, 2, (E,), generator=g) * 2.0 ** -25
    for b in (None, bias, torch.zeros(E)):
        b = None if b is None else b.cuda()
        sel, p = lib.route_experts(logits.cuda(), K, score=score, bias=b, groups=groups,
                                   top_groups=top)
        check_routed(logits, K, sel, p, score=score, bias=b, groups=groups, top_groups=top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_route_what_is_not_finite(score, groups):
    inf, nan = math.inf, math.nan
    logits = normal(12, 16, seed=9)
    logits[0, 3] = nan
    logits[1, :] = nan
    logits[2, 1:] = nan
    logits[3, :8] = -inf
    logits[4, :] = -inf
    logits[5, 6] = inf
    logits[6, [2, 9]] = inf
    logits[7, :12] = nan
    logits[8, :] = 200.0
    logits[9, :] = -200.0
    logits[10, :] = torch.finfo(F32).min
    logits[11, ::2] = torch.finfo(F32).min
    bias = normal(16, seed=4, by=0.1)
    masked = bias.clone()
    masked[[0, 5, 6, 7, 13]] = -inf
    for b in (None, bias, masked):
        for normalize in (True, False):
            sel, p = lib.route_experts(logits, 6, score=score, bias=b, groups=groups,
                                       top_groups=max(1, groups // 2 + 1), normalize=normalize)
            check_routed(logits, 6, sel, p, score=score, bias=b, groups=groups,
                         top_groups=max(1, groups // 2 + 1), normalize=normalize)
            assert not p.isnan().any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_weights_of_small_scores(score):
    """Scores down to 2^-140, whose quotient by the sum plus 1e-20 is far from
    small. A score under 2^-126 is off by half of 2^-149, and the divisor is at
    least 1e-20: 7.1e-26 a weight, and as much again for the sum."""
    logits = torch.linspace(-97, -30, 64).repeat(20, 1)[:, torch.randperm(64)]
    logits[:, 0] += torch.arange(20)
    if score == "softmax":
        logits[:, 5] = 0.0                       # the others' scores are as small
    sel, p = lib.route_experts(logits.cuda(), 24, score=score)
    want_sel, want_p = ref.route(logits, 24, score=score)
    assert torch.equal(sel.cpu(), want_sel)
    torch.testing.assert_close(p.cpu().double(), want_p, rtol=ref.WEIGHT_RTOL, atol=1.5e-25)
    low = logits - 60 * (logits > -60)
    sel, p = lib.route_experts(low.cuda(), 24, score="sigmoid")
    want_sel, want_p = ref.route(low, 24, score="sigmoid")
    assert torch.equal(sel.cpu(), want_sel)
    torch.testing.assert_close(p.cpu().double(), want_p, rtol=ref.WEIGHT_RTOL, atol=1.5e-25)


@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_groups_whose_scores_round_together(score, best):
    """Different logits whose float64 scores are the same number (1, or 0.5, or
    nearly the largest): groups of equal score go to the lower index."""
    g = torch.Generator().manual_seed(3)
    big = torch.randint(30, 60, (60, 32), generator=g).float()
    small = torch.randint(-4, 5, (60, 32), generator=g) * 1e-20
    mixed = torch.where(torch.rand(60, 32, generator=g) < 0.5, big, small)
    far = torch.randint(-3, 3, (60, 32), generator=g) * 400.0
    for logits in (big, small, mixed, far):
        for top in (1, 3):
            sel, p = lib.route_experts(logits.cuda(), 4, score=score, groups=8, top_groups=top,
                                       group_best=best)
            check_routed(logits, 4, sel, p, score=score, groups=8, top_groups=top, group_best=best)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_experts_kept_out_by_the_bias(score):
    logits = normal(200, 64, seed=6)
    bias = normal(64, seed=7, by=0.05)
    bias[8:24] = -math.inf                     # two groups of eight
    bias[40] = -math.inf
    for top in (3, 6):
        sel, p = lib.route_experts(logits, 8, score=score, bias=bias, groups=8, top_groups=top)
        check_routed(logits, 8, sel, p, score=score, bias=bias, groups=8, top_groups=top)
        assert not ((sel >= 8) & (sel < 24)).any() and not (sel == 40).any()
    sel, p = lib.route_experts(logits, 8, score=score, bias=bias)
    check_routed(logits, 8, sel, p, score=score, bias=bias)


def test_route_rows_of_a_wider_matrix_and_given_outputs():
    wide = normal(21, 70, seed=1, dtype=BF16)
    logits = wide[:, 3:67]
    sel = torch.full((23, 4), 77, dtype=torch.int32, device="cuda")
    p = torch.full((23, 4), 77.0, device="cuda")
    got = lib.route_experts(logits, 4, selected_experts=sel[1:22], mixture_weights=p[1:22])
    assert got[0].data_ptr() == sel[1].data_ptr()
    check_routed(logits.contiguous(), 4, sel[1:22], p[1:22])
    assert (sel[[0, 22]] == 77).all() and (p[[0, 22]] == 77).all()


def test_route_many_tokens_and_nothing_to_do():
    logits = normal(20011, 48, seed=2)
    bias = normal(48, seed=3, by=0.05)
    sel, p = lib.route_experts(logits, 6, score="sigmoid", bias=bias)
    score = torch.sigmoid(logits.double())
    want = (score + bias.double()).sort(dim=1, descending=True, stable=True).indices[:, :6]
    assert torch.equal(sel.long(), want)
    w = score.gather(1, want)
    torch.testing.assert_close(p.double(), w / w.sum(1, keepdim=True), rtol=ref.WEIGHT_RTOL, atol=0)
    for T, K in ((0, 4), (5, 0)):
        sel, p = lib.route_experts(logits[:T], K)
        assert sel.shape == (T, K) and p.shape == (T, K)


def test_route_refusals():
    x = normal(4, 64)
    for bad in (x.cpu(), x.half(), x[0], x.T):
        with pytest.raises(ValueError):
            lib.route_experts(bad, 2)
    for kw in (dict(K=65), dict(K=-1), dict(K=2, groups=3), dict(K=2, groups=0),
               dict(K=2, groups=4, top_groups=5), dict(K=2, groups=4, top_groups=0),
               dict(K=17, groups=4, top_groups=1), dict(K=2, group_best=3),
               dict(K=2, score="relu"), dict(K=2, bias=x[0].bfloat16()),
               dict(K=2, bias=x[0, :63]), dict(K=2, bias=x[0].cpu()),
               dict(K=2, bias=normal(64, 2)[:, 0]),
               dict(K=2, selected_experts=torch.empty(4, 3, dtype=torch.int32, device="cuda")),
               dict(K=2, mixture_weights=torch.empty(4, 2, dtype=BF16, device="cuda"))):
        with pytest.raises(ValueError):
            lib.route_experts(x, **kw)
    for kw in (dict(K=33), dict(K=2, groups=64)):
        with pytest.raises(lib.MXFP4Error):
            lib.route_experts(x, **kw)
    with pytest.raises(lib.MXFP4Error):
        lib.route_experts(normal(2, 1025), 2)
    with pytest.raises(lib.MXFP4Error):
        lib.route_experts(x, 2, scaling=math.inf)


def test_streams_and_graphs():
    """On another stream, and captured and replayed with new inputs."""
    logits, x = normal(33, 96, seed=1), normal(33, 320, seed=2, dtype=BF16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sel, p = lib.route_experts(logits, 5)
        packed, scales = lib.quantize_mxfp4(x)
        v = lib.dequantize_mxfp4(packed, scales)
    side.synchronize()
    check_routed(logits, 5, sel, p)
    check_quantized(x, packed, scales)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sel, p = lib.route_experts(logits, 5, score="sigmoid")
        packed, scales = lib.quantize_mxfp4(x)
        v = lib.dequantize_mxfp4(packed, scales)
    for seed in (7, 8):
        logits.copy_(normal(33, 96, seed=seed))
        x.copy_(normal(33, 320, seed=seed, dtype=BF16))
        graph.replay()
        torch.cuda.synchronize()
        check_routed(logits, 5, sel, p, score="sigmoid")
        check_quantized(x, packed, scales)
        assert torch.equal(v, lib.dequantize_mxfp4(packed, scales))
