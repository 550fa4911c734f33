"""Products on MXFP4 tokens, dense and routed, against plain 64-bit forms
(quantized_ref.py, with the derivation of the bound)."""
import math

import pytest
import torch

import mxfp4_routed_expert_route_gb300 as lib
import quantized_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def rows(*shape, seed=0, lo=118, hi=124):
    """Random MXFP4 rows (..., I): every code, scale bytes of [lo, hi]."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    lead, I = shape[:-1], shape[-1]
    return (torch.randint(0, 256, lead + (I // 32, 16), generator=g, device="cuda", dtype=torch.uint8),
            torch.randint(lo, hi + 1, lead + (I // 32,), generator=g, device="cuda",
                          dtype=torch.uint8))


def check(got, want, bound, dtype):
    half = torch.finfo(dtype).eps / 2
    err = (got.double() - want).abs()
    ok = err <= bound + half * want.abs()
    assert ok.all(), (float((err / (bound + half * want.abs() + 1e-300)).max()), (~ok).nonzero()[:4])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,I,O", [
    (1, 32, 1), (1, 256, 128), (7, 96, 5), (16, 2880, 144), (31, 544, 129), (33, 1056, 257),
    (32, 7168, 512), (191, 320, 127), (192, 512, 384), (193, 288, 130), (400, 2912, 700),
    (1000, 64, 33), (3, 7168, 4096), (1, 4096, 1), (5, 8192, 40)])
def test_linear(T, I, O, dtype):
    x, w = rows(T, I, seed=T), rows(O, I, seed=O + 1)
    got = lib.mxfp4_linear(*x, *w, dtype=dtype)
    assert got.shape == (T, O) and got.dtype == dtype
    vx, vw = ref.values(*x), ref.values(*w)
    check(got, vx @ vw.T, ref.product_bound(vx, vw, I, dtype), dtype)
    assert lib.wait_timeouts() == 0


@pytest.mark.parametrize("T,I,O", [(1500, 7168, 4000), (20, 7168, 30000), (2000, 256, 20000),
                                   (3000, 2880, 2000), (31, 512, 90000)])
def test_linear_many_units_per_sm(T, I, O):
    """Long and short sums, more tiles than the GPU holds at once: every ring of
    the kernel goes round many times."""
    x, w = rows(T, I, seed=T), rows(O, I, seed=O + 1)
    got = lib.mxfp4_linear(*x, *w, dtype=F32)
    vx, vw = ref.values(*x), ref.values(*w)
    check(got, vx @ vw.T, ref.product_bound(vx, vw, I, F32), F32)
    assert lib.wait_timeouts() == 0


def test_linear_of_whole_numbers_is_exact():
    """Sums of quarters under 2^20 fit float32, so every bit has to be right;
    each scale byte is its own, so a wrong one shows."""
    for T, I, O in ((5, 2048, 300), (70, 1312, 190), (300, 416, 260)):
        x, w = rows(T, I, seed=3, lo=127, hi=130), rows(O, I, seed=4, lo=126, hi=129)
        got = lib.mxfp4_linear(*x, *w, dtype=F32)
        assert torch.equal(got.double(), ref.values(*x) @ ref.values(*w).T)


def test_linear_one_value_at_a_time():
    """One nonzero code in each row: which row, column and group it meets, and
    under which scales."""
    I, O, T = 544, 140, 40
    wp = torch.zeros(O, I // 32, 16, dtype=torch.uint8, device="cuda")
    ws = torch.full((O, I // 32), 255 - 128, dtype=torch.uint8, device="cuda")
    xp, xs = rows(T, I, seed=8, lo=100, hi=150)
    at = [(7 * o + 13) % I for o in range(O)]
    for o, i in enumerate(at):
        wp[o, i // 32, i % 32 // 2] = 2 << (4 * (i % 2))          # 1.0
        ws[o] = torch.randint(60, 190, (I // 32,)).to(torch.uint8)
    got = lib.mxfp4_linear(xp, xs, wp, ws, dtype=F32)
    want = ref.values(xp, xs) @ ref.values(wp, ws).T
    assert torch.equal(got.double(), want)


def test_linear_scales_at_both_ends_and_nan():
    xp, xs = rows(20, 128, seed=1, lo=127, hi=127)
    wp, ws = rows(140, 128, seed=2, lo=127, hi=127)
    xs[3], ws[7] = 0, 254                      # 2^-127 and 2^127 cancel
    xs[4], ws[8] = 60, 80
    xs[5, 1] = 255
    ws[9, 2] = 255
    got = lib.mxfp4_linear(xp, xs, wp, ws, dtype=F32).double()
    vx, vw = ref.values(xp, xs), ref.values(wp, ws)
    want = vx @ vw.T
    assert torch.equal(got.isnan(), want.isnan())
    assert got[5].isnan().all() and got[:, 9].isnan().all() and got.isnan().sum() == 140 + 20 - 1
    small = (want.abs() < 2.0 ** 127) & ((want.abs() > 2.0 ** -100) | (want == 0))
    bound = ref.product_bound(vx, vw, 128, F32)
    ok = (got - want).abs() <= bound
    assert ok[small & ~want.isnan()].all()


def test_linear_repeats_bit_for_bit():
    x, w = rows(300, 2880, seed=1), rows(500, 2880, seed=2)
    a = lib.mxfp4_linear(*x, *w, dtype=F32)
    for _ in range(3):
        assert torch.equal(a, lib.mxfp4_linear(*x, *w, dtype=F32))
    # a token's result does not depend on where in a block it stands
    b = lib.mxfp4_linear(x[0][40:260].contiguous(), x[1][40:260].contiguous(), *w, dtype=F32)
    assert torch.equal(a[40:260], b)


def test_linear_scale_bytes_on_any_address():
    """Scale rows that start on odd addresses, at the very end of a buffer."""
    for G, O in ((9, 131), (10, 40), (17, 130)):
        xp, xs = rows(37, 32 * G, seed=G)
        wp, ws = rows(O, 32 * G, seed=O)
        want = lib.mxfp4_linear(xp, xs, wp, ws, dtype=F32)
        for skip in (1, 2, 3, 5):
            b = torch.empty(skip + ws.numel(), dtype=torch.uint8, device="cuda")
            ws2 = b[skip:].view(ws.shape)
            ws2.copy_(ws)
            c = torch.empty(skip + xs.numel(), dtype=torch.uint8, device="cuda")
            xs2 = c[skip:].view(xs.shape)
            xs2.copy_(xs)
            assert torch.equal(want, lib.mxfp4_linear(xp, xs2, wp, ws2, dtype=F32))


def make_routed(T, E, K, I, O, dtype, seed=0, picks=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, w = rows(T, I, seed=seed + 1), rows(E, O, I, seed=seed + 2)
    if picks is None:
        sel = torch.rand(T, E, generator=g, device="cuda").argsort(1)[:, :K].int()
    else:
        sel = torch.tensor(picks, device="cuda", dtype=torch.int32)
    p = torch.softmax(torch.randn(T, K, generator=g, device="cuda"), 1)
    ys = torch.randn(T, O, generator=g, device="cuda").to(dtype)
    return x, w, sel.contiguous(), p, ys


def check_routed(got, x, w, sel, p, ys, I, dtype):
    T, K = sel.shape
    vx = ref.values(*x)
    want, bound = ys.double(), torch.zeros_like(ys, dtype=torch.float64)
    terms = ys.double().abs()
    for e in sorted(set(sel.flatten().tolist())):
        if not 0 <= e < w[0].shape[0]:
            continue
        vw = ref.values(w[0][e], w[1][e])
        t, k = (sel == e).nonzero(as_tuple=True)
        q = p[t, k].double()[:, None]
        y = vx[t] @ vw.T * q
        want = want.index_add(0, t, y)
        bound.index_add_(0, t, ref.product_bound(vx[t], vw, I, dtype, more=4) * q.abs())
        terms.index_add_(0, t, y.abs())
    # the combine: K multiply-adds in float32 on top of the shared output, and
    # the addition of up to eight splits (in `more` above)
    bound += (K + 1) * 2.0 ** -24 * terms
    check(got, want, bound, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,E,K,I,O", [
    (1, 1, 1, 32, 1), (1, 8, 2, 256, 128), (8, 128, 4, 2880, 576), (16, 40, 8, 7168, 300),
    (33, 6, 2, 1056, 257), (300, 6, 2, 288, 130), (64, 2, 1, 512, 128), (700, 5, 3, 96, 65),
    (2000, 3, 2, 64, 40), (9000, 16, 1, 64, 8), (40, 600, 3, 64, 33), (5, 3, 3, 160, 1001),
    (3000, 24, 2, 2880, 700), (48, 100, 4, 1536, 1500)])
def test_experts(T, E, K, I, O, dtype):
    x, w, sel, p, ys = make_routed(T, E, K, I, O, dtype, seed=T)
    got = lib.mxfp4_expert_linear_quantized(*x, *w, sel, p, ys)
    assert got.dtype == dtype
    check_routed(got, x, w, sel, p, ys, I, dtype)
    assert torch.equal(got, lib.mxfp4_expert_linear_quantized(*x, *w, sel.long(), p, ys))
    assert lib.wait_timeouts() == 0 and lib.device_errors() == 0


@pytest.mark.parametrize("counts", [(31, 1), (32, 0, 1), (33,), (191, 193, 0, 192), (1, 500, 2),
                                    (0, 0, 40), (16, 17, 15, 96, 97)])
def test_experts_by_tokens_per_expert(counts):
    picks = [[e] for e, n in enumerate(counts) for _ in range(n)]
    g = torch.Generator().manual_seed(1)
    picks = [picks[i] for i in torch.randperm(len(picks), generator=g)]
    x, w, sel, p, ys = make_routed(len(picks), len(counts), 1, 544, 150, BF16, picks=picks)
    check_routed(lib.mxfp4_expert_linear_quantized(*x, *w, sel, p, ys), x, w, sel, p, ys, 544, BF16)


@pytest.mark.parametrize("T,K,E", [(255, 1, 100), (64, 4, 90), (257, 1, 200), (128, 2, 300),
                                   (32, 8, 3), (256, 1, 1), (43, 6, 40)])
def test_experts_around_the_kernels_own_lists(T, K, E):
    """Up to 256 pairs the product makes its routing lists itself."""
    g = torch.Generator().manual_seed(T)
    picks = torch.randint(-1, E + 1, (T, K), generator=g).tolist()
    x, w, sel, p, ys = make_routed(T, E, K, 96, 70, F32, seed=2, picks=picks)
    lib.device_errors()
    for ids in (sel, sel.long()):
        got = lib.mxfp4_expert_linear_quantized(*x, *w, ids, p, ys)
        check_routed(got, x, w, sel, p, ys, 96, F32)
        assert lib.device_errors() == sum(not 0 <= e < E for row in picks for e in row)


def test_a_chain_of_calls_without_waiting():
    """Router, quantiser and experts again and again, each on what the one before
    wrote: no kernel may start on what is not there yet."""
    T, E, K, I = 24, 12, 2, 256
    w = rows(E, I, I, seed=5, lo=114, hi=118)
    gate = torch.randn(I, E, generator=torch.Generator().manual_seed(1)).cuda()
    x0 = torch.randn(T, I, generator=torch.Generator().manual_seed(2)).cuda().to(BF16)

    def run(wait):
        x, out = x0, []
        for _ in range(30):
            sel, p = lib.route_experts(x.float() @ gate, K, score="sigmoid")
            q = lib.quantize_mxfp4(x)
            if wait:
                torch.cuda.synchronize()
            x = lib.mxfp4_expert_linear_quantized(*q, *w, sel, p, x)
            if wait:
                torch.cuda.synchronize()
            x = (x.float() / x.float().abs().amax(1, keepdim=True)).to(BF16)
            out.append(x)
        return out

    want = run(True)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(run(False), want))


@pytest.mark.parametrize("T", [4, 90])
def test_experts_the_same_id_twice_and_ids_out_of_range(T):
    picks = [[1, 1, 5] if t % 3 == 0 else [-1, 2, 1 << 30] if t % 3 == 1 else [4, -7, 0]
             for t in range(T)]
    x, w, sel, p, ys = make_routed(T, 5, 3, 288, 200, F32, picks=picks)
    lib.device_errors()
    got = lib.mxfp4_expert_linear_quantized(*x, *w, sel, p, ys)
    check_routed(got, x, w, sel, p, ys, 288, F32)
    bad = sum(not 0 <= e < 5 for row in picks for e in row)
    assert lib.device_errors() == bad


@pytest.mark.parametrize("T,E,K,I,O", [(4100, 4000, 1, 64, 40), (3000, 3500, 2, 32, 20),
                                       (50000, 2500, 1, 32, 136)])
def test_experts_long_lists(T, E, K, I, O):
    """Thousands of experts with tokens, narrow and wide blocks: the kernel's
    lists take shared memory from its ring of stages."""
    x, w, sel, p, ys = make_routed(T, E, K, I, O, F32, seed=1,
                                   picks=[[(t * 7 + k * 3) % E for k in range(K)] for t in range(T)])
    got = lib.mxfp4_expert_linear_quantized(*x, *w, sel, p, ys)
    vx, vw = ref.values(*x), ref.values(*w)
    want, bound = ys.double(), (K + 1) * 2.0 ** -24 * ys.double().abs()
    for k in range(K):
        m = vw[sel[:, k].long()]
        y = (m @ vx[:, :, None])[..., 0] * p[:, k:k + 1].double()
        want = want + y
        terms = (m.abs() @ vx.abs()[:, :, None])[..., 0] * p[:, k:k + 1].double()
        bound = bound + (I / 64 + 5) * 2.0 ** -22 * terms + (K + 1) * 2.0 ** -24 * y.abs()
    check(got, want, bound, F32)
    assert lib.wait_timeouts() == 0 and lib.device_errors() == 0


def test_calls_on_two_streams_at_once():
    x1, w1, sel1, p1, ys1 = make_routed(300, 6, 2, 288, 130, F32, seed=1)
    x2, w2 = rows(500, 2880, seed=2), rows(1500, 2880, seed=3)
    want1 = lib.mxfp4_expert_linear_quantized(*x1, *w1, sel1, p1, ys1)
    want2 = lib.mxfp4_linear(*x2, *w2, dtype=F32)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got1, got2 = [], []
    for _ in range(10):
        with torch.cuda.stream(streams[0]):
            got1.append(lib.mxfp4_expert_linear_quantized(*x1, *w1, sel1, p1, ys1))
        with torch.cuda.stream(streams[1]):
            got2.append(lib.mxfp4_linear(*x2, *w2, dtype=F32))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want1) for g in got1) and all(torch.equal(g, want2) for g in got2)


def test_experts_nothing_to_add():
    x, w, sel, p, ys = make_routed(5, 4, 2, 64, 70, BF16)
    none = torch.empty(5, 0, device="cuda")
    assert torch.equal(lib.mxfp4_expert_linear_quantized(*x, *w, none.int(), none, ys), ys)
    empty = (w[0][:0], w[1][:0])
    lib.device_errors()
    assert torch.equal(lib.mxfp4_expert_linear_quantized(*x, *empty, sel, p, ys), ys)
    assert lib.device_errors() == 10
    assert torch.equal(lib.mxfp4_expert_linear_quantized(*x, *w, sel - 9, p, ys), ys)
    assert lib.device_errors() == 10
    cut = (x[0][:0], x[1][:0], *w, sel[:0], p[:0], ys[:0])
    assert lib.mxfp4_expert_linear_quantized(*cut).shape == (0, 70)


def test_experts_match_the_linear_on_the_tokens_values():
    """The same layer through mxfp4_expert_linear on the values that the MXFP4
    tokens stand for."""
    for T in (6, 200):
        x, w, sel, p, ys = make_routed(T, 8, 2, 512, 256, F32, seed=T)
        got = lib.mxfp4_expert_linear_quantized(*x, *w, sel, p, ys)
        want = lib.mxfp4_expert_linear(lib.dequantize_mxfp4(*x, F32), *w, sel, p, ys)
        torch.testing.assert_close(got, want, rtol=1e-5, atol=1e-5 * float(want.abs().max()))


def test_a_run_of_them_together():
    """Router, quantiser and experts, as a layer runs them; on another stream
    and in a graph that is replayed with new tokens."""
    T, E, K, I, O = 50, 16, 3, 320, 192
    w = rows(E, O, I, seed=5)
    g = torch.Generator(device="cuda").manual_seed(6)
    gate = torch.randn(I, E, generator=g, device="cuda") / math.sqrt(I)
    bias = torch.randn(E, generator=g, device="cuda") * 0.01
    x = torch.randn(T, I, generator=g, device="cuda").to(BF16)

    def layer(x):
        sel, p = lib.route_experts(x.float() @ gate, K, score="sigmoid", bias=bias, groups=4,
                                   top_groups=2, scaling=2.0)
        return sel, p, lib.mxfp4_expert_linear_quantized(*lib.quantize_mxfp4(x), *w, sel, p,
                                                         x[:, :O].contiguous())

    def verify(x, sel, p, y):
        want_sel, want_p = ref.route((x.float() @ gate).cpu(), K, "sigmoid", bias.cpu(), 4, 2,
                                     scaling=2.0)
        assert torch.equal(sel.cpu(), want_sel)
        torch.testing.assert_close(p.double().cpu(), want_p, rtol=ref.WEIGHT_RTOL, atol=0)
        q = tuple(t.cuda() for t in ref.quantize(x))
        check_routed(y, q, w, sel, p, x[:, :O], I, BF16)

    verify(x, *layer(x))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = layer(x)
    side.synchronize()
    verify(x, *out)
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    x2 = x.clone()
    with torch.cuda.graph(graph):
        out = layer(x)
    with torch.cuda.graph(other):
        out2 = layer(x2)
    for seed in (1, 2):
        x.copy_(torch.randn(T, I, generator=g, device="cuda"))
        x2.copy_(torch.randn(T, I, generator=g, device="cuda"))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            other.replay()
        graph.replay()
        torch.cuda.synchronize()
        verify(x, *out)
        verify(x2, *out2)
    assert lib.wait_timeouts() == 0 and lib.device_errors() == 0


def test_outputs_are_written_where_asked_and_nowhere_else():
    x, w = rows(21, 288, seed=1), rows(70, 288, seed=2)
    buf = torch.full((23, 70), 9.0, device="cuda", dtype=BF16)
    got = lib.mxfp4_linear(*x, *w, out=buf[1:22])
    assert got.data_ptr() == buf[1].data_ptr() and (buf[[0, 22]] == 9).all()
    assert torch.equal(got, lib.mxfp4_linear(*x, *w))
    x, w, sel, p, ys = make_routed(21, 4, 2, 288, 70, BF16)
    buf.fill_(9.0)
    got = lib.mxfp4_expert_linear_quantized(*x, *w, sel, p, ys, out=buf[1:22])
    assert (buf[[0, 22]] == 9).all()
    assert torch.equal(got, lib.mxfp4_expert_linear_quantized(*x, *w, sel, p, ys))
    with pytest.raises(lib.MXFP4Error):
        lib.mxfp4_expert_linear_quantized(*x, *w, sel, p, ys, out=ys)


def test_refusals():
    x, w, sel, p, ys = make_routed(6, 4, 2, 64, 70, BF16)
    dense = (w[0][0], w[1][0])
    for args in ((x[0], x[1], w[0], w[1]), (x[0], x[1], dense[0][:, :1], dense[1][:, :1]),
                 (x[0], x[1][:5], *dense), (x[0].cpu(), x[1].cpu(), *dense),
                 (x[0], x[1], dense[0].cpu(), dense[1].cpu()),
                 (x[0].transpose(0, 1).contiguous().transpose(0, 1), x[1], *dense)):
        with pytest.raises((ValueError, TypeError)):
            lib.mxfp4_linear(*args)
    with pytest.raises(TypeError):
        lib.mxfp4_linear(*x, *dense, dtype=torch.float16)
    with pytest.raises(ValueError):
        lib.mxfp4_linear(*x, *dense, out=torch.empty(6, 71, dtype=BF16, device="cuda"))
    f = lib.mxfp4_expert_linear_quantized
    for args in ((*x, *dense, sel, p, ys), (*x, *w, sel[:5], p, ys), (*x, *w, sel, p[:, :1], ys),
                 (*x, *w, sel, p, ys[:, :69]), (*x, *w, sel.float(), p, ys),
                 (*x, *w, sel, p.double(), ys), (*x, *w, sel, p, ys.half()),
                 (*x, *w, sel.cpu(), p, ys), (*x, *w, sel, p, ys.cpu()),
                 (*x, *w, sel.T.contiguous().T, p, ys)):
        with pytest.raises((ValueError, TypeError)):
            f(*args)
