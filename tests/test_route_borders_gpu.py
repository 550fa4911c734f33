"""The router next to its borders: exact ties there, and choices whose float32
roundings are larger than what tells them apart. Against the plain 64-bit form."""
import pytest
import torch

import mxfp4_routed_expert_route_gb300 as lib
import quantized_ref as ref

pytestmark = pytest.mark.gpu


def check(logits, K, bias, **kw):
    sel, p = lib.route_experts(logits.cuda(), K, bias=bias.cuda(), **kw)
    want_sel, want_p = ref.route(logits, K, bias=bias, **kw)
    assert torch.equal(sel.cpu(), want_sel)
    torch.testing.assert_close(p.cpu().double(), want_p, rtol=ref.WEIGHT_RTOL, atol=2.0 ** -120)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("ties", [2, 3])
@pytest.mark.parametrize("above", [0, 1, 4])
def test_a_tie_at_the_border_and_a_better_one_behind_it(above, ties, score):
    """`ties` equal experts share the last place, and a later one that float32
    does not tell from them is truly higher."""
    E, rows = 64, []
    for j in range(8, 41):
        row = torch.full((E,), -20.0)
        if score == "sigmoid":                     # saturated: sigmoid(17) is 1 - 4e-8
            low, high = 16.0 + j / 8, 16.0 + j / 8 + 0.125
            row[40:40 + above] = 5.0
        else:                                      # half an ulp of a share, or a few
            low = -1.0 - j / 16
            high = low + 2.0 ** -22 * (1 + j % 3)
            row[40:40 + above] = 0.0
            row[63] = -0.5
        row[3:3 + ties] = low
        row[3 + ties + j % 5] = high
        rows.append(row)
    bias = torch.zeros(E)
    bias[40:40 + above] = 0.5
    extra = 0 if score == "sigmoid" else 1         # the softmax rows' expert 63
    for K in (above + extra + 1, above + extra + 2):
        check(torch.stack(rows), K, bias, score=score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top", [(1, 1), (4, 2)])
def test_many_ties_of_nearly_equal_choices(score, groups, top):
    g = torch.Generator().manual_seed(11)
    T, E = 200, 64
    if score == "sigmoid":
        logits = 16.0 + torch.randint(0, 12, (T, E), generator=g) / 8.0
    else:
        logits = torch.randint(-2, 0, (T, E), generator=g) * 1.0
        logits = logits * (1 + torch.randint(0, 4, (T, E), generator=g) * 2.0 ** -22)
        logits[:, 0] = 1.0
    for bias in (torch.zeros(E), torch.full((E,), 0.25)):
        for K in (1, 2, 5, 9, 16):
            check(logits, K, bias, score=score, groups=groups, top_groups=top)


def opposite(E, B):
    """Biases +B and -B in turn, exact in float32."""
    return torch.tensor([B, -B] * (E // 2), dtype=torch.float32)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("B", [1.0, 10.0, 64.0, 1e3, 3e4, 1e6])
def test_groups_of_large_biases_of_both_signs(B, score):
    """A group's two choices cancel, their roundings (at B's size) do not."""
    g = torch.Generator().manual_seed(int(B))
    T, E = 300, 64
    for by in (1.0, 1e-2, 1e-4):
        logits = by * torch.randn(T, E, generator=g)
        for top in (1, 8, 31):
            check(logits, 1, opposite(E, B), score=score, groups=32, top_groups=top)
        check(logits, 3, opposite(E, B), score=score, groups=8, top_groups=3)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_one_group_of_large_biases_among_small_ones(score):
    """The border lies between other groups, or at the one whose sums are rough."""
    g = torch.Generator().manual_seed(4)
    T, E = 400, 32
    bias = 0.01 * torch.randn(E, generator=g)
    bias[8:10] = torch.tensor([4096.0, -4096.0])
    bias[10:12] = -1e5
    for by in (1.0, 1e-3):
        logits = by * torch.randn(T, E, generator=g)
        for top in (1, 2, 4, 7):
            check(logits, 2, bias, score=score, groups=8, top_groups=top)


def test_group_sums_that_float32_puts_the_other_way_round():
    """Biases of 1000: a choice is rounded to multiples of u = 2^-14. Group 0's
    scores lie 0.6 u above such a multiple and are rounded up, group 1's 0.4 u
    above, one of them a whole u higher, and are rounded down: group 1's sum is
    the larger by 0.6 u and comes out smaller by u."""
    u = 2.0 ** -14
    s = torch.tensor([0.5 + 0.6 * u, 0.5 + 0.6 * u, 0.5 + 1.4 * u, 0.5 + 0.4 * u],
                     dtype=torch.float64)
    logits = torch.log(s / (1 - s)).float()[None].repeat(9, 1)
    bias = torch.tensor([1000.0, -1000.0, 1000.0, -1000.0])
    check(logits, 1, bias, score="sigmoid", groups=2, top_groups=1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_of_infinite_biases_and_of_sums_past_float32(score):
    g = torch.Generator().manual_seed(8)
    inf, big = float("inf"), 3.0e38
    logits = torch.randn(50, 16, generator=g)
    for values in ((inf, 0.0, inf, 1.0, 0.0, 0.0, -inf, 0.0), (big, big, 2.9e38, big, 0.0, 0.0, 1.0, 1.0),
                   (-big, -big, -big, -2.9e38, 0.0, -big, -inf, -inf), (inf, inf, big, big, inf, -big, 0.0, 0.0)):
        bias = torch.tensor(values).repeat(2)
        for groups, top in ((8, 1), (8, 2), (8, 5), (8, 7), (4, 2)):
            check(logits, 2, bias, score=score, groups=groups, top_groups=top)
            check(logits, 2, bias, score=score, groups=groups, top_groups=top, group_best=1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [31, 32, 33, 63, 64, 65, 96, 127, 128, 129, 160, 192, 255, 256, 257,
                               320, 383, 384, 385, 511, 512, 513, 768, 1023, 1024])
def test_every_width_and_its_edges(E, score):
    g = torch.Generator().manual_seed(E)
    logits = 2.0 * torch.randn(12, E, generator=g)
    bias = 0.1 * torch.randn(E, generator=g)
    for K in (1, 8, 17, min(E, 32)):
        check(logits, K, bias, score=score)
        check(logits, K, torch.zeros(E), score=score)
