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
