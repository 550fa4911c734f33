"""Arguments and values at the edge of what the attention operators accept,
against the 64-bit forms of attention_ref.py."""
import pytest
import torch

import mxfp4_routed_expert_route_gb300 as lib
from test_attention_gpu import BF16, F32, call, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("sinks", [1 << 30, (1 << 31) - 64, (1 << 31) - 1, 1 << 40])
def test_every_first_token_stays_visible(dtype, dim, decode, sinks):
    # More first tokens than any length: the window hides nothing.
    lens = [100, 1550, 3000, 40, 1]
    d = make(lens, [1] * 5 if decode else [70, 33, 5, 40, 1], dim=dim, dtype=dtype, fill=float("nan"))
    check(d, decode, window=50, sinks=sinks)
    check(d, decode, window=2000, sinks=sinks)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("window", [(1 << 30) - 1, 1 << 30, (1 << 31) - 2, (1 << 31) - 1, 1 << 40])
def test_windows_past_every_length_hide_nothing(dtype, decode, window):
    # Rows with negative positions among them: they still see nothing.
    d = make([3, 40, 700], [1] * 3 if decode else [10, 60, 300], dtype=dtype, fill=float("nan"))
    got = check(d, decode, window=window, sinks=4)
    assert torch.equal(got, call(d, decode))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("decode", [True, False])
def test_lengths_near_the_end_of_32_bits_are_cut(dtype, decode):
    d = make([48, 31], [1, 1] if decode else [5, 31], dtype=dtype)
    d["table"] = d["table"][:, :3].contiguous()      # room for 48 keys
    want = call(d, decode, window=20, sinks=2)
    d["seq_lens"] = torch.tensor([(1 << 31) - 1, 31], dtype=torch.int32, device="cuda")
    lib.page_errors()
    assert torch.equal(call(d, decode, window=20, sinks=2), want)
    assert lib.page_errors() > 0
