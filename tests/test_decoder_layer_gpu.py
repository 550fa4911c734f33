"""The operators together, as a decoder layer runs them (examples/decoder_layer.py)."""
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def _run(layer, x, splits, table):
    """Two sequences' tokens through the layer, in the given pieces of each:
    prompts or chunks in one call, single tokens as decode steps."""
    import mxfp4_routed_expert_route_gb300 as lib
    done = [0, 0]
    out = [[], []]
    for pieces in splits:
        lens = [done[b] + pieces[b] for b in range(2)]
        rows = torch.cat([x[b][done[b]:lens[b]] for b in range(2)])
        offsets = torch.tensor([0, pieces[0], sum(pieces)], dtype=torch.int32, device="cuda")
        seqs = lib.PagedSequences(table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                  None if pieces == (1, 1) else offsets)
        y = layer(rows, seqs)
        out[0].append(y[:pieces[0]])
        out[1].append(y[pieces[0]:])
        done = lens
    assert lib.page_errors() == 0 and lib.wait_timeouts() == 0
    return [torch.cat(o) for o in out]


@pytest.mark.parametrize("dtype,tol", [
    # Between the three orders the sums differ by rounding only. float32: the
    # expert projections are within 1e-5 of their sums of magnitudes, about 16
    # times the results here; three stages. bf16: attention and experts each
    # round their inputs and results to 2^-8, a few times over.
    (torch.float32, 5e-4), (torch.bfloat16, 3e-2)])
@pytest.mark.parametrize("window,sinks", [(None, 0), (24, 3)])
def test_prompts_chunks_and_steps_agree(dtype, tol, window, sinks):
    from decoder_layer import DecoderLayer
    layer = DecoderLayer(dtype=dtype, window=window, sinks=sinks, seed=5)
    g = torch.Generator(device="cuda").manual_seed(6)
    x = [torch.randn(n, 256, generator=g, device="cuda").to(dtype) for n in (45, 103)]
    table = torch.randperm(64, generator=g, device="cuda", dtype=torch.int32)[:32].view(2, 16)
    whole = _run(layer, x, [(45, 103)], table)
    chunks = _run(layer, x, [(20, 1), (0, 60), (25, 42)], table)
    steps = _run(layer, x, [(42, 100), (1, 1), (1, 1), (1, 1)], table)
    for other in (chunks, steps):
        for a, b in zip(whole, other):
            # A router tie that rounding decides the other way changes a token
            # wholly; most tokens must agree, and those that do to rounding.
            rel = (a.double() - b.double()).norm(dim=1) / a.double().norm(dim=1)
            agree = rel <= tol
            assert agree.float().mean() >= (1.0 if dtype == torch.float32 else 0.9), rel


def test_the_example_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "decoder_layer.py")],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.count("tokens") == 5
