"""The operators around the MXFP4 routed experts on quantised tokens: experts
and mixture weights from router logits, rows of values to MXFP4 and back, and
products of MXFP4 tokens with MXFP4 weights, dense and routed.

Like the rest of the package this is the thin Python face of the C library
(header ``include/mxfp4el_quantized.h``): it checks and marshals arguments;
the work is done by the library's CUDA kernels on the current stream.

MXFP4 rows are two uint8 tensors, packed (..., I/32, 16) and scales (..., I/32),
as the experts' weights are.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _native

__all__ = ["route_experts", "quantize_mxfp4", "dequantize_mxfp4", "mxfp4_linear",
           "mxfp4_expert_linear_quantized"]

_DTYPES = {torch.float32: _native.DTYPE_F32, torch.bfloat16: _native.DTYPE_BF16}
_INDEX_DTYPES = {torch.int32: _native.INDEX_I32, torch.int64: _native.INDEX_I64}
_SCORES = {"softmax": _native.SCORE_SOFTMAX, "sigmoid": _native.SCORE_SIGMOID}
_U8, _I32, _F32 = torch.uint8, torch.int32, torch.float32

# The current stream's handle of a device by index (see attention.py).
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_empty = torch.empty


# As in attention.py: the calls are short next to what Python spends on them, so
# each writes its checks out once, and what it refuses is worked out only then.
def _call(f, name: str, index: int, *args) -> None:
    """One library call on device `index`, its current stream last."""
    if _current_device() == index:
        rc = f(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = f(*args, _raw_stream(index))
    if rc:
        _native.check(rc, name)


def _check_out(name: str, t: torch.Tensor, shape: tuple, dtype: torch.dtype, index: int) -> None:
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {tuple(shape)} {dtype} tensor on the "
                         "inputs' device")


def route_experts(logits: torch.Tensor, K: int, *, score: str = "softmax",
                  bias: torch.Tensor | None = None, groups: int = 1,
                  top_groups: int | None = None, group_best: int = 2, normalize: bool = True,
                  scaling: float = 1.0, selected_experts: torch.Tensor | None = None,
                  mixture_weights: torch.Tensor | None = None
                  ) -> tuple[torch.Tensor, torch.Tensor]:
    """(selected_experts (T, K) int32, mixture_weights (T, K) float32) of the
    router logits (T, E), float32 or bfloat16, rows of contiguous elements.

    Scores are the softmax over the experts or the sigmoid of each logit;
    ``bias`` (E) float32 is added for the choice alone. With ``groups`` > 1
    only the experts of the ``top_groups`` best groups (default: all) take
    part, a group's score being the sum of its ``group_best`` highest choices.
    The K highest are selected, highest first, ties to the lower index, as
    float64 scores rank them; their weights are their scores, normalised to
    sum to ``scaling`` or, without ``normalize``, times ``scaling``. Slots that
    NaN logits leave over get id -1 and weight 0. At most 1024 experts, 32
    groups and K = 32; fast up to some 16 picks. :func:`router_topk` computes the same
    without groups and for a sigmoid alone, and ranks by float32 choices, as the
    calls that route for themselves do. See mxfp4_route_experts in the C header.
    """
    shape, stride, dtype, index = logits.shape, logits.stride(), logits.dtype, logits.get_device()
    if index < 0 or dtype not in _DTYPES or len(shape) != 2:
        raise ValueError("logits must be a (T, E) float32 or bfloat16 CUDA tensor")
    T, E = shape
    if stride[1] != 1 and E > 1:
        raise ValueError("the rows of logits must be contiguous")
    if score not in _SCORES:
        raise ValueError("score must be 'softmax' or 'sigmoid'")
    if groups < 1 or E < 1 or E % groups:
        raise ValueError("groups must divide the number of experts")
    if top_groups is None:
        top_groups = groups
    if not 1 <= top_groups <= groups:
        raise ValueError("need 1 <= top_groups <= groups")
    if not 0 <= K <= top_groups * (E // groups):
        raise ValueError("K must be at most the experts of top_groups groups")
    if group_best != 2 and group_best != 1:
        raise ValueError("group_best must be 1 or 2")
    if bias is not None and (bias.dtype is not _F32 or bias.get_device() != index
                             or bias.shape != (E,) or not bias.is_contiguous()):
        raise ValueError("bias must be a contiguous (E,) float32 tensor on the logits' device")
    device = logits.device
    if selected_experts is None:
        selected_experts = _empty((T, K), dtype=_I32, device=device)
    else:
        _check_out("selected_experts", selected_experts, (T, K), _I32, index)
    if mixture_weights is None:
        mixture_weights = _empty((T, K), dtype=_F32, device=device)
    else:
        _check_out("mixture_weights", mixture_weights, (T, K), _F32, index)
    if T and K:
        _call(_native.load().mxfp4_route_experts, "route_experts", index,
              logits.data_ptr(), _DTYPES[dtype], stride[0],
              None if bias is None else bias.data_ptr(), T, E, K, _SCORES[score], groups,
              top_groups, group_best, 1 if normalize else 0, scaling,
              selected_experts.data_ptr(), mixture_weights.data_ptr())
    return selected_experts, mixture_weights


def quantize_mxfp4(x: torch.Tensor, packed: torch.Tensor | None = None,
                   scales: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """(packed (..., I/32, 16), scales (..., I/32)) uint8 of x (..., I), float32
    or bfloat16, I a multiple of 32.

    x may be a view whose rows of I contiguous elements lie evenly apart (a
    slice of a wider matrix). A group of 32 with largest magnitude a has the
    scale 2^(floor(log2 a) - 2); its values are rounded to the nearest E2M1
    number, ties to the even code, larger ones to 6. A group with an infinity
    or a NaN reads back as NaN. See mxfp4_quantize in the C header.
    """
    *lead, I = x.shape if x.dim() else (0,)
    dtype, index = x.dtype, x.get_device()
    if index < 0 or dtype not in _DTYPES or x.dim() == 0:
        raise ValueError("x must be a (..., I) float32 or bfloat16 CUDA tensor")
    if I == 0 or I & 31:
        raise ValueError("the last dimension must be a positive multiple of 32")
    if x.is_contiguous():
        rows, stride = x.numel() // I, I
    else:
        try:
            flat = x.view(-1, I) if x.dim() != 2 else x
        except RuntimeError:
            flat = None
        if flat is None or flat.stride(1) != 1 or (flat.shape[0] > 1 and flat.stride(0) < I):
            raise ValueError("the rows of x must be contiguous and evenly apart")
        rows, stride = flat.shape[0], flat.stride(0)
    G, device = I >> 5, x.device
    if packed is None:
        packed = _empty((*lead, G, 16), dtype=_U8, device=device)
    else:
        _check_out("packed", packed, (*lead, G, 16), _U8, index)
    if scales is None:
        scales = _empty((*lead, G), dtype=_U8, device=device)
    else:
        _check_out("scales", scales, (*lead, G), _U8, index)
    if rows:
        _call(_native.load().mxfp4_quantize, "quantize_mxfp4", index, x.data_ptr(),
              _DTYPES[dtype], stride, rows, I, packed.data_ptr(), scales.data_ptr())
    return packed, scales


def _mxfp4_rows(what: str, packed: torch.Tensor, scales: torch.Tensor, index: int) -> torch.Size:
    """The shape of packed; refuses anything but MXFP4 rows of device `index`
    that the library can read."""
    shape = packed.shape
    if packed.dtype is _U8 and scales.dtype is _U8 and len(shape) > 1 and shape[-1] == 16 \
            and shape[:-1] == scales.shape and shape[-2] and packed.get_device() == index \
            and scales.get_device() == index and index >= 0 and packed.is_contiguous() \
            and scales.is_contiguous():
        return shape
    if packed.dtype is not _U8 or scales.dtype is not _U8:
        raise TypeError(f"{what}: packed and scales must be uint8")
    if index < 0 or packed.get_device() != index or scales.get_device() != index:
        raise ValueError(f"{what}: packed and scales must be on one CUDA device with the rest")
    if not packed.is_contiguous() or not scales.is_contiguous():
        raise ValueError(f"{what}: packed and scales must be contiguous")
    raise ValueError(f"{what}: expected packed (..., I/32, 16) and scales (..., I/32)")


def dequantize_mxfp4(packed: torch.Tensor, scales: torch.Tensor,
                     dtype: torch.dtype = torch.bfloat16,
                     out: torch.Tensor | None = None) -> torch.Tensor:
    """The values (..., I) that MXFP4 rows packed (..., I/32, 16) and scales
    (..., I/32) stand for, float32 or bfloat16: exact in both. A scale byte of
    255 gives NaN. See mxfp4_dequantize in the C header."""
    index = packed.get_device()
    *lead, G, _ = _mxfp4_rows("dequantize_mxfp4", packed, scales, index)
    if dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {dtype}")
    I = 32 * G
    if out is None:
        out = _empty((*lead, I), dtype=dtype, device=packed.device)
    else:
        _check_out("out", out, (*lead, I), dtype, index)
    rows = packed.numel() // (16 * G)
    if rows:
        _call(_native.load().mxfp4_dequantize, "dequantize_mxfp4", index, packed.data_ptr(),
              scales.data_ptr(), rows, I, out.data_ptr(), _DTYPES[dtype])
    return out


# The scratch of a call depends on its sizes alone.
@functools.lru_cache(maxsize=4096)
def _workspace_bytes(name: str, *sizes: int) -> int:
    n = getattr(_native.load(), name)(*sizes)
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("sizes rejected by the library")
    return n


def mxfp4_linear(x_packed: torch.Tensor, x_scales: torch.Tensor, packed_weights: torch.Tensor,
                 scale_bytes: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
                 out: torch.Tensor | None = None) -> torch.Tensor:
    """out (T, O) = X W^T of MXFP4 tokens X (x_packed (T, I/32, 16), x_scales
    (T, I/32)) and MXFP4 weights W (packed_weights (O, I/32, 16), scale_bytes
    (O, I/32)), in float32 or bfloat16. Products are exact, sums float32. See
    mxfp4_linear in the C header."""
    index = x_packed.get_device()
    xs = _mxfp4_rows("tokens", x_packed, x_scales, index)
    ws = _mxfp4_rows("weights", packed_weights, scale_bytes, index)
    if len(xs) != 3 or len(ws) != 3 or xs[1] != ws[1]:
        raise ValueError("expected tokens (T, I/32, 16) and weights (O, I/32, 16)")
    if dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {dtype}")
    T, I, O = xs[0], 32 * xs[1], ws[0]
    if out is None:
        out = _empty((T, O), dtype=dtype, device=x_packed.device)
    else:
        _check_out("out", out, (T, O), dtype, index)
    if T and O:
        need = _workspace_bytes("mxfp4_linear_workspace_size", T, I, O)
        work = _empty(need, dtype=_U8, device=x_packed.device) if need else None
        _call(_native.load().mxfp4_linear, "mxfp4_linear", index, x_packed.data_ptr(),
              x_scales.data_ptr(), packed_weights.data_ptr(), scale_bytes.data_ptr(),
              out.data_ptr(), T, I, O, _DTYPES[dtype],
              None if work is None else work.data_ptr(), need)
    return out


def mxfp4_expert_linear_quantized(x_packed: torch.Tensor, x_scales: torch.Tensor,
                                  packed_weights: torch.Tensor, scale_bytes: torch.Tensor,
                                  selected_experts: torch.Tensor, mixture_weights: torch.Tensor,
                                  shared_output: torch.Tensor,
                                  out: torch.Tensor | None = None) -> torch.Tensor:
    """The routed expert linear on MXFP4 tokens: out[t] = shared_output[t] +
    sum_k mixture_weights[t, k] W_{selected_experts[t, k]} x_t.

    Tokens are x_packed (T, I/32, 16) and x_scales (T, I/32) uint8, as
    :func:`quantize_mxfp4` makes them; packed_weights (E, O, I/32, 16) and
    scale_bytes (E, O, I/32) uint8; selected_experts (T, K) int32 or int64;
    mixture_weights (T, K) float32; shared_output (T, O) float32 or bfloat16,
    whose dtype the result has. All contiguous, on one CUDA device. An expert
    id out of range contributes nothing (see ``device_errors``). See
    mxfp4_expert_linear_quantized in the C header.
    """
    sel, p, ys = selected_experts, mixture_weights, shared_output
    index = x_packed.get_device()
    xs = _mxfp4_rows("tokens", x_packed, x_scales, index)
    ws = _mxfp4_rows("weights", packed_weights, scale_bytes, index)
    if len(xs) != 3 or len(ws) != 4 or xs[1] != ws[2]:
        raise ValueError("expected tokens (T, I/32, 16) and weights (E, O, I/32, 16)")
    T, I, (E, O) = xs[0], 32 * xs[1], ws[:2]
    shape = sel.shape
    if len(shape) != 2 or shape[0] != T or p.shape != shape or ys.shape != (T, O):
        raise ValueError("routing or shared-output shape mismatch")
    if sel.dtype not in _INDEX_DTYPES or p.dtype is not _F32:
        raise TypeError("selected_experts must be int32 or int64, mixture_weights float32")
    dtype, K = ys.dtype, shape[1]
    if dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {dtype}")
    if sel.get_device() != index or p.get_device() != index or ys.get_device() != index:
        raise ValueError("routing and shared_output must be on the tokens' device")
    if not (sel.is_contiguous() and p.is_contiguous() and ys.is_contiguous()):
        raise ValueError("routing and shared_output must be contiguous")
    if out is None:
        out = torch.empty_like(ys)
    else:
        _check_out("out", out, (T, O), dtype, index)
    if T and O:
        need = _workspace_bytes("mxfp4_expert_linear_quantized_workspace_size", T, E, I, O, K)
        work = _empty(need, dtype=_U8, device=ys.device)
        _call(_native.load().mxfp4_expert_linear_quantized, "mxfp4_expert_linear_quantized",
              index, x_packed.data_ptr(), x_scales.data_ptr(), packed_weights.data_ptr(),
              scale_bytes.data_ptr(), sel.data_ptr(), p.data_ptr(), ys.data_ptr(),
              out.data_ptr(), T, E, I, O, K, _DTYPES[dtype], _INDEX_DTYPES[sel.dtype],
              work.data_ptr(), need)
    return out
