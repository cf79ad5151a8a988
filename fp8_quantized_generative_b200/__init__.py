"""B200-native FP8 W8A8 linear layers (per-channel weights, per-token
dynamic activations, FP8 tensor-core GEMM with FP32 accumulation and a fused
dequantize + FP16 epilogue; dense and MoE grouped).

The compute runs in libfp8q.so (hand-written sm_100a kernels behind a C ABI,
include/fp8q.h).  This module only marshals torch tensors into that ABI:
PyTorch provides device memory and streams.  There is no CPU fallback; a
missing library raises ImportError at the first call.

    Xq, s_x = quantize_rows_dynamic(X)          # X fp16 [M,K] on cuda
    Wq, s_w = quantize_weight_per_channel(W)    # offline, W fp16 [N,K]
    Y = linear(Xq, s_x, Wq, s_w)                # fp16 [M,N]
    Y = moe_grouped_linear(Xq, s_x, offsets, Wq_e, s_w_e)

Variants from the pages: activations in E5M2 (quantize_rows_dynamic(X,
fmt="e5m2") with linear(..., x_fmt="e5m2")), per-tensor weight scales
(quantize_weight_per_tensor) and 128x128 block-scaled MoE expert weights
(quantize_weight_blockwise with moe_grouped_linear_blockscaled).

Around the linears, the rest of an FFN block: bias, activation and residual in
the linear's epilogue, the MoE router, and a whole MoE FFN for a few tokens.

    Y = linear_epilogue(Xq, s_x, Wq, s_w, bias=b, activation="gelu", residual=R)
    r = moe_route(logits, topk)                 # experts, weights, grouped row layout
    out = moe_layer(X, r.experts, r.weights, Wq_up, s_up, Wq_down, s_down, activation="silu", gated=True)
"""
from __future__ import annotations

import functools
from typing import NamedTuple

import torch

from . import _lib
from ._lib import Fp8qError, check, lib

__all__ = [
    "Fp8qError", "lib", "quantize_rows_dynamic", "quantize_weight_per_channel", "quantize_weight_per_tensor",
    "quantize_weight_blockwise", "linear", "moe_grouped_linear", "moe_grouped_linear_gather",
    "moe_grouped_linear_combine", "quantize_rows_dispatch", "quantized_linear_overlapped", "overlap_workspace",
    "moe_grouped_linear_blockscaled",
    "quantized_linear", "e4m3_encode_f32", "device_error", "set_gemm_tuning",
    "linear_epilogue", "MoeRoute", "moe_route", "moe_layer", "moe_layer_workspace",
]


def _fmt(name: str) -> int:
    try:
        return _lib.FORMATS[name]
    except KeyError:
        raise ValueError(f"unknown FP8 format {name!r} (e4m3 or e5m2)") from None


def _stream(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _need(t: torch.Tensor, dtype, name: str, ndim: int | None = None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must be {ndim}-D, got shape {tuple(t.shape)}")


def quantize_rows_dynamic(X: torch.Tensor, out: tuple | None = None, fmt: str = "e4m3"):
    """Per-token dynamic FP8 quantization: fp16 [M,K] -> (uint8 [M,K], fp32 [M]).
    fmt: "e4m3" (the path) or "e5m2" (the activation-format variant)."""
    _need(X, torch.float16, "X", 2)
    M, K = X.shape
    Xq, s = out if out is not None else (
        torch.empty((M, K), dtype=torch.uint8, device=X.device),
        torch.empty((M,), dtype=torch.float32, device=X.device))
    if fmt == "e4m3":
        check(_lib.fp8q_quantize_rows_dynamic(X.data_ptr(), M, K, Xq.data_ptr(), s.data_ptr(), _stream(X)),
              "fp8q_quantize_rows_dynamic")
    else:
        check(_lib.fp8q_quantize_rows_dynamic_fmt(X.data_ptr(), M, K, _fmt(fmt), Xq.data_ptr(), s.data_ptr(),
                                                  _stream(X)), "fp8q_quantize_rows_dynamic_fmt")
    return Xq, s


def quantize_rows_dispatch(X: torch.Tensor, token_rows: torch.Tensor, rows: int, out: tuple | None = None,
                           fmt: str = "e4m3"):
    """Per-token quantization of X fp16 [T,K] written to the expert-grouped
    rows: token t's codes and scale go to rows token_rows[t, j] (int32
    [T, topk], -1 = none) of the returned (uint8 [rows,K], fp32 [rows])."""
    _need(X, torch.float16, "X", 2)
    _need(token_rows, torch.int32, "token_rows", 2)
    T, K = X.shape
    if token_rows.shape[0] != T:
        raise ValueError("token_rows must be [T, topk]")
    Xq, s = out if out is not None else (
        torch.empty((rows, K), dtype=torch.uint8, device=X.device),
        torch.empty((rows,), dtype=torch.float32, device=X.device))
    check(_lib.fp8q_quantize_rows_dispatch(X.data_ptr(), T, K, _fmt(fmt), token_rows.data_ptr(), token_rows.shape[1],
                                           rows, Xq.data_ptr(), s.data_ptr(), _stream(X)),
          "fp8q_quantize_rows_dispatch")
    return Xq, s


def quantize_weight_per_channel(W: torch.Tensor, out: tuple | None = None):
    """Offline per-output-channel E4M3 quantization: fp16 [N,K] or [E,N,K]."""
    _need(W, torch.float16, "W")
    if W.dim() not in (2, 3):
        raise ValueError("W must be [N,K] or [E,N,K]")
    K = W.shape[-1]
    rows = W.numel() // K
    Wq, s = out if out is not None else (torch.empty(W.shape, dtype=torch.uint8, device=W.device),
                                         torch.empty(W.shape[:-1], dtype=torch.float32, device=W.device))
    check(_lib.fp8q_quantize_weight_per_channel(W.data_ptr(), rows, K, Wq.data_ptr(), s.data_ptr(), _stream(W)),
          "fp8q_quantize_weight_per_channel")
    return Wq, s


def quantize_weight_per_tensor(W: torch.Tensor):
    """Offline per-tensor E4M3 quantization of fp16 [N,K]: one scale for the
    matrix, returned replicated as fp32 [N] (the form linear() takes)."""
    _need(W, torch.float16, "W", 2)
    N, K = W.shape
    Wq = torch.empty((N, K), dtype=torch.uint8, device=W.device)
    s = torch.empty((N,), dtype=torch.float32, device=W.device)
    check(_lib.fp8q_quantize_weight_per_tensor(W.data_ptr(), N, K, Wq.data_ptr(), s.data_ptr(), _stream(W)),
          "fp8q_quantize_weight_per_tensor")
    return Wq, s


def linear(Xq: torch.Tensor, s_x: torch.Tensor, Wq: torch.Tensor, s_w: torch.Tensor,
           out: torch.Tensor | None = None, x_fmt: str = "e4m3") -> torch.Tensor:
    """FP8 W8A8 linear with fused dequantization: fp16 [M,N].  x_fmt: the
    format of the activation codes Xq ("e4m3" or "e5m2"); weights are E4M3."""
    _need(Xq, torch.uint8, "Xq", 2)
    _need(Wq, torch.uint8, "Wq", 2)
    _need(s_x, torch.float32, "s_x", 1)
    _need(s_w, torch.float32, "s_w", 1)
    M, K = Xq.shape
    N = Wq.shape[0]
    if Wq.shape[1] != K or s_x.shape[0] != M or s_w.shape[0] != N:
        raise ValueError("shape mismatch")
    Y = out if out is not None else torch.empty((M, N), dtype=torch.float16, device=Xq.device)
    if x_fmt == "e4m3":
        check(_lib.fp8q_linear(Xq.data_ptr(), s_x.data_ptr(), Wq.data_ptr(), s_w.data_ptr(), M, N, K, Y.data_ptr(),
                               _stream(Xq)), "fp8q_linear")
    else:
        check(_lib.fp8q_linear_fmt(Xq.data_ptr(), _fmt(x_fmt), s_x.data_ptr(), Wq.data_ptr(), s_w.data_ptr(), M, N, K,
                                   Y.data_ptr(), _stream(Xq)), "fp8q_linear_fmt")
    return Y


FUSED_MAX_ROWS = 64


def quantized_linear(X: torch.Tensor, Wq: torch.Tensor, s_w: torch.Tensor,
                     out: torch.Tensor | None = None, fused: bool = False) -> torch.Tensor:
    """fp16 activations in, fp16 out: per-token quantization + FP8 linear +
    dequantization.  fused=True runs one kernel (up to 64 rows, no workspace);
    otherwise the two steps through a workspace allocated here."""
    _need(X, torch.float16, "X", 2)
    _need(Wq, torch.uint8, "Wq", 2)
    _need(s_w, torch.float32, "s_w", 1)
    M, K = X.shape
    N = Wq.shape[0]
    if Wq.shape[1] != K or s_w.shape[0] != N:
        raise ValueError("shape mismatch")
    Y = out if out is not None else torch.empty((M, N), dtype=torch.float16, device=X.device)
    if fused and M <= FUSED_MAX_ROWS:
        st = _lib.fp8q_quantized_linear(X.data_ptr(), Wq.data_ptr(), s_w.data_ptr(), M, N, K, Y.data_ptr(), 0, 0,
                                        _stream(X))
        if st == _lib.FP8Q_OK:
            return Y
    Xq = torch.empty((M, K), dtype=torch.uint8, device=X.device)
    s_x = torch.empty((M,), dtype=torch.float32, device=X.device)
    check(_lib.fp8q_quantized_linear(X.data_ptr(), Wq.data_ptr(), s_w.data_ptr(), M, N, K, Y.data_ptr(),
                                     Xq.data_ptr(), s_x.data_ptr(), _stream(X)), "fp8q_quantized_linear")
    return Y


def overlap_workspace(M: int, K: int, device) -> tuple:
    """Workspace of quantized_linear_overlapped for M rows of K: (codes uint8
    [M,K], scales fp32 [M], sync words int32, zero-filled).  Reusable across
    calls that do not overlap on the GPU."""
    words = int(_lib.fp8q_overlap_sync_words(M))
    return (torch.empty((M, K), dtype=torch.uint8, device=device),
            torch.empty((M,), dtype=torch.float32, device=device),
            torch.zeros((words,), dtype=torch.int32, device=device))


def quantized_linear_overlapped(X: torch.Tensor, Wq: torch.Tensor, s_w: torch.Tensor,
                                workspace: tuple | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """quantized_linear as one kernel for M > 128: the GEMM's own warps
    quantize the rows while its tensor cores start on the rows already done.
    The workspace (see overlap_workspace) then holds the codes and scales."""
    _need(X, torch.float16, "X", 2)
    _need(Wq, torch.uint8, "Wq", 2)
    _need(s_w, torch.float32, "s_w", 1)
    M, K = X.shape
    N = Wq.shape[0]
    if Wq.shape[1] != K or s_w.shape[0] != N:
        raise ValueError("shape mismatch")
    Xq, s_x, sync = workspace if workspace is not None else overlap_workspace(M, K, X.device)
    if tuple(Xq.shape) != (M, K) or s_x.shape[0] != M or sync.numel() < _lib.fp8q_overlap_sync_words(M):
        raise ValueError("workspace does not fit this X")
    Y = out if out is not None else torch.empty((M, N), dtype=torch.float16, device=X.device)
    check(_lib.fp8q_quantized_linear_overlapped(X.data_ptr(), Wq.data_ptr(), s_w.data_ptr(), M, N, K, Y.data_ptr(),
                                                Xq.data_ptr(), s_x.data_ptr(), sync.data_ptr(), _stream(X)),
          "fp8q_quantized_linear_overlapped")
    return Y


def moe_grouped_linear(Xq: torch.Tensor, s_x: torch.Tensor, offsets: torch.Tensor, Wq: torch.Tensor,
                       s_w: torch.Tensor, out: torch.Tensor | None = None, x_fmt: str = "e4m3") -> torch.Tensor:
    """Expert-grouped FP8 linear.  offsets: int32 [E+1] on the device; x_fmt
    the format of the activation codes ("e4m3" or "e5m2")."""
    _need(Xq, torch.uint8, "Xq", 2)
    _need(s_x, torch.float32, "s_x", 1)
    _need(offsets, torch.int32, "offsets", 1)
    _need(Wq, torch.uint8, "Wq", 3)
    _need(s_w, torch.float32, "s_w", 2)
    rows, K = Xq.shape
    E, N, K2 = Wq.shape
    if K2 != K or offsets.shape[0] != E + 1 or tuple(s_w.shape) != (E, N) or s_x.shape[0] != rows:
        raise ValueError("shape mismatch")
    Y = out if out is not None else torch.empty((rows, N), dtype=torch.float16, device=Xq.device)
    if x_fmt == "e4m3":
        check(_lib.fp8q_moe_grouped_linear(Xq.data_ptr(), s_x.data_ptr(), offsets.data_ptr(), E, rows, Wq.data_ptr(),
                                           s_w.data_ptr(), N, K, Y.data_ptr(), _stream(Xq)),
              "fp8q_moe_grouped_linear")
    else:
        check(_lib.fp8q_moe_grouped_linear_fmt(Xq.data_ptr(), _fmt(x_fmt), s_x.data_ptr(), offsets.data_ptr(), E, rows,
                                               Wq.data_ptr(), s_w.data_ptr(), N, K, Y.data_ptr(), _stream(Xq)),
              "fp8q_moe_grouped_linear_fmt")
    return Y


def moe_grouped_linear_gather(Xq_tok: torch.Tensor, s_x_tok: torch.Tensor, row_token: torch.Tensor,
                              offsets: torch.Tensor, Wq: torch.Tensor, s_w: torch.Tensor,
                              out: torch.Tensor | None = None) -> torch.Tensor:
    """Expert-grouped FP8 linear whose row r reads token row_token[r] of the
    per-token codes Xq_tok [T,K] (scales s_x_tok [T]); rows in expert order
    (offsets int32 [E+1]); returns fp16 [len(row_token), N]."""
    _need(Xq_tok, torch.uint8, "Xq_tok", 2)
    _need(s_x_tok, torch.float32, "s_x_tok", 1)
    _need(row_token, torch.int32, "row_token", 1)
    _need(offsets, torch.int32, "offsets", 1)
    _need(Wq, torch.uint8, "Wq", 3)
    _need(s_w, torch.float32, "s_w", 2)
    T, K = Xq_tok.shape
    rows = row_token.shape[0]
    E, N, K2 = Wq.shape
    if K2 != K or offsets.shape[0] != E + 1 or tuple(s_w.shape) != (E, N) or s_x_tok.shape[0] != T:
        raise ValueError("shape mismatch")
    Y = out if out is not None else torch.empty((rows, N), dtype=torch.float16, device=Xq_tok.device)
    check(_lib.fp8q_moe_grouped_linear_gather(Xq_tok.data_ptr(), s_x_tok.data_ptr(), T, row_token.data_ptr(),
                                              offsets.data_ptr(), E, rows, Wq.data_ptr(), s_w.data_ptr(), N, K,
                                              Y.data_ptr(), _stream(Xq_tok)), "fp8q_moe_grouped_linear_gather")
    return Y


def moe_grouped_linear_combine(Xq: torch.Tensor, s_x: torch.Tensor, offsets: torch.Tensor, Wq: torch.Tensor,
                               s_w: torch.Tensor, row_token: torch.Tensor, row_weight: torch.Tensor, tokens: int,
                               out: torch.Tensor | None = None) -> torch.Tensor:
    """Expert-grouped FP8 linear whose row r is weighted by row_weight[r] and
    added (fp16) into row row_token[r] of the [tokens, N] output (the MoE
    down projection with the top-k combine)."""
    _need(Xq, torch.uint8, "Xq", 2)
    _need(s_x, torch.float32, "s_x", 1)
    _need(offsets, torch.int32, "offsets", 1)
    _need(Wq, torch.uint8, "Wq", 3)
    _need(s_w, torch.float32, "s_w", 2)
    _need(row_token, torch.int32, "row_token", 1)
    _need(row_weight, torch.float32, "row_weight", 1)
    rows, K = Xq.shape
    E, N, K2 = Wq.shape
    if (K2 != K or offsets.shape[0] != E + 1 or tuple(s_w.shape) != (E, N) or s_x.shape[0] != rows
            or row_token.shape[0] != rows or row_weight.shape[0] != rows):
        raise ValueError("shape mismatch")
    Y = out if out is not None else torch.empty((tokens, N), dtype=torch.float16, device=Xq.device)
    check(_lib.fp8q_moe_grouped_linear_combine(Xq.data_ptr(), s_x.data_ptr(), offsets.data_ptr(), E, rows,
                                               Wq.data_ptr(), s_w.data_ptr(), N, K, row_token.data_ptr(),
                                               row_weight.data_ptr(), tokens, Y.data_ptr(), _stream(Xq)),
          "fp8q_moe_grouped_linear_combine")
    return Y


BLOCK = 128


def quantize_weight_blockwise(W: torch.Tensor):
    """Offline 128x128 block-wise E4M3 quantization: fp16 [N,K] or [E,N,K] ->
    (uint8 same shape, fp32 scales [..., ceil(N/128), ceil(K/128)])."""
    _need(W, torch.float16, "W")
    if W.dim() not in (2, 3):
        raise ValueError("W must be [N,K] or [E,N,K]")
    E = W.shape[0] if W.dim() == 3 else 1
    N, K = W.shape[-2], W.shape[-1]
    Wq = torch.empty(W.shape, dtype=torch.uint8, device=W.device)
    s = torch.empty(W.shape[:-2] + (-(-N // BLOCK), -(-K // BLOCK)), dtype=torch.float32, device=W.device)
    check(_lib.fp8q_quantize_weight_blockwise(W.data_ptr(), E, N, K, Wq.data_ptr(), s.data_ptr(), _stream(W)),
          "fp8q_quantize_weight_blockwise")
    return Wq, s


def moe_grouped_linear_blockscaled(Xq: torch.Tensor, s_x: torch.Tensor, offsets: torch.Tensor, Wq: torch.Tensor,
                                   s_wb: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """Expert-grouped FP8 linear with 128x128 block-scaled expert weights
    (Wq [E,N,K] and s_wb [E, ceil(N/128), ceil(K/128)] from
    quantize_weight_blockwise); per-token activation scales."""
    _need(Xq, torch.uint8, "Xq", 2)
    _need(s_x, torch.float32, "s_x", 1)
    _need(offsets, torch.int32, "offsets", 1)
    _need(Wq, torch.uint8, "Wq", 3)
    _need(s_wb, torch.float32, "s_wb", 3)
    rows, K = Xq.shape
    E, N, K2 = Wq.shape
    if (K2 != K or offsets.shape[0] != E + 1 or s_x.shape[0] != rows
            or tuple(s_wb.shape) != (E, -(-N // BLOCK), -(-K // BLOCK))):
        raise ValueError("shape mismatch")
    Y = out if out is not None else torch.empty((rows, N), dtype=torch.float16, device=Xq.device)
    check(_lib.fp8q_moe_grouped_linear_blockscaled(Xq.data_ptr(), s_x.data_ptr(), offsets.data_ptr(), E, rows,
                                                   Wq.data_ptr(), s_wb.data_ptr(), N, K, Y.data_ptr(), _stream(Xq)),
          "fp8q_moe_grouped_linear_blockscaled")
    return Y


def _act(name) -> int:
    try:
        return _lib.ACTIVATIONS[name]
    except (KeyError, TypeError):
        raise ValueError(f"unknown activation {name!r} (none, relu, gelu, gelu_tanh or silu)") from None


# The FFN operators below serve single tokens, where a call's host time counts:
# arguments pass through one plain expression (what it refuses, _refuse explains),
# the stream handle is read without building a Stream object, and sizes that
# the library computes are remembered.

_U8, _F16, _F32, _I32 = torch.uint8, torch.float16, torch.float32, torch.int32
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _refuse(**args) -> None:
    """Raise for the first argument that is not a contiguous CUDA tensor of its
    dtype and rank, or that lies on another device than the first one; name =
    (tensor, dtype, rank)."""
    first = None
    for name, (t, dtype, ndim) in args.items():
        _need(t, dtype, name, ndim)
        first = t if first is None else first
        if t.device != first.device:
            raise ValueError(f"{name} is on {t.device}, not on {first.device}")
    raise ValueError("shape mismatch")


def _extra(t: torch.Tensor, dtype, shape: tuple, dev: int, name: str, kind: str) -> int:
    """Address of an optional argument, which must have this exact shape; 0 for None."""
    if t is None:
        return 0
    if isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dtype and t.get_device() == dev \
            and t.is_contiguous():
        return t.data_ptr()
    _need(t, dtype, name, len(shape))
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")
    raise ValueError(f"{name} must be {kind}")


def linear_epilogue(Xq: torch.Tensor, s_x: torch.Tensor, Wq: torch.Tensor, s_w: torch.Tensor,
                    bias: torch.Tensor | None = None, activation: str | None = None,
                    residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
                    x_fmt: str = "e4m3") -> torch.Tensor:
    """linear() with bias, activation and residual in its epilogue:
    fp16(act(linear + bias) + residual), computed in fp32 and rounded once.
    bias fp16 [N]; activation "none", "relu", "gelu", "gelu_tanh" or "silu";
    residual fp16 [M,N], which may be `out` itself."""
    act = _act(activation)
    fmt = _fmt(x_fmt)
    try:
        dev = Xq.get_device()
        (M, K), (N, K2), (M2,), (N2,) = Xq.shape, Wq.shape, s_x.shape, s_w.shape
        fits = (K2 == K and M2 == M and N2 == N and dev >= 0 and Xq.dtype is _U8 and Wq.dtype is _U8
                and s_x.dtype is _F32 and s_w.dtype is _F32 and Wq.get_device() == dev and s_x.get_device() == dev
                and s_w.get_device() == dev and Xq.is_contiguous() and Wq.is_contiguous() and s_x.is_contiguous()
                and s_w.is_contiguous())
    except (AttributeError, ValueError):
        fits = False
    if not fits:
        _refuse(Xq=(Xq, _U8, 2), Wq=(Wq, _U8, 2), s_x=(s_x, _F32, 1), s_w=(s_w, _F32, 1))
    b = _extra(bias, _F16, (N,), dev, "bias", "[N]")
    r = _extra(residual, _F16, (M, N), dev, "residual", "[M,N]")
    y = _extra(out, _F16, (M, N), dev, "out", "[M,N]")
    if dev != torch.cuda.current_device():   # the library launches on the current device
        with torch.cuda.device(dev):
            return linear_epilogue(Xq, s_x, Wq, s_w, bias, activation, residual, out, x_fmt)
    if out is None:
        out = torch.empty(M, N, dtype=_F16, device=Xq.device)
        y = out.data_ptr()
    check(lib().fp8q_linear_epilogue(Xq.data_ptr(), fmt, s_x.data_ptr(), Wq.data_ptr(), s_w.data_ptr(), M, N, K, b, act,
                                     r, y, _raw_stream(dev)), "fp8q_linear_epilogue")
    return out


class MoeRoute(NamedTuple):
    """What moe_route returns; all on the device, T tokens, E experts, rows = T * topk."""
    experts: torch.Tensor      # int32 [T, topk], best first
    weights: torch.Tensor      # fp32 [T, topk]
    offsets: torch.Tensor      # int32 [E+1]: grouped rows of expert e are offsets[e] .. offsets[e+1]-1
    row_token: torch.Tensor    # int32 [rows]
    row_weight: torch.Tensor   # fp32 [rows]
    token_rows: torch.Tensor   # int32 [T, topk]: the grouped row of each (token, choice)


@functools.lru_cache(maxsize=1024)
def _route_workspace_words(T: int, E: int) -> int:
    return int(_lib.fp8q_moe_route_workspace_words(T, E))


def moe_route(logits: torch.Tensor, topk: int, renormalize: bool = True) -> MoeRoute:
    """MoE router on the device: the topk experts of each token from fp16 gate
    logits [T,E] (ties to the lower expert), their softmax weights (over the
    chosen logits, or over all with renormalize=False), and the expert-grouped
    rows in the form that quantize_rows_dispatch (token_rows), the grouped
    linears (offsets), the combine (row_token, row_weight) and moe_layer
    (experts, weights) read."""
    _need(logits, _F16, "logits", 2)
    dev = logits.get_device()
    T, E = logits.shape
    if not 1 <= topk <= min(8, E):
        raise ValueError("topk must be in [1, min(8, E)]")
    if dev != torch.cuda.current_device():   # the library launches on the current device
        with torch.cuda.device(dev):
            return moe_route(logits, topk, renormalize)
    # one allocation for all outputs and the workspace
    rows = T * topk
    words = _route_workspace_words(T, E)
    i32 = torch.empty(5 * rows + E + 1 + words, dtype=_I32, device=logits.device)
    base, step = i32.data_ptr(), 4 * rows
    check(lib().fp8q_moe_route(logits.data_ptr(), T, E, topk, 1 if renormalize else 0, base, base + step,
                               base + 5 * step, base + 2 * step, base + 3 * step, base + 4 * step,
                               base + 5 * step + 4 * (E + 1) if words else 0, _raw_stream(dev)), "fp8q_moe_route")
    f32 = i32.view(_F32)
    shape, strides = (T, topk), (topk, 1)
    return MoeRoute(i32.as_strided(shape, strides, 0), f32.as_strided(shape, strides, rows),
                    i32.as_strided((E + 1,), (1,), 5 * rows), i32.as_strided((rows,), (1,), 2 * rows),
                    f32.as_strided((rows,), (1,), 3 * rows), i32.as_strided(shape, strides, 4 * rows))


@functools.lru_cache(maxsize=1024)
def _layer_workspace_bytes(T: int, topk: int, F: int, N: int) -> int:
    return int(_lib.fp8q_moe_layer_workspace_bytes(T, topk, F, N))


def moe_layer_workspace(T: int, topk: int, F: int, N: int, device) -> torch.Tensor:
    """Workspace of moe_layer for up to T tokens (uint8); reusable across calls
    that do not overlap on the GPU."""
    return torch.empty(_layer_workspace_bytes(T, topk, F, N), dtype=torch.uint8, device=device)


def moe_layer(X: torch.Tensor, experts: torch.Tensor, weights: torch.Tensor, Wq_up: torch.Tensor, s_up: torch.Tensor,
              Wq_down: torch.Tensor, s_down: torch.Tensor, activation: str | None = "silu", gated: bool = False,
              residual: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """A whole MoE FFN for a few tokens (up to 128): X fp16 [T,K] and the
    router's experts int32 / weights fp32 [T,topk] (-1: no expert) in, fp16
    [T,N] out.  Wq_up uint8 [E,F,K], or [E,2F,K] with gated=True (rows 0..F-1
    are activated and multiply rows F..2F-1), Wq_down uint8 [E,N,F], with
    per-channel scales s_up, s_down from quantize_weight_per_channel; residual
    fp16 [T,N] is added (it may be `out` itself).  Larger batches, and batches with
    more than about ten rows an expert, where they are faster: moe_route and
    the grouped linears, with the activation applied to the up projection's
    output (they have none)."""
    act = _act(activation)
    try:
        dev = X.get_device()
        (T, K), (T2, topk), (E, up, K2), (E2, N, F) = X.shape, experts.shape, Wq_up.shape, Wq_down.shape
        fits = (T2 == T and K2 == K and E2 == E and up == (2 * F if gated else F) and weights.shape == (T, topk)
                and s_up.shape == (E, up) and s_down.shape == (E, N) and dev >= 0 and X.dtype is _F16
                and experts.dtype is _I32 and weights.dtype is _F32 and Wq_up.dtype is _U8 and s_up.dtype is _F32
                and Wq_down.dtype is _U8 and s_down.dtype is _F32 and experts.get_device() == dev
                and weights.get_device() == dev and Wq_up.get_device() == dev and s_up.get_device() == dev
                and Wq_down.get_device() == dev and s_down.get_device() == dev and X.is_contiguous()
                and experts.is_contiguous() and weights.is_contiguous() and Wq_up.is_contiguous()
                and s_up.is_contiguous() and Wq_down.is_contiguous() and s_down.is_contiguous())
    except (AttributeError, ValueError):
        fits = False
    if not fits:
        _refuse(X=(X, _F16, 2), experts=(experts, _I32, 2), weights=(weights, _F32, 2), Wq_up=(Wq_up, _U8, 3),
                s_up=(s_up, _F32, 2), Wq_down=(Wq_down, _U8, 3), s_down=(s_down, _F32, 2))
    r = _extra(residual, _F16, (T, N), dev, "residual", "[T,N]")
    y = _extra(out, _F16, (T, N), dev, "out", "[T,N]")
    need = _layer_workspace_bytes(T, topk, F, N)
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or workspace.get_device() != dev or workspace.dtype is not _U8 \
                or not workspace.is_contiguous():
            _refuse(X=(X, _F16, 2), workspace=(workspace, _U8, None))
        if workspace.numel() < need:
            raise ValueError("workspace does not fit this call")
    if dev != torch.cuda.current_device():   # the library launches on the current device
        with torch.cuda.device(dev):
            return moe_layer(X, experts, weights, Wq_up, s_up, Wq_down, s_down, activation, gated, residual, workspace,
                             out)
    device = X.device
    if out is None:
        out = torch.empty(T, N, dtype=_F16, device=device)
        y = out.data_ptr()
    if workspace is None:
        workspace = torch.empty(need, dtype=_U8, device=device)
    check(lib().fp8q_moe_layer(X.data_ptr(), T, experts.data_ptr(), weights.data_ptr(), topk, E, Wq_up.data_ptr(),
                               s_up.data_ptr(), Wq_down.data_ptr(), s_down.data_ptr(), K, F, N, act, 1 if gated else 0,
                               r, y, workspace.data_ptr(), _raw_stream(dev)), "fp8q_moe_layer")
    return out


def e4m3_encode_f32(x: torch.Tensor) -> torch.Tensor:
    """The device E4M3 cast alone (diagnostic): fp32 -> uint8 codes."""
    _need(x, torch.float32, "x")
    out = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    check(_lib.fp8q_e4m3_encode_f32(x.data_ptr(), x.numel(), out.data_ptr(), _stream(x)), "fp8q_e4m3_encode_f32")
    return out


def set_gemm_tuning(kernel_family: int = 0, tile_n: int = 0, ksplit: int = 0) -> None:
    """Override the dense-linear kernel choice (0 = automatic; see include/fp8q.h)."""
    check(_lib.fp8q_set_gemm_tuning(kernel_family, tile_n, ksplit), "fp8q_set_gemm_tuning")


def device_error(device=None) -> int:
    """Synchronize the current stream and return (and clear) the device error word."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    st, flags = _lib.fp8q_device_error(torch.cuda.current_stream(dev).cuda_stream)
    if st not in (_lib.FP8Q_OK, _lib.FP8Q_ERR_TIMEOUT, _lib.FP8Q_ERR_DEVICE_CHECK):
        check(st, "fp8q_device_error")
    return flags
