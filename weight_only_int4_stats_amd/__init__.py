"""AWQ W4A16 hot path on AMD Instinct MI355X (gfx950).

Thin Python binding of the C ABI declared in include/awq.h.  Each function has
the name of the C entry point it calls and only marshals arguments: torch
provides device memory (outputs and workspaces are allocated with torch when
the caller does not pass them) and the current HIP stream; every step of the
computation runs in the library's HIP kernels.  There is no CPU fallback: the
functions raise if the library is missing or a tensor is not on the GPU.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _abi
from ._abi import (AWQ_ACT_GELU, AWQ_ACT_GELU_TANH, AWQ_ACT_NONE, AWQ_ACT_RELU, AWQ_ACT_SILU, AWQ_ACT_SWIGLU,  # noqa: F401
                   AWQ_BF16, AWQ_F16, AWQ_F32, AWQ_GROUP, AWQ_OP_ACT_STATS, AWQ_OP_BALANCE_LOSS,
                   AWQ_OP_BIAS_ACT_BACKWARD, AWQ_OP_GEMM_DX, AWQ_OP_LAYER_NORM_BACKWARD, AWQ_OP_LINEAR,
                   AWQ_OP_EXPERTS_DOWN, AWQ_OP_EXPERTS_UP, AWQ_OP_GEMM, AWQ_OP_LORA, AWQ_OP_QUANTIZE,
                   AWQ_OP_SEARCH, AWQ_SCORE_SIGMOID, AWQ_SCORE_SOFTMAX, AwqError, lib)

__all__ = ["awq_act_stats", "awq_search_scales", "awq_search_scales_ex", "awq_quantize_pack", "awq_quantize_codes",
           "awq_w4a16_gemm", "awq_w4a16_gemm_noalloc", "awq_read_stream", "awq_fold_scales", "awq_salient_channels", "awq_workspace_bytes",
           "awq_route_experts", "awq_w4a16_experts_up", "awq_w4a16_experts_down", "awq_lora_add",
           "awq_w4a16_linear", "awq_bias_act_backward", "awq_w4a16_gemm_dx", "awq_layer_norm", "awq_layer_norm_backward",
           "awq_balance_loss", "awq_balance_loss_backward", "AwqError", "lib"]

_DT = {torch.float16: AWQ_F16, torch.bfloat16: AWQ_BF16, torch.float32: AWQ_F32}


def _dev(t: torch.Tensor, name: str) -> None:
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError(f"{name} must be a tensor on the GPU")


def _ptr(t: torch.Tensor | None) -> ctypes.c_void_p | None:
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device: torch.device, stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _rows(x: torch.Tensor, name: str) -> tuple[int, int, int]:
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError(f"{name} must be 2-D with unit column stride")
    return x.shape[0], x.shape[1], x.stride(0)


def _workspace(nbytes: int, device, ws: torch.Tensor | None) -> tuple[torch.Tensor | None, int]:
    if nbytes == 0:
        return ws, 0 if ws is None else ws.numel() * ws.element_size()
    if ws is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return ws, ws.numel() * ws.element_size()


def awq_workspace_bytes(op: int, M: int = 0, N: int = 0, K: int = 0, T: int = 0, n_alpha: int = 0) -> int:
    return int(lib().awq_workspace_bytes(op, M, N, K, T, n_alpha))


def awq_act_stats(x: torch.Tensor, mean_abs: torch.Tensor | None = None,
                  ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """mean |x[:, j]| over rows, float32 [K]."""
    _dev(x, "x")
    T, K, ldx = _rows(x, "x")
    if mean_abs is None:
        mean_abs = torch.empty(K, dtype=torch.float32, device=x.device)
    ws, wsb = _workspace(awq_workspace_bytes(AWQ_OP_ACT_STATS, 0, 0, K, T, 0), x.device, ws)
    st = lib().awq_act_stats(_ptr(x), _DT.get(x.dtype, -1), T, K, ldx, _ptr(mean_abs), _ptr(ws),
                             wsb, _stream(x.device, stream))
    _abi.check("awq_act_stats", st)
    return mean_abs


def awq_search_scales(w: torch.Tensor, x_calib: torch.Tensor, mean_abs: torch.Tensor,
                      alphas: torch.Tensor, group_size: int = AWQ_GROUP,
                      s_out: torch.Tensor | None = None, inv_s_out: torch.Tensor | None = None,
                      loss_out: torch.Tensor | None = None, best_idx_out: torch.Tensor | None = None,
                      ws: torch.Tensor | None = None, stream=None, *, bits: int = 4,
                      symmetric: bool = False, kept: torch.Tensor | None = None):
    """Returns (s [K] f32, inv_s [K] f32, losses [n] f64, best index int32 [1]).
    With the defaults this calls awq_search_scales (the 4-bit asymmetric grid);
    bits / symmetric (another grid) or kept (uint8 [K]: channels kept in
    16-bit, the mixed-precision baseline) call awq_search_scales_ex."""
    ex = bits != 4 or bool(symmetric) or kept is not None
    return _search(w, x_calib, mean_abs, alphas, group_size, s_out, inv_s_out, loss_out,
                   best_idx_out, ws, stream, (bits, symmetric, kept) if ex else None)


def awq_search_scales_ex(w: torch.Tensor, x_calib: torch.Tensor, mean_abs: torch.Tensor,
                         alphas: torch.Tensor, group_size: int = AWQ_GROUP, bits: int = 4,
                         symmetric: bool = False, kept: torch.Tensor | None = None,
                         s_out: torch.Tensor | None = None, inv_s_out: torch.Tensor | None = None,
                         loss_out: torch.Tensor | None = None,
                         best_idx_out: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                         stream=None):
    """awq_search_scales_ex: the search under the grid (bits, symmetric) with
    the channels marked in kept (uint8 [K] or None) left in 16-bit."""
    return _search(w, x_calib, mean_abs, alphas, group_size, s_out, inv_s_out, loss_out,
                   best_idx_out, ws, stream, (bits, symmetric, kept))


def _search(w, x_calib, mean_abs, alphas, group_size, s_out, inv_s_out, loss_out, best_idx_out,
            ws, stream, variant):
    for t, n in ((w, "w"), (x_calib, "x_calib"), (mean_abs, "mean_abs"), (alphas, "alphas")):
        _dev(t, n)
    if not w.is_contiguous() or w.dim() != 2:
        raise ValueError("w must be a contiguous [N, K] tensor")
    if alphas.dtype != torch.float64:
        raise ValueError("alphas must be float64")
    N, K = w.shape
    T, Kx, ldx = _rows(x_calib, "x_calib")
    if Kx != K or x_calib.dtype != w.dtype:
        raise ValueError("x_calib must be [T, K] with w's dtype")
    n_alpha = alphas.numel()
    dev = w.device
    s_out = torch.empty(K, dtype=torch.float32, device=dev) if s_out is None else s_out
    inv_s_out = torch.empty(K, dtype=torch.float32, device=dev) if inv_s_out is None else inv_s_out
    loss_out = torch.empty(n_alpha, dtype=torch.float64, device=dev) if loss_out is None else loss_out
    best_idx_out = torch.empty(1, dtype=torch.int32, device=dev) if best_idx_out is None else best_idx_out
    ws, wsb = _workspace(awq_workspace_bytes(AWQ_OP_SEARCH, 0, N, K, T, n_alpha), dev, ws)
    head = (_ptr(w), _DT.get(w.dtype, -1), N, K, _ptr(x_calib), T, ldx, _ptr(mean_abs),
            _ptr(alphas), n_alpha, group_size)
    tail = (_ptr(s_out), _ptr(inv_s_out), _ptr(loss_out), _ptr(best_idx_out), _ptr(ws), wsb,
            _stream(dev, stream))
    if variant is None:
        st = lib().awq_search_scales(*head, *tail)
        _abi.check("awq_search_scales", st)
    else:
        bits, symmetric, kept = variant
        st = lib().awq_search_scales_ex(*head, bits, int(bool(symmetric)), _ptr(kept), *tail)
        _abi.check("awq_search_scales_ex", st)
    return s_out, inv_s_out, loss_out, best_idx_out


def awq_quantize_pack(w: torch.Tensor, s: torch.Tensor | None = None, group_size: int = AWQ_GROUP,
                      qweight: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                      zeros: torch.Tensor | None = None, scales_f32_dbg: torch.Tensor | None = None,
                      stream=None):
    """Returns (qweight int32 [N, K/8], scales fp16 [N, K/g], zeros uint8 [N, K/g])."""
    _dev(w, "w")
    if not w.is_contiguous() or w.dim() != 2:
        raise ValueError("w must be a contiguous [N, K] tensor")
    N, K = w.shape
    dev = w.device
    G = K // group_size if group_size > 0 else 0
    qweight = torch.empty((N, K // 8), dtype=torch.int32, device=dev) if qweight is None else qweight
    scales = torch.empty((N, G), dtype=torch.float16, device=dev) if scales is None else scales
    zeros = torch.empty((N, G), dtype=torch.uint8, device=dev) if zeros is None else zeros
    st = lib().awq_quantize_pack(_ptr(w), _DT.get(w.dtype, -1), N, K, _ptr(s), group_size,
                                 _ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(scales_f32_dbg),
                                 _stream(dev, stream))
    _abi.check("awq_quantize_pack", st)
    return qweight, scales, zeros


def awq_quantize_codes(w: torch.Tensor, s: torch.Tensor | None = None, group_size: int = AWQ_GROUP,
                       bits: int = 4, symmetric: bool = False, codes: torch.Tensor | None = None,
                       scales: torch.Tensor | None = None, zeros: torch.Tensor | None = None,
                       stream=None):
    """Returns (codes uint8 [N, K], scales fp16 [N, K/g], zeros uint8 [N, K/g])."""
    _dev(w, "w")
    if not w.is_contiguous() or w.dim() != 2:
        raise ValueError("w must be a contiguous [N, K] tensor")
    N, K = w.shape
    dev = w.device
    G = K // group_size if group_size > 0 else 0
    codes = torch.empty((N, K), dtype=torch.uint8, device=dev) if codes is None else codes
    scales = torch.empty((N, G), dtype=torch.float16, device=dev) if scales is None else scales
    zeros = torch.empty((N, G), dtype=torch.uint8, device=dev) if zeros is None else zeros
    st = lib().awq_quantize_codes(_ptr(w), _DT.get(w.dtype, -1), N, K, _ptr(s), group_size, bits,
                                  int(bool(symmetric)), _ptr(codes), _ptr(scales), _ptr(zeros),
                                  _stream(dev, stream))
    _abi.check("awq_quantize_codes", st)
    return codes, scales, zeros


def awq_salient_channels(mean_abs: torch.Tensor, n_keep: int, kept: torch.Tensor | None = None,
                         stream=None) -> torch.Tensor:
    """uint8 [K]: 1 for the n_keep channels of largest mean |x| (ties: lower index)."""
    _dev(mean_abs, "mean_abs")
    if mean_abs.dtype != torch.float32 or mean_abs.dim() != 1 or not mean_abs.is_contiguous():
        raise ValueError("mean_abs must be a contiguous float32 vector")
    K = mean_abs.numel()
    kept = torch.empty(K, dtype=torch.uint8, device=mean_abs.device) if kept is None else kept
    st = lib().awq_salient_channels(_ptr(mean_abs), K, n_keep, _ptr(kept), _stream(mean_abs.device, stream))
    _abi.check("awq_salient_channels", st)
    return kept


def awq_w4a16_gemm(x: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor,
                   zeros: torch.Tensor, inv_s: torch.Tensor | None = None,
                   out_dtype: torch.dtype | None = None, y: torch.Tensor | None = None,
                   group_size: int = AWQ_GROUP, ws: torch.Tensor | None = None, stream=None):
    """y = x (dequant W)^T, [M, N] of out_dtype (default x.dtype)."""
    _dev(x, "x")
    _dev(qweight, "qweight")
    M, K, ldx = _rows(x, "x")
    N = qweight.shape[0]
    if qweight.shape[1] * 8 != K:
        raise ValueError("qweight must be [N, K/8]")
    dev = x.device
    if y is None:
        y = torch.empty((M, N), dtype=out_dtype or x.dtype, device=dev)
    ldy = y.stride(0) if y.dim() == 2 else N
    ws, wsb = _workspace(awq_workspace_bytes(AWQ_OP_GEMM, M, N, K, 0, 0), dev, ws)
    st = lib().awq_w4a16_gemm(_ptr(x), _DT.get(x.dtype, -1), M, K, ldx, _ptr(qweight), _ptr(scales),
                              _ptr(zeros), N, group_size, _ptr(inv_s), _ptr(y), _DT.get(y.dtype, -1),
                              ldy, _ptr(ws), wsb, _stream(dev, stream))
    _abi.check("awq_w4a16_gemm", st)
    return y


def awq_w4a16_gemm_noalloc(x: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor,
                           zeros: torch.Tensor, inv_s: torch.Tensor | None = None,
                           y: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
                           group_size: int = AWQ_GROUP, stream=None):
    """awq_w4a16_gemm without a workspace: the library's own per-GPU scratch
    array serves the product (calls that overlap on one GPU race).  Pass y to
    call it without any allocation."""
    _dev(x, "x")
    _dev(qweight, "qweight")
    M, K, ldx = _rows(x, "x")
    N = qweight.shape[0]
    if qweight.shape[1] * 8 != K:
        raise ValueError("qweight must be [N, K/8]")
    if y is None:
        y = torch.empty((M, N), dtype=out_dtype or x.dtype, device=x.device)
    ldy = y.stride(0) if y.dim() == 2 else N
    st = lib().awq_w4a16_gemm_noalloc(_ptr(x), _DT.get(x.dtype, -1), M, K, ldx, _ptr(qweight),
                                      _ptr(scales), _ptr(zeros), N, group_size, _ptr(inv_s), _ptr(y),
                                      _DT.get(y.dtype, -1), ldy, _stream(x.device, stream))
    _abi.check("awq_w4a16_gemm_noalloc", st)
    return y


def awq_read_stream(buf: torch.Tensor, blocks: int, unroll: int = 4, block_xor: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """A plain streaming read of buf's bytes (a multiple of 1024); returns the
    per-block XOR of the 32-bit words read (int32 [blocks]).  The rate the
    products are measured against."""
    _dev(buf, "buf")
    if not buf.is_contiguous():
        raise ValueError("buf must be contiguous")
    if block_xor is None:
        block_xor = torch.empty(blocks, dtype=torch.int32, device=buf.device)
    st = lib().awq_read_stream(_ptr(buf), buf.numel() * buf.element_size(), blocks, unroll,
                               _ptr(block_xor), _stream(buf.device, stream))
    _abi.check("awq_read_stream", st)
    return block_xor


def awq_fold_scales(v: torch.Tensor, s: torch.Tensor, axis: int = 1, stream=None) -> torch.Tensor:
    """In place: v[i][j] /= s[j] (axis 1) or s[i] (axis 0); a 1-D v is one row."""
    _dev(v, "v")
    _dev(s, "s")
    if s.dtype != torch.float32 or s.dim() != 1 or not s.is_contiguous():
        raise ValueError("s must be a contiguous float32 vector")
    v2 = v.view(1, -1) if v.dim() == 1 else v
    rows, cols, ld = _rows(v2, "v")
    if s.numel() != (cols if axis == 1 else rows):
        raise ValueError("s must have one entry per column (axis 1) or per row (axis 0)")
    st = lib().awq_fold_scales(_ptr(v2), _DT.get(v.dtype, -1), rows, cols, ld, _ptr(s), axis,
                               _stream(v.device, stream))
    _abi.check("awq_fold_scales", st)
    return v


# ---- operators whose weight depends on the row ---------------------------------
_SCORES = {"softmax": AWQ_SCORE_SOFTMAX, "sigmoid": AWQ_SCORE_SIGMOID}
_ACTS = {"none": AWQ_ACT_NONE, "swiglu": AWQ_ACT_SWIGLU}


def _same(t: torch.Tensor | None, name: str, dev: int, dtype: torch.dtype, shape: tuple) -> int | None:
    """Address of a contiguous tensor of this type, shape and GPU (None for None)."""
    if t is None:
        return None
    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or t.get_device() != dev
            or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)} on cuda:{dev}")
    return t.data_ptr()


def _act_rows(x: torch.Tensor, name: str) -> tuple[int, int, int]:
    """rows, columns and row stride of a 2-D tensor; a single row's stride is its length."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        _dev(x, name)
    if x.dim() != 2:
        raise ValueError(f"{name} must be 2-D with unit column stride")
    rows, cols = x.shape
    if x.is_contiguous():
        return rows, cols, cols
    ld, step = x.stride()
    if rows and cols > 1 and step != 1:
        raise ValueError(f"{name} must be 2-D with unit column stride")
    return rows, cols, ld if rows > 1 else cols


def _new(rows: int, cols: int, dtype: torch.dtype, dev: torch.device) -> torch.Tensor:
    """An output (the strided form is 0.4 us a tensor cheaper on the host than empty)."""
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=dev)


def _out(y: torch.Tensor | None, name: str, dev: torch.device, dtype: torch.dtype | None, rows: int,
         cols: int) -> tuple[torch.Tensor, int]:
    """The output (a new one of dtype if y is None) and its row stride."""
    if y is None:
        return _new(rows, cols, dtype, dev), cols
    r, c, ld = _act_rows(y, name)
    if (r, c) != (rows, cols) or y.device != dev or (dtype is not None and y.dtype is not dtype):
        raise ValueError(f"{name} must be a {dtype or y.dtype} tensor of shape [{rows}, {cols}] on {dev}")
    return y, ld


def _launch(name: str, dev: int, args: tuple) -> None:
    """Calls the entry point on the tensors' GPU and its current stream."""
    fn = getattr(lib(), name)
    if dev == torch._C._cuda_getDevice():
        st = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _abi.check(name, st)


def _on_stream(stream, t: torch.Tensor):
    """Makes a given stream (or its handle) the current one, so that outputs
    and workspaces made for the call belong to it."""
    _dev(t, "the first tensor")
    if getattr(stream, "device", t.device) != t.device:
        raise ValueError(f"stream must belong to {t.device}, where the tensors are")
    if not isinstance(stream, torch.cuda.Stream):
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        stream = torch.cuda.ExternalStream(raw, t.device) if raw else torch.cuda.default_stream(t.device)
    return torch.cuda.stream(stream)


@functools.lru_cache(maxsize=4096)
def _ws_need(op: int, M: int, N: int, K: int, T: int, n: int, dev: int) -> int:
    """What one call of the operators below needs on GPU dev: a function of the sizes and of its compute units."""
    if dev == torch._C._cuda_getDevice():
        return lib().awq_workspace_bytes_exact(op, M, N, K, T, n)
    with torch.cuda.device(dev):
        return lib().awq_workspace_bytes_exact(op, M, N, K, T, n)


def _ws(op: int, dev: torch.device, ws: torch.Tensor | None, M: int, N: int, K: int, T: int,
        n: int) -> tuple[torch.Tensor | None, int | None, int]:
    if ws is None:
        need = _ws_need(op, M, N, K, T, n, dev.index)
        if not need:
            return None, None, 0
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
        return ws, ws.data_ptr(), need
    if ws.device != dev or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous tensor on {dev}")
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def awq_route_experts(logits: torch.Tensor, top_k: int, bias: torch.Tensor | None = None, score: str = "softmax",
                      n_group: int = 1, topk_group: int = 1, group_top: int = 1, renormalize: bool = True,
                      scale: float = 1.0, ids: torch.Tensor | None = None, weights: torch.Tensor | None = None,
                      stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Which experts serve each token: (ids int32 [T, top_k], weights float32 [T, top_k]).

    score is "softmax" or "sigmoid"; bias (float32 [E]) only chooses; with
    n_group > 1 only the topk_group best groups of consecutive experts stay,
    a group worth the sum of its group_top (1 or 2) best choices.  A logit of
    -inf or NaN switches an expert off; where fewer than top_k are left the ids
    are -1 with weight 0."""
    if stream is not None:
        with _on_stream(stream, logits):
            return awq_route_experts(logits, top_k, bias, score, n_group, topk_group, group_top, renormalize, scale,
                                     ids, weights)
    T, E, ldl = _act_rows(logits, "logits")
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}")
    device, dev = logits.device, logits.get_device()
    if ids is None:
        ids = _new(T, top_k, torch.int32, device)
    else:
        _same(ids, "ids", dev, torch.int32, (T, top_k))
    if weights is None:
        weights = _new(T, top_k, torch.float32, device)
    else:
        _same(weights, "weights", dev, torch.float32, (T, top_k))
    _launch("awq_route_experts", dev,
            (logits.data_ptr(), _DT.get(logits.dtype, -1), T, E, ldl,
             _same(bias, "bias", dev, torch.float32, (E,)), _SCORES[score], n_group, topk_group, group_top, top_k,
             int(bool(renormalize)), scale, ids.data_ptr(), weights.data_ptr()))
    return ids, weights


def _experts(name, op, x, ids, weights, qweight, scales, zeros, act, out_dtype, y, group_size, ws, stream):
    if stream is not None:
        with _on_stream(stream, x):
            return _experts(name, op, x, ids, weights, qweight, scales, zeros, act, out_dtype, y, group_size, ws, None)
    rows, K, ldx = _act_rows(x, "x")
    device, dev = x.device, x.get_device()
    if ids.dim() != 2:
        raise ValueError("ids must be [tokens, top_k]")
    M, top_k = ids.shape
    if rows != (M if weights is None else M * top_k):
        raise ValueError("x must have one row per token (up) or per slot (down)")
    packed = qweight.shape
    if len(packed) != 3 or packed[2] * 8 != K:
        raise ValueError("qweight must be [experts, N, K/8]")
    if group_size not in (64, 128, 256):
        raise ValueError("group_size must be 64, 128 or 256")
    E, N, _ = packed
    groups = (E, N, K // group_size)
    swiglu = act == AWQ_ACT_SWIGLU
    out_rows, cols = (M * top_k, N // 2 if swiglu else N) if weights is None else (M, N)
    y, ldy = _out(y, "y", device, out_dtype if y is not None else out_dtype or x.dtype, out_rows, cols)
    ws, wsp, wsb = _ws(op, device, ws, M, N, K, E, top_k)
    head = (x.data_ptr(), _DT.get(x.dtype, -1), M, K, ldx, _same(ids, "ids", dev, torch.int32, (M, top_k)))
    packed = (_same(qweight, "qweight", dev, torch.int32, packed), _same(scales, "scales", dev, torch.float16, groups),
              _same(zeros, "zeros", dev, torch.uint8, groups))
    tail = (y.data_ptr(), _DT.get(y.dtype, -1), ldy, wsp, wsb)
    if weights is None:
        args = head + (top_k,) + packed + (E, N, group_size, act) + tail
    else:
        args = head + (_same(weights, "weights", dev, torch.float32, (M, top_k)), top_k) + packed + (E, N, group_size) + tail
    _launch(name, dev, args)
    return y


def awq_w4a16_experts_up(x: torch.Tensor, ids: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor,
                         zeros: torch.Tensor, act: str = "none", out_dtype: torch.dtype | None = None,
                         y: torch.Tensor | None = None, group_size: int = AWQ_GROUP,
                         ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Each token's row through its experts' packed weights, [M top_k, N] (act
    "swiglu": silu(first N/2 rows) * the other N/2, [M top_k, N/2]).

    x [M, K]; ids int32 [M, top_k] (outside [0, experts): no expert, a row of
    zeros); qweight [experts, N, K/8], scales and zeros [experts, N, K/g] as
    awq_quantize_pack writes them for the [experts N, K] rows."""
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}")
    return _experts("awq_w4a16_experts_up", AWQ_OP_EXPERTS_UP, x, ids, None, qweight, scales, zeros, _ACTS[act],
                    out_dtype, y, group_size, ws, stream)


def awq_w4a16_experts_down(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, qweight: torch.Tensor,
                           scales: torch.Tensor, zeros: torch.Tensor, out_dtype: torch.dtype | None = None,
                           y: torch.Tensor | None = None, group_size: int = AWQ_GROUP,
                           ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[m] = sum_j weights[m, j] W_{ids[m, j]} x[m top_k + j], [M, N]; x has one
    row per (token, choice), as awq_w4a16_experts_up writes them."""
    return _experts("awq_w4a16_experts_down", AWQ_OP_EXPERTS_DOWN, x, ids, weights, qweight, scales, zeros, None,
                    out_dtype, y, group_size, ws, stream)


def awq_lora_add(x: torch.Tensor, adapter: torch.Tensor, a: torch.Tensor, b: torch.Tensor,
                 base: torch.Tensor | None = None, scaling: torch.Tensor | None = None,
                 ranks: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
                 y: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """base + scaling[i] b[i] (a[i] x) per row with i = adapter[row]; rows whose
    adapter is outside [0, adapters) are base (0 without one).

    x [M, K]; adapter int32 [M]; a [adapters, R, K] and b [adapters, N, R] of
    x's dtype; ranks int32 [adapters] (None: R); scaling float32 [adapters].
    base has the output's dtype and may be y itself."""
    if stream is not None:
        with _on_stream(stream, x):
            return awq_lora_add(x, adapter, a, b, base, scaling, ranks, out_dtype, y, ws)
    M, K, ldx = _act_rows(x, "x")
    device, dev = x.device, x.get_device()
    if a.dim() != 3 or b.dim() != 3:
        raise ValueError("a must be [adapters, R, K] and b [adapters, N, R]")
    L, R = a.shape[:2]
    N = b.shape[1]
    want = out_dtype or (base.dtype if base is not None else x.dtype if y is None else y.dtype)
    y, ldy = _out(y, "y", device, want, M, N)
    ldb, basep = 0, None
    if base is not None:
        base, ldb = _out(base, "base", device, y.dtype, M, N)
        basep = base.data_ptr()
    ws, wsp, wsb = _ws(AWQ_OP_LORA, device, ws, M, N, K, L, R)
    _launch("awq_lora_add", dev,
            (x.data_ptr(), _DT.get(x.dtype, -1), M, K, ldx, _same(adapter, "adapter", dev, torch.int32, (M,)),
             _same(a, "a", dev, x.dtype, (L, R, K)), _same(b, "b", dev, x.dtype, (L, N, R)), L, R,
             _same(ranks, "ranks", dev, torch.int32, (L,)), _same(scaling, "scaling", dev, torch.float32, (L,)),
             basep, ldb, N, y.data_ptr(), _DT.get(y.dtype, -1), ldy, wsp, wsb))
    return y


# ---- operators of a block around the packed linears ------------------------------
_LINEAR_ACTS = {"none": AWQ_ACT_NONE, "relu": AWQ_ACT_RELU, "gelu": AWQ_ACT_GELU, "gelu_tanh": AWQ_ACT_GELU_TANH,
                "silu": AWQ_ACT_SILU}


def _act_of(act: str) -> int:
    if act not in _LINEAR_ACTS:
        raise ValueError(f"act must be one of {sorted(_LINEAR_ACTS)}")
    return _LINEAR_ACTS[act]


def _vector(t: torch.Tensor | None, name: str, dev: int, n: int) -> tuple[int | None, int]:
    """Address and type of a contiguous vector of n values of any of the three types (None: NULL)."""
    if t is None:
        return None, AWQ_F32
    dt = _DT.get(t.dtype) if isinstance(t, torch.Tensor) else None
    if dt is None or t.shape != (n,) or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {n} values (float16, bfloat16 or float32) on cuda:{dev}")
    return t.data_ptr(), dt


def _packed(qweight: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor, group_size: int, dev: int) -> tuple:
    """(qweight, scales, zeros addresses, N, K) of one packed linear."""
    if not isinstance(qweight, torch.Tensor) or qweight.dim() != 2:
        raise ValueError("qweight must be [N, K/8]")
    if group_size not in (64, 128, 256):
        raise ValueError("group_size must be 64, 128 or 256")
    N, words = qweight.shape
    K = words * 8
    groups = (N, K // group_size)
    return (_same(qweight, "qweight", dev, torch.int32, qweight.shape), _same(scales, "scales", dev, torch.float16, groups),
            _same(zeros, "zeros", dev, torch.uint8, groups), N, K)


def _rows_like(t: torch.Tensor | None, name: str, dev: torch.device, dtype: torch.dtype, rows: int,
               cols: int) -> tuple[int | None, int]:
    """Address and row stride of an optional [rows, cols] tensor of dtype."""
    if t is None:
        return None, 0
    t, ld = _out(t, name, dev, dtype, rows, cols)
    return t.data_ptr(), ld


def _mask(mask: torch.Tensor | None, dev: int, T: int) -> int | None:
    if mask is None:
        return None
    return _same(mask, "mask", dev, torch.bool if isinstance(mask, torch.Tensor) and mask.dtype is torch.bool else torch.uint8, (T,))


def awq_w4a16_linear(x: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
                     bias: torch.Tensor | None = None, act: str = "none", residual: torch.Tensor | None = None,
                     pre: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
                     y: torch.Tensor | None = None, group_size: int = AWQ_GROUP, ws: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """act(x (dequant W)^T + bias) + residual, [M, N].

    act: "none", "relu", "gelu" (erf), "gelu_tanh" or "silu"; bias [N] of any
    type; residual [M, N] of the output's type, which may be y itself.  pre, an
    [M, N] tensor of the output's type, receives the value before the
    activation, for awq_bias_act_backward.  The output's type is out_dtype, or
    y's, or residual's, or x's."""
    if stream is not None:
        with _on_stream(stream, x):
            return awq_w4a16_linear(x, qweight, scales, zeros, bias, act, residual, pre, out_dtype, y, group_size, ws)
    kind = _act_of(act)
    M, K, ldx = _act_rows(x, "x")
    device, dev = x.device, x.get_device()
    qp, sp, zp, N, Kw = _packed(qweight, scales, zeros, group_size, dev)
    if Kw != K:
        raise ValueError("qweight must be [N, K/8]")
    want = out_dtype or (residual.dtype if y is None and residual is not None else x.dtype if y is None else y.dtype)
    y, ldy = _out(y, "y", device, want, M, N)
    resp, ldr = _rows_like(residual, "residual", device, y.dtype, M, N)
    prep, ldp = _rows_like(pre, "pre", device, y.dtype, M, N)
    bp, bdt = _vector(bias, "bias", dev, N)
    ws, wsp, wsb = _ws(AWQ_OP_LINEAR, device, ws, M, N, K, 0, 0)
    _launch("awq_w4a16_linear", dev,
            (x.data_ptr(), _DT.get(x.dtype, -1), M, K, ldx, qp, sp, zp, N, group_size, bp, bdt, kind, resp, ldr, prep, ldp,
             y.data_ptr(), _DT.get(y.dtype, -1), ldy, wsp, wsb))
    return y


def awq_bias_act_backward(dy: torch.Tensor, pre: torch.Tensor | None = None, act: str = "none",
                          dz: torch.Tensor | None = None, dbias: torch.Tensor | bool = True,
                          ws: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """Backward pass of awq_w4a16_linear's epilogue: (dz [M, N] of dy's type,
    dbias float32 [N]).  pre is what the forward pass wrote there.  With act
    "none" dz is dy itself; dbias=False leaves the bias's gradient out; dz may
    be dy or pre."""
    if stream is not None:
        with _on_stream(stream, dy):
            return awq_bias_act_backward(dy, pre, act, dz, dbias, ws)
    kind = _act_of(act)
    M, N, lddy = _act_rows(dy, "dy")
    device, dev = dy.device, dy.get_device()
    pp, ldp, dzp, lddz = None, 0, None, 0
    if kind == AWQ_ACT_NONE:
        if dz is not None and dz is not dy:
            raise ValueError("with act \"none\" dz is dy itself")
        dz = dy
    else:
        if pre is None:
            raise ValueError("pre is needed where there is an activation")
        pp, ldp = _rows_like(pre, "pre", device, dy.dtype, M, N)
        dz, lddz = _out(dz, "dz", device, dy.dtype, M, N)
        dzp = dz.data_ptr()
    if isinstance(dbias, bool):
        dbias = torch.empty(N, dtype=torch.float32, device=device) if dbias else None
    dbp = _same(dbias, "dbias", dev, torch.float32, (N,))
    wsp, wsb = None, 0
    if dbias is not None:
        ws, wsp, wsb = _ws(AWQ_OP_BIAS_ACT_BACKWARD, device, ws, M, N, 0, 0, 0)
    if kind != AWQ_ACT_NONE or dbias is not None:
        _launch("awq_bias_act_backward", dev,
                (dy.data_ptr(), _DT.get(dy.dtype, -1), M, N, lddy, pp, ldp, kind, dzp, lddz, dbp, wsp, wsb))
    return dz, dbias


def awq_w4a16_gemm_dx(dz: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
                      out_dtype: torch.dtype | None = None, dx: torch.Tensor | None = None, group_size: int = AWQ_GROUP,
                      ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """dz (dequant W), [M, K]: the gradient of the W4A16 product's input."""
    if stream is not None:
        with _on_stream(stream, dz):
            return awq_w4a16_gemm_dx(dz, qweight, scales, zeros, out_dtype, dx, group_size, ws)
    M, N, lddz = _act_rows(dz, "dz")
    device, dev = dz.device, dz.get_device()
    qp, sp, zp, Nw, K = _packed(qweight, scales, zeros, group_size, dev)
    if Nw != N:
        raise ValueError("qweight must have one row per column of dz")
    dx, lddx = _out(dx, "dx", device, out_dtype if dx is not None else out_dtype or dz.dtype, M, K)
    ws, wsp, wsb = _ws(AWQ_OP_GEMM_DX, device, ws, M, N, K, 0, 0)
    _launch("awq_w4a16_gemm_dx", dev,
            (dz.data_ptr(), _DT.get(dz.dtype, -1), M, N, lddz, qp, sp, zp, K, group_size, dx.data_ptr(),
             _DT.get(dx.dtype, -1), lddx, wsp, wsb))
    return dx


def awq_layer_norm(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None, eps: float = 1e-5,
                   rms: bool = False, out_dtype: torch.dtype | None = None, y: torch.Tensor | None = None,
                   stats: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """(x - mean) / sqrt(var + eps) * weight + bias of each row (rms: mean 0),
    [M, K] of out_dtype (default x's).  weight and bias [K] of any type; y may
    be x.  stats, a float32 [2, M] tensor, receives each row's mean and
    1 / sqrt(var + eps), for awq_layer_norm_backward."""
    if stream is not None:
        with _on_stream(stream, x):
            return awq_layer_norm(x, weight, bias, eps, rms, out_dtype, y, stats)
    M, K, ldx = _act_rows(x, "x")
    device, dev = x.device, x.get_device()
    if weight is None:
        raise ValueError("weight must be a vector")
    wp, wdt = _vector(weight, "weight", dev, K)
    bp, bdt = _vector(bias, "bias", dev, K)
    y, ldy = _out(y, "y", device, out_dtype if y is not None else out_dtype or x.dtype, M, K)
    sp = _same(stats, "stats", dev, torch.float32, (2, M))
    _launch("awq_layer_norm", dev,
            (x.data_ptr(), _DT.get(x.dtype, -1), M, K, ldx, wp, wdt, bp, bdt, eps, int(bool(rms)), y.data_ptr(),
             _DT.get(y.dtype, -1), ldy, sp, None if sp is None else sp + 4 * M))
    return y


def awq_layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, stats: torch.Tensor,
                            rms: bool = False, bias: bool = True, dx: torch.Tensor | None = None,
                            dweight: torch.Tensor | bool = True, ws: torch.Tensor | None = None, stream=None):
    """Backward pass of awq_layer_norm: (dx [M, K] of x's type, dweight float32
    [K], dbias float32 [K]).  stats as the forward pass wrote it.  bias=False
    (a norm without a bias) and dweight=False leave those sums out (None);
    tensors given for them receive them.  dx may be dy or x."""
    if stream is not None:
        with _on_stream(stream, dy):
            return awq_layer_norm_backward(dy, x, weight, stats, rms, bias, dx, dweight, ws)
    M, K, lddy = _act_rows(dy, "dy")
    device, dev = dy.device, dy.get_device()
    if x.device != device or x.shape != dy.shape:
        raise ValueError(f"x must be a tensor of shape [{M}, {K}] on {device}")
    _, _, ldx = _act_rows(x, "x")
    if weight is None or stats is None:
        raise ValueError("weight and stats must be tensors")
    wp, wdt = _vector(weight, "weight", dev, K)
    sp = _same(stats, "stats", dev, torch.float32, (2, M))
    dx, lddx = _out(dx, "dx", device, x.dtype, M, K)
    dbias = bias
    if isinstance(dbias, bool):
        dbias = torch.empty(K, dtype=torch.float32, device=device) if dbias else None
    if isinstance(dweight, bool):
        dweight = torch.empty(K, dtype=torch.float32, device=device) if dweight else None
    wsp, wsb = None, 0
    if dweight is not None or dbias is not None:
        ws, wsp, wsb = _ws(AWQ_OP_LAYER_NORM_BACKWARD, device, ws, M, 0, K, 0, 0)
    _launch("awq_layer_norm_backward", dev,
            (dy.data_ptr(), _DT.get(dy.dtype, -1), M, K, lddy, x.data_ptr(), _DT.get(x.dtype, -1), ldx, wp, wdt, sp,
             sp + 4 * M, int(bool(rms)), dx.data_ptr(), lddx, _same(dweight, "dweight", dev, torch.float32, (K,)),
             _same(dbias, "dbias", dev, torch.float32, (K,)), wsp, wsb))
    return dx, dweight, dbias


def awq_balance_loss(logits: torch.Tensor, ids: torch.Tensor, coef: float = 1.0, score: str = "softmax",
                     mask: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None):
    """The balance loss of a router: (loss float32 [1], counts int32 [E], slope
    float32 [E]), loss = coef E sum_e (counts_e / n) mean_t p_te over the tokens
    that count, slope its derivative by each p.

    logits [T, E]; ids int32 [T, top_k] as awq_route_experts writes them; score
    "softmax" or "sigmoid" (divided by the row's sum); mask (bool or uint8 [T]):
    tokens with 0 do not count, nor do tokens whose logits are all -inf or NaN."""
    if stream is not None:
        with _on_stream(stream, logits):
            return awq_balance_loss(logits, ids, coef, score, mask, ws)
    T, E, ldl = _act_rows(logits, "logits")
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}")
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise ValueError("ids must be [tokens, top_k]")
    device, dev = logits.device, logits.get_device()
    top_k = ids.shape[1]
    loss = torch.empty(1, dtype=torch.float32, device=device)
    counts = torch.empty(E, dtype=torch.int32, device=device)
    slope = torch.empty(E, dtype=torch.float32, device=device)
    ws, wsp, wsb = _ws(AWQ_OP_BALANCE_LOSS, device, ws, T, 0, 0, E, 0)
    _launch("awq_balance_loss", dev,
            (logits.data_ptr(), _DT.get(logits.dtype, -1), T, E, ldl, _same(ids, "ids", dev, torch.int32, (T, top_k)),
             top_k, _mask(mask, dev, T), _SCORES[score], coef, loss.data_ptr(), counts.data_ptr(), slope.data_ptr(),
             wsp, wsb))
    return loss, counts, slope


def awq_balance_loss_backward(logits: torch.Tensor, slope: torch.Tensor, grad: torch.Tensor | None = None,
                              score: str = "softmax", mask: torch.Tensor | None = None,
                              dlogits: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The gradient of awq_balance_loss's loss by the logits, [T, E] of their
    type.  slope as awq_balance_loss returned it, score and mask as given to it;
    grad: float32 [1], the gradient of the loss (None: 1).  dlogits may be
    logits."""
    if stream is not None:
        with _on_stream(stream, logits):
            return awq_balance_loss_backward(logits, slope, grad, score, mask, dlogits)
    T, E, ldl = _act_rows(logits, "logits")
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}")
    device, dev = logits.device, logits.get_device()
    if slope is None:
        raise ValueError("slope must be a tensor")
    dlogits, ldd = _out(dlogits, "dlogits", device, logits.dtype, T, E)
    _launch("awq_balance_loss_backward", dev,
            (logits.data_ptr(), _DT.get(logits.dtype, -1), T, E, ldl, _same(slope, "slope", dev, torch.float32, (E,)),
             _same(grad, "grad", dev, torch.float32, (1,)), _mask(mask, dev, T), _SCORES[score], dlogits.data_ptr(), ldd))
    return dlogits
