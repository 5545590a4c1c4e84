"""Thin torch-facing wrappers of the C ABI (argument marshalling only)."""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _lib
from ._lib import lib


class BlockFFNError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = lib.blockffn_status_string(status).decode()
        detail = lib.blockffn_last_error_message().decode()
        super().__init__(f"{where}: {msg}" + (f" ({detail})" if detail else ""))
        self.status = status


def _check(status: int, where: str) -> None:
    if status != _lib.OK:
        raise BlockFFNError(status, where)


_DT = {torch.float32: _lib.F32, torch.bfloat16: _lib.BF16}


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype not in _DT:
        raise TypeError(f"unsupported dtype {t.dtype}: use float32 or bfloat16")
    return _DT[t.dtype]


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


# the raw handle without building a Stream object: 0.3 us instead of 3 a call (private to torch, so
# its absence only costs that)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream() -> int:
    """The current device's current stream."""
    device = torch.cuda.current_device()
    return torch.cuda.current_stream(device).cuda_stream if _raw_stream is None else _raw_stream(device)


def _empty(rows: int, cols: int, dtype: torch.dtype, device: torch.device) -> torch.Tensor:
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)


def version() -> int:
    return lib.blockffn_version()


def num_sms() -> int:
    return lib.blockffn_num_sms()


def set_wait_limit_ns(ns: int) -> None:
    """Bound of every in-kernel spin-wait (nanoseconds) for later launches."""
    lib.blockffn_set_wait_limit_ns(int(ns))


def debug_skip_flag(unit: int) -> None:
    """Failure-test support: the finisher of expert-in unit ``unit`` never publishes
    its ready flag (-1 turns this off); see include/blockffn.h."""
    lib.blockffn_debug_skip_flag(int(unit))


def debug_set_trace(buf: Optional[torch.Tensor]) -> None:
    """Attach (or detach with None) a zeroed int64 CUDA tensor of num_sms()*64
    entries that later bf16 forward launches fill with per-block timestamps."""
    if buf is not None and (buf.dtype != torch.int64 or buf.numel() < 64 * num_sms()):
        raise ValueError("trace buffer: int64 tensor of at least num_sms()*64 entries")
    lib.blockffn_debug_set_trace(None if buf is None else _ptr(buf))


def route(x: torch.Tensor, W_r: torch.Tensor, gamma: torch.Tensor, eps: float,
          b_r: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """gates [T, E] fp32 = RMSNorm(ReLU(x W_r^T + b_r)) over the experts."""
    T, d_h = x.shape
    E = W_r.shape[0]
    if out is None:
        out = torch.empty((T, E), dtype=torch.float32, device=x.device)
    st = lib.blockffn_route(_ptr(x), _ptr(W_r), _ptr(b_r), _ptr(gamma), float(eps), T, d_h, E,
                            _dtype_code(x), _ptr(out), _stream())
    _check(st, "blockffn_route")
    return out


def residual_layernorm(y: torch.Tensor, x: torch.Tensor, ln_gamma: torch.Tensor,
                       ln_beta: Optional[torch.Tensor], eps: float = 1e-5,
                       out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out [T, d_h] = LayerNorm(y + x) over d_h (scale ln_gamma, shift ln_beta or none, fp32)."""
    T, d_h = x.shape
    if out is None:
        out = torch.empty_like(x)
    st = lib.blockffn_residual_layernorm(_ptr(y), _ptr(x), _ptr(ln_gamma), _ptr(ln_beta), float(eps),
                                         T, d_h, _dtype_code(x), _ptr(out), _stream())
    _check(st, "blockffn_residual_layernorm")
    return out


def chunk_union(gates: torch.Tensor, n: int):
    """Per-chunk union of active experts: (counts [C], idx [C,E], tmask [C,E] as int32)."""
    T, E = gates.shape
    C = (T + n - 1) // n
    dev = gates.device
    counts = torch.empty(C, dtype=torch.int32, device=dev)
    idx = torch.empty((C, E), dtype=torch.int32, device=dev)
    tmask = torch.empty((C, E), dtype=torch.int32, device=dev)  # bits of a uint32
    st = lib.blockffn_chunk_union(_ptr(gates), T, E, n, _ptr(counts), _ptr(idx), _ptr(tmask),
                                  _stream())
    _check(st, "blockffn_chunk_union")
    return counts, idx, tmask


def workspace_bytes(T: int, d_h: int, E: int, d_e: int, n: int, dtype: torch.dtype,
                    with_router: bool, with_bias: bool = False) -> int:
    flags = (_lib.WS_ROUTER if with_router else 0) | (_lib.WS_EXPERT_BIAS if with_bias else 0)
    return int(lib.blockffn_forward_workspace_bytes(T, d_h, E, d_e, n, _DT[dtype], flags))


class Workspace:
    """Device scratch for ``forward`` (zeroed once; the library keeps state in it)."""

    def __init__(self, nbytes: int, device=None):
        self.buf = torch.empty(max(int(nbytes), 256), dtype=torch.uint8,
                               device=device or torch.device("cuda"))
        self.reset()

    @property
    def nbytes(self) -> int:
        return self.buf.numel()

    def reset(self) -> None:
        _launch("blockffn_workspace_reset", lib.blockffn_workspace_reset, self.buf.device, self.buf.data_ptr(),
                self.nbytes)

    @classmethod
    def for_int8_linear(cls, T: int, K: int, O: int, device=None) -> "Workspace":
        nb = int(lib.blockffn_int8_linear_workspace_bytes(T, K, O))
        if nb == 0:
            raise BlockFFNError(_lib.ERR_INVALID_ARG, "blockffn_int8_linear_workspace_bytes")
        return cls(nb, device)

    @classmethod
    def for_forward_int8(cls, T: int, d_h: int, E: int, d_e: int, device=None) -> "Workspace":
        nb = int(lib.blockffn_forward_int8_workspace_bytes(T, d_h, E, d_e))
        if nb == 0:
            raise BlockFFNError(_lib.ERR_INVALID_ARG, "blockffn_forward_int8_workspace_bytes")
        return cls(nb, device)

    @classmethod
    def for_shapes(cls, T, d_h, E, d_e, n, dtype, with_router, device=None,
                   with_bias: bool = False) -> "Workspace":
        nb = workspace_bytes(T, d_h, E, d_e, n, dtype, with_router, with_bias)
        if nb == 0:
            raise BlockFFNError(_lib.ERR_INVALID_ARG, "blockffn_forward_workspace_bytes")
        return cls(nb, device)


def forward(x: torch.Tensor, W_in: torch.Tensor, W_out: torch.Tensor, n: int,
            gates: Optional[torch.Tensor] = None, W_r: Optional[torch.Tensor] = None,
            b_r: Optional[torch.Tensor] = None, gamma: Optional[torch.Tensor] = None,
            eps: float = 2.0 ** -23, y: Optional[torch.Tensor] = None,
            workspace: Optional[Workspace] = None, union=None,
            b_in: Optional[torch.Tensor] = None, b_out: Optional[torch.Tensor] = None,
            ln_weight: Optional[torch.Tensor] = None, ln_bias: Optional[torch.Tensor] = None,
            ln_eps: float = 1e-5) -> torch.Tensor:
    """y [T, d_h] = sum over each chunk's union experts of
    gate * (W_out_e Swish(W_in_e x + b_in_e) + b_out_e), then LayerNorm(y + x) when
    ``ln_weight`` is given.

    ``union``: optional (counts, idx, tmask) as ``chunk_union`` returns them for
    these gates and n; the forward then uses them instead of forming the union.
    ``b_in`` [E, d_e], ``b_out`` [E, d_h], ``ln_weight``/``ln_bias`` [d_h]: fp32,
    optional (a workspace for ``b_out`` is sized with ``with_bias=True``)."""
    T, d_h = x.shape
    E, d_e, _ = W_in.shape
    if y is None:
        y = torch.empty((T, d_h), dtype=x.dtype, device=x.device)
    if workspace is None:
        workspace = Workspace.for_shapes(T, d_h, E, d_e, n, x.dtype, gates is None, x.device,
                                         with_bias=b_out is not None)
    counts, idx, tmask = union if union is not None else (None, None, None)
    opts = None
    if b_in is not None or b_out is not None or ln_weight is not None:
        opts = ctypes.byref(_lib.LayerOpts(_ptr(b_in), _ptr(b_out), _ptr(ln_weight), _ptr(ln_bias),
                                           float(ln_eps)))
    st = lib.blockffn_forward(_ptr(x), _ptr(gates), _ptr(W_r), _ptr(b_r), _ptr(gamma), float(eps),
                              _ptr(counts), _ptr(idx), _ptr(tmask),
                              _ptr(W_in), _ptr(W_out), T, d_h, E, d_e, n, _dtype_code(x), opts,
                              _ptr(y), workspace.buf.data_ptr(), workspace.nbytes, _stream())
    _check(st, "blockffn_forward")
    return y


# ------------------------------------------------ top-k routing, 8-bit products --
_SCORES = {"softmax": _lib.SOFTMAX, "sigmoid": _lib.SIGMOID}


def _scores_code(scores: str) -> int:
    if scores not in _SCORES:
        raise ValueError(f"scores must be 'softmax' or 'sigmoid', not {scores!r}")
    return _SCORES[scores]


def _want(t: torch.Tensor, what: str, dtype, shape, device) -> torch.Tensor:
    """``t`` itself, once its type, shape and device are as they have to be."""
    if t.dtype != dtype:
        raise TypeError(f"{what}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{what}: on {t.device}, expected {device}")
    return t


def _same_device(workspace: "Workspace", device: torch.device) -> None:
    if workspace.buf.device != device:
        raise ValueError(f"workspace: on {workspace.buf.device}, expected {device}")


def _launch(where: str, fn, device: torch.device, *args) -> None:
    """Call ``fn(*args, stream)`` with the tensors' device current, on its current stream."""
    if device.index == torch.cuda.current_device():
        _check(fn(*args, _stream()), where)
    else:
        with torch.cuda.device(device):
            _check(fn(*args, _stream()), where)


def route_topk(logits: torch.Tensor, k: int, scores: str = "softmax", bias: Optional[torch.Tensor] = None,
               n_group: int = 1, topk_group: Optional[int] = None, renormalize: bool = True, scale: float = 1.0,
               out=None):
    """Top-k routing of router logits [T, E] (fp32 or bf16): (gates [T, E] fp32, ids [T, k]
    int32, weights [T, k] fp32).

    The k experts of largest score (``scores``: "softmax" over the experts or "sigmoid"
    of each) plus ``bias`` [E] fp32, out of the ``topk_group`` best of ``n_group`` groups
    of neighbouring experts (a group counts the sum of its two best); weights are the
    chosen scores without the bias, divided by their sum when ``renormalize`` is set,
    times ``scale``.  ``gates`` holds them densely, as ``chunk_union`` and the forwards
    take them.  Ties go to the lowest index; an expert whose logit is -inf is never
    chosen (ids -1 and weight 0 where too few are left).  ``out``: the three outputs.
    No call of the package records a gradient: ``route_topk_backward`` gives this one's."""
    T, E = logits.shape
    dev = logits.device
    if bias is not None:
        _want(bias, "bias", torch.float32, (E,), dev)
    if out is None:
        gates = _empty(T, E, torch.float32, dev)
        ids = _empty(T, k, torch.int32, dev)
        weights = _empty(T, k, torch.float32, dev)
    else:
        gates, ids, weights = out
        _want(gates, "gates", torch.float32, (T, E), dev)
        _want(ids, "ids", torch.int32, (T, k), dev)
        _want(weights, "weights", torch.float32, (T, k), dev)
    _launch("blockffn_route_topk", lib.blockffn_route_topk, dev, _ptr(logits), _dtype_code(logits), _ptr(bias),
            T, E, k, _scores_code(scores), n_group, n_group if topk_group is None else topk_group,
            int(bool(renormalize)), float(scale), _ptr(gates), _ptr(ids), _ptr(weights))
    return gates, ids, weights


def route_topk_backward(logits: torch.Tensor, ids: torch.Tensor, d_weights: torch.Tensor, scores: str = "softmax",
                        renormalize: bool = True, scale: float = 1.0,
                        d_logits: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient [T, E] (the logits' type) of ``route_topk``'s weights with respect to the
    logits, the choice ``ids`` held fixed, for ``d_weights`` [T, k] fp32."""
    T, E = logits.shape
    dev = logits.device
    k = ids.shape[-1]
    _want(ids, "ids", torch.int32, (T, k), dev)
    _want(d_weights, "d_weights", torch.float32, (T, k), dev)
    if d_logits is None:
        d_logits = torch.empty_like(logits)
    else:
        _want(d_logits, "d_logits", logits.dtype, (T, E), dev)
    _launch("blockffn_route_topk_backward", lib.blockffn_route_topk_backward, dev, _ptr(logits), _dtype_code(logits),
            _ptr(ids), _ptr(d_weights), T, E, k, _scores_code(scores), int(bool(renormalize)), float(scale),
            _ptr(d_logits))
    return d_logits


def quantize_int8(w: torch.Tensor):
    """(q int8 of w's shape, scale fp32 of w's shape without the last axis): every row of
    the last axis in 8 bits, w about q * scale.  Lays out weights for the 8-bit
    products: [O, K] for ``int8_linear``, [E, d_e, d_h] and [E, d_h, d_e] for
    ``forward_int8``."""
    if w.dim() < 1 or w.shape[-1] < 1:
        raise ValueError(f"w: shape {tuple(w.shape)} has no rows to round")
    cols = w.shape[-1]
    rows = w.numel() // cols
    if rows >= 2 ** 31 or cols >= 2 ** 31:
        raise ValueError(f"w: shape {tuple(w.shape)} has too many rows or columns")
    q = torch.empty(w.shape, dtype=torch.int8, device=w.device)
    scale = torch.empty(w.shape[:-1], dtype=torch.float32, device=w.device)
    _launch("blockffn_quantize_int8", lib.blockffn_quantize_int8, w.device, _ptr(w), rows, cols, _dtype_code(w),
            _ptr(q), _ptr(scale))
    return q, scale


def int8_linear(x: torch.Tensor, W: torch.Tensor, s_w: torch.Tensor, bias: Optional[torch.Tensor] = None,
                out_dtype: Optional[torch.dtype] = None, y: Optional[torch.Tensor] = None,
                workspace: Optional[Workspace] = None) -> torch.Tensor:
    """y [T, O] = x W^T in 8-bit integers: x [T, K] (fp32 or bf16) is rounded to 8 bits with
    a scale for each token, W [O, K] int8 has the scales ``s_w`` [O] fp32
    (``quantize_int8``), ``bias`` [O] fp32 is optional.  ``out_dtype``: fp32 or bf16
    (default: x's)."""
    T, K = x.shape
    O = W.shape[0]
    dev = x.device
    _want(W, "W", torch.int8, (O, K), dev)
    _want(s_w, "s_w", torch.float32, (O,), dev)
    if bias is not None:
        _want(bias, "bias", torch.float32, (O,), dev)
    if y is None:
        y = _empty(T, O, out_dtype or x.dtype, dev)
    else:
        _want(y, "y", out_dtype or y.dtype, (T, O), dev)
    if workspace is None:
        workspace = Workspace.for_int8_linear(T, K, O, dev)
    _same_device(workspace, dev)
    _launch("blockffn_int8_linear", lib.blockffn_int8_linear, dev, _ptr(x), _dtype_code(x), _ptr(W), _ptr(s_w),
            _ptr(bias), T, K, O, _dtype_code(y), _ptr(y), _ptr(workspace.buf), workspace.nbytes)
    return y


def forward_int8(x: torch.Tensor, gates: torch.Tensor, W_in: torch.Tensor, s_in: torch.Tensor,
                 W_out: torch.Tensor, s_out: torch.Tensor, y: Optional[torch.Tensor] = None,
                 workspace: Optional[Workspace] = None, b_in: Optional[torch.Tensor] = None,
                 b_out: Optional[torch.Tensor] = None, ln_weight: Optional[torch.Tensor] = None,
                 ln_bias: Optional[torch.Tensor] = None, ln_eps: float = 1e-5) -> torch.Tensor:
    """y [T, d_h] = sum of gate * expert(x) over each token's active experts (gate != 0) with
    both expert products in 8-bit integers, then LayerNorm(y + x) when ``ln_weight`` is
    given.

    ``x`` [T, d_h] bf16 and Swish's result are rounded to 8 bits with a scale per token
    (and expert); ``W_in`` [E, d_e, d_h] and ``W_out`` [E, d_h, d_e] int8 have the channel
    scales ``s_in`` [E, d_e] and ``s_out`` [E, d_h] fp32 (``quantize_int8``).  ``gates``
    [T, E] fp32, as ``route`` and ``route_topk`` return them.  The optional parts are those
    of ``forward``."""
    T, d_h = x.shape
    E, d_e, _ = W_in.shape
    dev = x.device
    _want(gates, "gates", torch.float32, (T, E), dev)
    _want(W_in, "W_in", torch.int8, (E, d_e, d_h), dev)
    _want(s_in, "s_in", torch.float32, (E, d_e), dev)
    _want(W_out, "W_out", torch.int8, (E, d_h, d_e), dev)
    _want(s_out, "s_out", torch.float32, (E, d_h), dev)
    opts = None
    if b_in is not None or b_out is not None or ln_weight is not None:
        for t, what, shape in ((b_in, "b_in", (E, d_e)), (b_out, "b_out", (E, d_h)), (ln_weight, "ln_weight", (d_h,)),
                               (ln_bias, "ln_bias", (d_h,))):
            if t is not None:
                _want(t, what, torch.float32, shape, dev)
        opts = ctypes.byref(_lib.LayerOpts(_ptr(b_in), _ptr(b_out), _ptr(ln_weight), _ptr(ln_bias), float(ln_eps)))
    if y is None:
        y = _empty(T, d_h, x.dtype, dev)
    else:
        _want(y, "y", x.dtype, (T, d_h), dev)
    if workspace is None:
        workspace = Workspace.for_forward_int8(T, d_h, E, d_e, dev)
    _same_device(workspace, dev)
    _launch("blockffn_forward_int8", lib.blockffn_forward_int8, dev, _ptr(x), _ptr(gates), _ptr(W_in), _ptr(s_in),
            _ptr(W_out), _ptr(s_out), T, d_h, E, d_e, _dtype_code(x), opts, _ptr(y), _ptr(workspace.buf),
            workspace.nbytes)
    return y


def device_status(workspace: Workspace):
    """(status, detail) of the workspace's device status word (synchronizes the current stream of the
    workspace's device)."""
    detail = ctypes.c_int32(0)
    device = workspace.buf.device

    def read() -> int:
        return lib.blockffn_get_device_status(workspace.buf.data_ptr(), _stream(), ctypes.byref(detail))

    if device.index == torch.cuda.current_device():
        st = read()
    else:
        with torch.cuda.device(device):
            st = read()
    return int(st), int(detail.value)
