"""Training-side operators (declared in include/conv_train.h): group norm with
its activation and gradients, the softmax cross entropy of a 1x1 head with
its gradients, and the orthogonalised update of weight matrices.

Argument marshalling only, as in ``_lib``: every step of the computation runs
in the HIP library, on the current torch stream or on ``stream``. Outputs and
scratch memory are allocated when they are not given; torch's allocator ties
them to the current stream, so a caller that passes another ``stream`` gives
``ws`` and the outputs too, or keeps the two streams ordered.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence, Tuple

import torch

from . import _lib

NORM_ACTS = dict(_lib.ACTS, silu=4)
_FLOATS = {torch.float32: 0, torch.bfloat16: 1}


class _NormDesc(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("h", ctypes.c_int64), ("w", ctypes.c_int64), ("c", ctypes.c_int64),
                ("x_pixel_stride", ctypes.c_int64), ("groups", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("act", ctypes.c_int32), ("eps", ctypes.c_float)]


class _HeadDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("c", ctypes.c_int64), ("classes", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("label_bytes", ctypes.c_int32)]


class _OrthoDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("steps", ctypes.c_int32), ("a", ctypes.c_float), ("b", ctypes.c_float),
                ("c", ctypes.c_float), ("eps", ctypes.c_float)]


_bound = None


def _L():
    """The library with the argument types of this module's entry points."""
    global _bound
    if _bound is None:
        L = _lib.lib()
        P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        ND = ctypes.POINTER(_NormDesc)
        L.conv_group_norm_ws_bytes.argtypes = [ND, I32]
        L.conv_group_norm_ws_bytes.restype = I64
        L.conv_group_norm.argtypes = [ND, P, P, P, P, P, P, I64, P]
        L.conv_group_norm.restype = ctypes.c_int
        L.conv_group_norm_grad.argtypes = [ND] + [P] * 9 + [I64, P]
        L.conv_group_norm_grad.restype = ctypes.c_int
        HD, OD = ctypes.POINTER(_HeadDesc), ctypes.POINTER(_OrthoDesc)
        L.conv_head_loss_ws_bytes.argtypes = [HD, I32]
        L.conv_head_loss_ws_bytes.restype = I64
        L.conv_head_loss.argtypes = [HD] + [P] * 7 + [I64, P]
        L.conv_head_loss.restype = ctypes.c_int
        L.conv_head_loss_grad.argtypes = [HD] + [P] * 9 + [I64, P]
        L.conv_head_loss_grad.restype = ctypes.c_int
        L.conv_orthogonalize_ws_bytes.argtypes = [OD]
        L.conv_orthogonalize_ws_bytes.restype = I64
        L.conv_orthogonalize.argtypes = [OD, P, P, P, I64, P]
        L.conv_orthogonalize.restype = ctypes.c_int
        _bound = L
    return _bound


def _dev(t: torch.Tensor, name: str, dt, shape):
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    if t.dtype != dt:
        raise ValueError("%s dtype %s, expected %s" % (name, t.dtype, dt))
    if t.shape != shape:
        raise ValueError("%s shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _scratch(need: int, ws: Optional[torch.Tensor], device, what: str) -> Optional[torch.Tensor]:
    """ws as given, or scratch of `need` bytes (a negative need is the
    library's refusal of the description)."""
    if need < 0:
        _lib._check(int(need), what)
    if ws is not None:
        if not ws.is_cuda or not ws.is_contiguous():
            raise ValueError("ws must be a contiguous device tensor")
        return ws
    return torch.empty(need, dtype=torch.uint8, device=device) if need else None


def _ws_args(ws: Optional[torch.Tensor]) -> Tuple[Optional[int], int]:
    return (None, 0) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size())


# ------------------------------------------------------------------ group norm --

def _norm_desc(x: torch.Tensor, groups: int, eps: float, act: str) -> _NormDesc:
    if x.dim() != 4 or x.dtype not in _FLOATS or not x.is_cuda:
        raise ValueError("x must be a [n, h, w, c] float32 or bfloat16 device tensor")
    if act not in NORM_ACTS:
        raise ValueError("act %r, expected one of %s" % (act, ", ".join(NORM_ACTS)))
    n, h, w, c = x.shape
    pitch = 0
    if not x.is_contiguous():
        # one step from pixel to pixel over the whole map: a channel slice of a wider NHWC map
        pitch = x.stride(2) if w > 1 else x.stride(1) if h > 1 else x.stride(0) if n > 1 else c
        if ((c > 1 and x.stride(3) != 1) or (w > 1 and x.stride(2) != pitch) or (h > 1 and x.stride(1) != w * pitch) or
                (n > 1 and x.stride(0) != h * w * pitch)):
            raise ValueError("x must be NHWC with evenly spaced pixels (a contiguous map or a channel slice of one)")
    return _NormDesc(n, h, w, c, pitch, groups, _FLOATS[x.dtype], NORM_ACTS[act], eps)


def _affine(gamma, beta, c):
    for t, name in ((gamma, "gamma"), (beta, "beta")):
        if t is not None:
            _dev(t, name, torch.float32, (c,))


def group_norm_ws_bytes(x: torch.Tensor, groups: int, eps: float = 1e-5, act: str = "none", grad: bool = False) -> int:
    """Bytes of ``ws`` that group_norm (or group_norm_grad) takes for x."""
    need = _L().conv_group_norm_ws_bytes(_norm_desc(x, groups, eps, act), int(grad))
    if need < 0:
        _lib._check(int(need), "conv_group_norm_ws_bytes")
    return int(need)


def group_norm(x: torch.Tensor, groups: int, gamma: Optional[torch.Tensor] = None,
               beta: Optional[torch.Tensor] = None, eps: float = 1e-5, act: str = "none",
               y: Optional[torch.Tensor] = None, stats: Optional[torch.Tensor] = None,
               ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y = act(gamma * (x - mean) / sqrt(var + eps) + beta) with the mean and
    variance of each (image, group of c / groups channels).

    x [n, h, w, c] float32 or bfloat16, contiguous or a channel slice of a
    wider map; gamma, beta float32 [c]; act "none", "relu", "relu6", "mish"
    or "silu". stats float32 [n, groups, 2] receives (mean, 1/sqrt(var + eps)),
    which group_norm_grad takes."""
    L = _L()
    d = _norm_desc(x, groups, eps, act)
    _affine(gamma, beta, x.shape[3])
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    else:
        _dev(y, "y", x.dtype, x.shape)
    if stats is not None:
        _dev(stats, "stats", torch.float32, (x.shape[0], groups, 2))
    ws = _scratch(L.conv_group_norm_ws_bytes(d, 0), ws, x.device, "conv_group_norm")
    st = L.conv_group_norm(d, x.data_ptr(), _ptr(gamma), _ptr(beta), y.data_ptr(), _ptr(stats), *_ws_args(ws),
                           _lib._stream_handle(stream))
    _lib._check(st, "conv_group_norm")
    return y


def group_norm_grad(dy: torch.Tensor, x: torch.Tensor, stats: torch.Tensor, gamma: Optional[torch.Tensor] = None,
                    beta: Optional[torch.Tensor] = None, act: str = "none", dx: Optional[torch.Tensor] = None,
                    dgamma: Optional[torch.Tensor] = None, dbeta: Optional[torch.Tensor] = None,
                    ws: Optional[torch.Tensor] = None, stream=None):
    """(dx, dgamma, dbeta) of group_norm for the upstream gradient dy (x's
    shape and dtype, contiguous), from the x, gamma, beta and act of the
    forward call and the stats it wrote."""
    L = _L()
    if stats.dim() != 3:
        raise ValueError("stats must be [n, groups, 2]")
    groups = stats.shape[1]
    d = _norm_desc(x, groups, 0.0, act)  # eps is in the stats
    c = x.shape[3]
    _dev(stats, "stats", torch.float32, (x.shape[0], groups, 2))
    _dev(dy, "dy", x.dtype, x.shape)
    _affine(gamma, beta, c)
    if dx is None:
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    else:
        _dev(dx, "dx", x.dtype, x.shape)
    if dgamma is None:
        dgamma = torch.empty(c, dtype=torch.float32, device=x.device)
    if dbeta is None:
        dbeta = torch.empty(c, dtype=torch.float32, device=x.device)
    _affine(dgamma, dbeta, c)
    ws = _scratch(L.conv_group_norm_ws_bytes(d, 1), ws, x.device, "conv_group_norm_grad")
    st = L.conv_group_norm_grad(d, x.data_ptr(), dy.data_ptr(), stats.data_ptr(), _ptr(gamma), _ptr(beta),
                                dx.data_ptr(), dgamma.data_ptr(), dbeta.data_ptr(), *_ws_args(ws),
                                _lib._stream_handle(stream))
    _lib._check(st, "conv_group_norm_grad")
    return dx, dgamma, dbeta


# ------------------------------------------------------------------- head loss --

def _head_desc(x, w, labels, weights) -> _HeadDesc:
    if w.dim() == 4 and w.shape[1] == w.shape[2] == 1:
        classes, c = w.shape[0], w.shape[3]  # OHWI of a 1x1 layer
    elif w.dim() == 2:
        classes, c = w.shape
    else:
        raise ValueError("w must be [classes, c] (or OHWI [classes, 1, 1, c])")
    if x.dim() < 2 or x.shape[-1] != c:
        raise ValueError("x must be [..., c] with w's %d channels" % c)
    rows = x.numel() // c if c else 0
    _dev(x, "x", torch.bfloat16, x.shape)
    _dev(w, "w", torch.bfloat16, w.shape)
    if labels.dtype not in (torch.int32, torch.int64):
        raise ValueError("labels must be int32 or int64")
    _dev(labels, "labels", labels.dtype, x.shape[:-1])
    if weights is not None:
        _dev(weights, "weights", torch.float32, x.shape[:-1])
    return _HeadDesc(rows, c, classes, _lib.DTYPES["bf16"], labels.element_size())


def head_loss_ws_bytes(rows: int, c: int, classes: int, grad: bool = False) -> int:
    """Bytes of ``ws`` that head_loss (or head_loss_grad) takes."""
    need = _L().conv_head_loss_ws_bytes(_HeadDesc(rows, c, classes, _lib.DTYPES["bf16"], 8), int(grad))
    if need < 0:
        _lib._check(int(need), "conv_head_loss_ws_bytes")
    return int(need)


def head_loss(x: torch.Tensor, w: torch.Tensor, labels: torch.Tensor, weights: Optional[torch.Tensor] = None,
              loss: Optional[torch.Tensor] = None, total: Optional[torch.Tensor] = None,
              ws: Optional[torch.Tensor] = None, stream=None):
    """(total, loss): the softmax cross entropy of each pixel of x [..., c]
    under the 1x1 head w [classes, c] (both bfloat16) and its weighted sum,
    or mean when weights is None, as float32. labels [...] int32 or int64; a
    pixel whose label lies outside 0 .. classes-1 is left out."""
    L = _L()
    d = _head_desc(x, w, labels, weights)
    loss, total = _loss_outputs(x, loss, total)
    ws = _scratch(L.conv_head_loss_ws_bytes(d, 0), ws, x.device, "conv_head_loss")
    st = L.conv_head_loss(d, x.data_ptr(), w.data_ptr(), labels.data_ptr(), _ptr(weights), loss.data_ptr(),
                          total.data_ptr(), *_ws_args(ws), _lib._stream_handle(stream))
    _lib._check(st, "conv_head_loss")
    return total, loss


def _loss_outputs(x, loss, total):
    if loss is None:
        loss = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    else:
        _dev(loss, "loss", torch.float32, x.shape[:-1])
    if total is None:
        total = torch.empty((), dtype=torch.float32, device=x.device)
    else:
        _dev(total, "total", torch.float32, ())
    return loss, total


def head_loss_grad(x: torch.Tensor, w: torch.Tensor, labels: torch.Tensor, weights: Optional[torch.Tensor] = None,
                   loss: Optional[torch.Tensor] = None, total: Optional[torch.Tensor] = None,
                   dx: Optional[torch.Tensor] = None, dw: Optional[torch.Tensor] = None,
                   ws: Optional[torch.Tensor] = None, stream=None):
    """(total, loss, dx, dw): head_loss and the gradients of total, bfloat16
    in the shapes of x and w."""
    L = _L()
    d = _head_desc(x, w, labels, weights)
    loss, total = _loss_outputs(x, loss, total)
    if dx is None:
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    else:
        _dev(dx, "dx", x.dtype, x.shape)
    if dw is None:
        dw = torch.empty(w.shape, dtype=w.dtype, device=w.device)
    else:
        _dev(dw, "dw", w.dtype, w.shape)
    ws = _scratch(L.conv_head_loss_ws_bytes(d, 1), ws, x.device, "conv_head_loss_grad")
    st = L.conv_head_loss_grad(d, x.data_ptr(), w.data_ptr(), labels.data_ptr(), _ptr(weights), loss.data_ptr(),
                               total.data_ptr(), dx.data_ptr(), dw.data_ptr(), *_ws_args(ws),
                               _lib._stream_handle(stream))
    _lib._check(st, "conv_head_loss_grad")
    return total, loss, dx, dw


# ------------------------------------------------------------ orthogonalisation --

MUON_COEFFS = (3.4445, -4.7750, 2.0315)


def _ortho_desc(g, steps, coeffs, eps) -> _OrthoDesc:
    if g.dim() < 2 or g.dtype not in _FLOATS:
        raise ValueError("g must be float32 or bfloat16, [m, n], [batch, m, n] or OHWI [c_out, kh, kw, c_in]")
    _dev(g, "g", g.dtype, g.shape)
    if g.dim() == 3:
        batch, rows, cols = g.shape
    else:
        batch, rows = 1, g.shape[0]
        cols = g.numel() // rows if rows else 0
    a, b, c = coeffs
    return _OrthoDesc(batch, rows, cols, _FLOATS[g.dtype], steps, a, b, c, eps)


def orthogonalize_ws_bytes(batch: int, rows: int, cols: int) -> int:
    """Bytes of ``ws`` that orthogonalize takes for [batch, rows, cols]."""
    need = _L().conv_orthogonalize_ws_bytes(_OrthoDesc(batch, rows, cols, 0, 1, 1.0, 0.0, 0.0, 0.0))
    if need < 0:
        _lib._check(int(need), "conv_orthogonalize_ws_bytes")
    return int(need)


def orthogonalize(g: torch.Tensor, steps: int = 5, coeffs: Sequence[float] = MUON_COEFFS, eps: float = 1e-7,
                  out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The Newton-Schulz orthogonalisation of g, bfloat16 in g's shape: g
    [m, n], a batch [b, m, n] of matrices, or one layer's OHWI weight gradient
    [c_out, kh, kw, c_in] as the matrix [c_out, kh kw c_in]."""
    L = _L()
    d = _ortho_desc(g, steps, coeffs, eps)
    if out is None:
        out = torch.empty(g.shape, dtype=torch.bfloat16, device=g.device)
    else:
        _dev(out, "out", torch.bfloat16, g.shape)
    ws = _scratch(L.conv_orthogonalize_ws_bytes(d), ws, g.device, "conv_orthogonalize")
    st = L.conv_orthogonalize(d, g.data_ptr(), out.data_ptr(), *_ws_args(ws), _lib._stream_handle(stream))
    _lib._check(st, "conv_orthogonalize")
    return out
