"""Training-side operators (declared in include/conv_train.h): group norm with
its activation and gradients, the softmax cross entropy of a 1x1 head with
its gradients, and the orthogonalised update of weight matrices.

Argument marshalling only, as in ``_lib``: every step of the computation runs
in the HIP library, on the current torch stream or on ``stream`` (a torch
stream or a HIP stream's address). A call with ``stream`` is the call under
``torch.cuda.stream(stream)``: outputs and scratch memory that are not given
come from that stream's memory, so they cannot be handed out again while its
work is still to run. As under that context, the caller orders the streams that
make the inputs and use the outputs.

Nothing here is recorded by autograd: a tensor that requires a gradient is read
like any other and the results carry no graph. The gradients are the *_grad
functions' results.
"""
from __future__ import annotations

import ctypes
import functools
from operator import index
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
        L.conv_group_norm_describe.argtypes = [ND, I32, I32, ctypes.c_char_p, I32]
        L.conv_group_norm_describe.restype = ctypes.c_int
        L.conv_group_norm.argtypes = [ND, P, P, P, P, P, P, I64, P]
        L.conv_group_norm.restype = ctypes.c_int
        L.conv_group_norm_grad.argtypes = [ND] + [P] * 9 + [I64, P]
        L.conv_group_norm_grad.restype = ctypes.c_int
        HD, OD = ctypes.POINTER(_HeadDesc), ctypes.POINTER(_OrthoDesc)
        L.conv_head_loss_ws_bytes.argtypes = [HD, I32]
        L.conv_head_loss_ws_bytes.restype = I64
        L.conv_head_loss_describe.argtypes = [HD, I32, I32, ctypes.c_char_p, I32]
        L.conv_head_loss_describe.restype = ctypes.c_int
        L.conv_head_loss.argtypes = [HD] + [P] * 7 + [I64, P]
        L.conv_head_loss.restype = ctypes.c_int
        L.conv_head_loss_grad.argtypes = [HD] + [P] * 9 + [I64, P]
        L.conv_head_loss_grad.restype = ctypes.c_int
        L.conv_orthogonalize_ws_bytes.argtypes = [OD]
        L.conv_orthogonalize_ws_bytes.restype = I64
        L.conv_orthogonalize_describe.argtypes = [OD, ctypes.c_char_p, I32]
        L.conv_orthogonalize_describe.restype = ctypes.c_int
        L.conv_orthogonalize.argtypes = [OD, P, P, P, I64, P]
        L.conv_orthogonalize.restype = ctypes.c_int
        _bound = L
    return _bound


def _dev(t: torch.Tensor, name: str, dt, shape):
    if t.dtype is dt and t.shape == shape and t.is_cuda and t.is_contiguous():
        return
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    if t.dtype != dt:
        raise ValueError("%s dtype %s, expected %s" % (name, t.dtype, dt))
    if t.shape != shape:
        raise ValueError("%s shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    raise ValueError("%s must be contiguous" % name)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _like(t: torch.Tensor) -> torch.Tensor:
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _scratch(need: int, ws: Optional[torch.Tensor], t: torch.Tensor, what: str):
    """(ws, its address, its bytes): ws as given, or scratch of `need` bytes
    on t's device (a negative need is the library's refusal)."""
    if need < 0:
        _lib._check(need, what)
    if ws is None:
        if not need:
            return None, None, 0
        ws = torch.empty(need, dtype=torch.uint8, device=t.device)
        return ws, ws.data_ptr(), need
    if not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous device tensor")
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def _on(stream, t: torch.Tensor):
    """The context in which a call with `stream` allocates and enqueues."""
    if not t.is_cuda:
        raise ValueError("a call on a stream takes device tensors")
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_lib._stream_handle(stream), device=t.device)
    return torch.cuda.stream(stream)


def _stream(t: torch.Tensor) -> int:
    """The handle of the current stream of t's device."""
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _need(need: int, what: str) -> int:
    if need < 0:
        _lib._check(need, what)
    return need


# The descriptions below and their scratch sizes depend on sizes, types and
# plain numbers alone: they are computed once for each. Callers convert what they
# are given to plain numbers first: a tensor's hash is its identity, and a value
# changed in place would find the description of the old one.
_once = functools.lru_cache(maxsize=4096)


# ------------------------------------------------------------------ group norm --

@_once
def _norm_call(n, h, w, c, pitch, groups, dtype, act, eps, grad):
    d = _NormDesc(n, h, w, c, pitch, groups, _FLOATS[dtype], NORM_ACTS[act], eps)
    return d, int(_L().conv_group_norm_ws_bytes(d, int(grad)))


def _pixel_pitch(x: torch.Tensor) -> int:
    """Elements from one pixel of x to the next; 0 (the library's "c") for a
    contiguous map."""
    if x.is_contiguous():
        return 0
    # one step from pixel to pixel over the whole map: a channel slice of a wider NHWC map
    n, h, w, c = x.shape
    sn, sh, sw, sc = x.stride()
    pitch = sw if w > 1 else sh if h > 1 else sn if n > 1 else c
    # a step below c, that of a broadcast map above all, would be read as another layout
    if (pitch < c or (c > 1 and sc != 1) or (h > 1 and sh != w * pitch) or (n > 1 and sn != h * w * pitch)):
        raise ValueError("x must be NHWC with evenly spaced pixels (a contiguous map or a channel slice of one)")
    return pitch


def _norm_of(x: torch.Tensor, groups: int, eps: float, act: str, grad: bool):
    """(description, scratch bytes) of the norm of x."""
    if x.dim() != 4 or x.dtype not in _FLOATS or not x.is_cuda:
        raise ValueError("x must be a [n, h, w, c] float32 or bfloat16 device tensor")
    if act not in NORM_ACTS:
        raise ValueError("act %r, expected one of %s" % (act, ", ".join(NORM_ACTS)))
    n, h, w, c = x.shape
    pitch = _pixel_pitch(x)
    return _norm_call(n, h, w, c, pitch, index(groups), x.dtype, act, float(eps), grad)


def _affine(gamma, beta, c):
    for t, name in ((gamma, "gamma"), (beta, "beta")):
        if t is not None:
            _dev(t, name, torch.float32, (c,))


def group_norm_ws_bytes(x: torch.Tensor, groups: int, eps: float = 1e-5, act: str = "none", grad: bool = False) -> int:
    """Bytes of ``ws`` that group_norm (or group_norm_grad) takes for x."""
    return _need(_norm_of(x, groups, eps, act, grad)[1], "conv_group_norm_ws_bytes")


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
    if stream is not None:
        with _on(stream, x):
            return group_norm(x, groups, gamma, beta, eps, act, y, stats, ws)
    d, need = _norm_of(x, groups, eps, act, False)
    _affine(gamma, beta, x.shape[3])
    if y is None:
        y = _like(x)
    else:
        _dev(y, "y", x.dtype, x.shape)
    if stats is not None:
        _dev(stats, "stats", torch.float32, (x.shape[0], groups, 2))
    ws, at, size = _scratch(need, ws, x, "conv_group_norm")
    st = _L().conv_group_norm(d, x.data_ptr(), _ptr(gamma), _ptr(beta), y.data_ptr(), _ptr(stats), at, size,
                              _stream(x))
    if st:
        _lib._check(st, "conv_group_norm")
    return y


def group_norm_grad(dy: torch.Tensor, x: torch.Tensor, stats: torch.Tensor, gamma: Optional[torch.Tensor] = None,
                    beta: Optional[torch.Tensor] = None, act: str = "none", dx: Optional[torch.Tensor] = None,
                    dgamma: Optional[torch.Tensor] = None, dbeta: Optional[torch.Tensor] = None,
                    ws: Optional[torch.Tensor] = None, stream=None):
    """(dx, dgamma, dbeta) of group_norm for the upstream gradient dy (x's
    shape and dtype, contiguous), from the x, gamma, beta and act of the
    forward call and the stats it wrote."""
    if stream is not None:
        with _on(stream, x):
            return group_norm_grad(dy, x, stats, gamma, beta, act, dx, dgamma, dbeta, ws)
    if stats.dim() != 3:
        raise ValueError("stats must be [n, groups, 2]")
    groups = stats.shape[1]
    d, need = _norm_of(x, groups, 0.0, act, True)  # eps is in the stats
    c = x.shape[3]
    _dev(stats, "stats", torch.float32, (x.shape[0], groups, 2))
    _dev(dy, "dy", x.dtype, x.shape)
    _affine(gamma, beta, c)
    if dx is None:
        dx = _like(x)
    else:
        _dev(dx, "dx", x.dtype, x.shape)
    if dgamma is None:
        dgamma = torch.empty(c, dtype=torch.float32, device=x.device)
    else:
        _dev(dgamma, "dgamma", torch.float32, (c,))
    if dbeta is None:
        dbeta = torch.empty(c, dtype=torch.float32, device=x.device)
    else:
        _dev(dbeta, "dbeta", torch.float32, (c,))
    ws, at, size = _scratch(need, ws, x, "conv_group_norm_grad")
    st = _L().conv_group_norm_grad(d, x.data_ptr(), dy.data_ptr(), stats.data_ptr(), _ptr(gamma), _ptr(beta),
                                   dx.data_ptr(), dgamma.data_ptr(), dbeta.data_ptr(), at, size, _stream(x))
    if st:
        _lib._check(st, "conv_group_norm_grad")
    return dx, dgamma, dbeta


# ------------------------------------------------------------------- head loss --

@_once
def _head_call(rows, c, classes, label_bytes, grad):
    d = _HeadDesc(rows, c, classes, _lib.DTYPES["bf16"], label_bytes)
    return d, int(_L().conv_head_loss_ws_bytes(d, int(grad)))


def _head_of(x, w, labels, weights, grad):
    """(description, scratch bytes) of the loss of x under w."""
    if w.dim() == 4 and w.shape[1] == w.shape[2] == 1:
        classes, c = w.shape[0], w.shape[3]  # OHWI of a 1x1 layer
    elif w.dim() == 2:
        classes, c = w.shape
    else:
        raise ValueError("w must be [classes, c] (or OHWI [classes, 1, 1, c])")
    pixels = x.shape[:-1]
    if x.dim() < 2 or x.shape[-1] != c:
        raise ValueError("x must be [..., c] with w's %d channels" % c)
    rows = x.numel() // c if c else 0
    _dev(x, "x", torch.bfloat16, x.shape)
    _dev(w, "w", torch.bfloat16, w.shape)
    if labels.dtype not in (torch.int32, torch.int64):
        raise ValueError("labels must be int32 or int64")
    _dev(labels, "labels", labels.dtype, pixels)
    if weights is not None:
        _dev(weights, "weights", torch.float32, pixels)
    return _head_call(rows, c, classes, 8 if labels.dtype is torch.int64 else 4, grad)


def head_loss_ws_bytes(rows: int, c: int, classes: int, grad: bool = False) -> int:
    """Bytes of ``ws`` that head_loss (or head_loss_grad) takes."""
    return _need(_head_call(index(rows), index(c), index(classes), 8, bool(grad))[1], "conv_head_loss_ws_bytes")


def head_loss(x: torch.Tensor, w: torch.Tensor, labels: torch.Tensor, weights: Optional[torch.Tensor] = None,
              loss: Optional[torch.Tensor] = None, total: Optional[torch.Tensor] = None,
              ws: Optional[torch.Tensor] = None, stream=None):
    """(total, loss): the softmax cross entropy of each pixel of x [..., c]
    under the 1x1 head w [classes, c] (both bfloat16) and its weighted sum,
    or mean when weights is None, as float32. labels [...] int32 or int64; a
    pixel whose label lies outside 0 .. classes-1 is left out."""
    if stream is not None:
        with _on(stream, x):
            return head_loss(x, w, labels, weights, loss, total, ws)
    d, need = _head_of(x, w, labels, weights, False)
    loss, total = _loss_outputs(x, loss, total)
    ws, at, size = _scratch(need, ws, x, "conv_head_loss")
    st = _L().conv_head_loss(d, x.data_ptr(), w.data_ptr(), labels.data_ptr(), _ptr(weights), loss.data_ptr(),
                             total.data_ptr(), at, size, _stream(x))
    if st:
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
    if stream is not None:
        with _on(stream, x):
            return head_loss_grad(x, w, labels, weights, loss, total, dx, dw, ws)
    d, need = _head_of(x, w, labels, weights, True)
    loss, total = _loss_outputs(x, loss, total)
    if dx is None:
        dx = torch.empty_like(x)
    else:
        _dev(dx, "dx", x.dtype, x.shape)
    if dw is None:
        dw = torch.empty_like(w)
    else:
        _dev(dw, "dw", w.dtype, w.shape)
    ws, at, size = _scratch(need, ws, x, "conv_head_loss_grad")
    st = _L().conv_head_loss_grad(d, x.data_ptr(), w.data_ptr(), labels.data_ptr(), _ptr(weights), loss.data_ptr(),
                                  total.data_ptr(), dx.data_ptr(), dw.data_ptr(), at, size, _stream(x))
    if st:
        _lib._check(st, "conv_head_loss_grad")
    return total, loss, dx, dw


# ------------------------------------------------------------ orthogonalisation --

MUON_COEFFS = (3.4445, -4.7750, 2.0315)


@_once
def _ortho_call(batch, rows, cols, dtype, steps, a, b, c, eps):
    d = _OrthoDesc(batch, rows, cols, _FLOATS[dtype], steps, a, b, c, eps)
    return d, int(_L().conv_orthogonalize_ws_bytes(d))


def _ortho_of(batch, rows, cols, dtype, steps, a, b, c, eps):
    """(description, scratch bytes) of the update."""
    return _ortho_call(batch, rows, cols, dtype, index(steps), float(a), float(b), float(c), float(eps))


def orthogonalize_ws_bytes(batch: int, rows: int, cols: int) -> int:
    """Bytes of ``ws`` that orthogonalize takes for [batch, rows, cols]."""
    return _need(_ortho_call(index(batch), index(rows), index(cols), torch.float32, 1, 1.0, 0.0, 0.0, 0.0)[1],
                 "conv_orthogonalize_ws_bytes")


def orthogonalize(g: torch.Tensor, steps: int = 5, coeffs: Sequence[float] = MUON_COEFFS, eps: float = 1e-7,
                  out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The Newton-Schulz orthogonalisation of g, bfloat16 in g's shape: g
    [m, n], a batch [b, m, n] of matrices, or one layer's OHWI weight gradient
    [c_out, kh, kw, c_in] as the matrix [c_out, kh kw c_in]."""
    if stream is not None:
        with _on(stream, g):
            return orthogonalize(g, steps, coeffs, eps, out, ws)
    if g.dim() < 2 or g.dtype not in _FLOATS:
        raise ValueError("g must be float32 or bfloat16, [m, n], [batch, m, n] or OHWI [c_out, kh, kw, c_in]")
    shape = g.shape
    _dev(g, "g", g.dtype, shape)
    if len(shape) == 3:
        batch, rows, cols = shape
    else:
        batch, rows = 1, shape[0]
        cols = g.numel() // rows if rows else 0
    a, b, c = coeffs
    d, need = _ortho_of(batch, rows, cols, g.dtype, steps, a, b, c, eps)
    if out is None:
        out = torch.empty_like(g, dtype=torch.bfloat16)
    else:
        _dev(out, "out", torch.bfloat16, shape)
    ws, at, size = _scratch(need, ws, g, "conv_orthogonalize")
    st = _L().conv_orthogonalize(d, g.data_ptr(), out.data_ptr(), at, size, _stream(g))
    if st:
        _lib._check(st, "conv_orthogonalize")
    return out
