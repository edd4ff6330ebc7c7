"""ctypes binding of the operators around the layer (include/ttt.h): the gated
delta rule, rotary positions over three axes and layer norm.

Like the layer's binding this marshals arguments and allocates outputs that
are not given; types, shapes, strides and devices are checked here because the
C function sees plain pointers (TTTError with TTT_ERR_INVALID_ARG), the rest in
the library.  Work goes to the tensors' device, on `stream` or that device's
current stream; what a call allocates belongs to that stream.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import _binding as B

_P, _I32, _I64, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t


class ttt_delta_config(ctypes.Structure):
    _fields_ = [("heads", _I32), ("qk_heads", _I32), ("d", _I32), ("precision", _I32),
                ("scale", ctypes.c_float)]


class ttt_delta_tokens(ctypes.Structure):
    _fields_ = [("Q", _P), ("K", _P), ("V", _P), ("log_decay", _P), ("beta", _P), ("ldq", _I64),
                ("ldk", _I64), ("ldv", _I64), ("n", _I64), ("offsets", _P), ("seqs", _I64)]


# the same as bytes: a struct of this size is faster packed than filled field by field
_pack_tokens = struct.Struct("=QQQQQqqqqQq").pack


class ttt_rope_config(ctypes.Structure):
    _fields_ = [("d", _I32), ("rot", _I32 * 3), ("base", ctypes.c_float * 3), ("layout", _I32),
                ("freq", _I32), ("precision", _I32)]


class ttt_norm_config(ctypes.Structure):
    _fields_ = [("dim", _I64), ("eps", ctypes.c_float), ("precision", _I32)]


_F32 = torch.float32
DEVICE_ERR_OFFSETS = 8  # TTT_DEVICE_ERR_OFFSETS
ROPE_HALF, ROPE_PAIRS = 0, 1
ROPE_FREQ_AXIS, ROPE_FREQ_HEAD = 0, 1

_typed = None


def _lib():
    global _typed
    if _typed is None:
        L = B.lib()
        dc, dt = ctypes.POINTER(ttt_delta_config), _P  # dt: a ttt_delta_tokens, or its bytes
        rc, nc = ctypes.POINTER(ttt_rope_config), ctypes.POINTER(ttt_norm_config)
        for name, args, res in (
                ("ttt_delta_workspace_bytes", [dc, _I64, _I64, _I32], _SZ),
                ("ttt_delta_chunk", [dc, dt, _P, _P, _P, _P, _SZ, _P], ctypes.c_int),
                ("ttt_delta_step", [dc, dt, _P, _I64, _P, _P, _P, _P], ctypes.c_int),
                ("ttt_delta_backward", [dc, dt] + [_P] * 10 + [_SZ, _P], ctypes.c_int),
                ("ttt_rope", [rc, _P, _I64, _I32, _P, _I64, _I32, _P, _I64, _P, _I64, _P, _I64,
                              _I32, _P], ctypes.c_int),
                ("ttt_norm_workspace_bytes", [nc, _I64], _SZ),
                ("ttt_layer_norm", [nc, _P, _I64, _I64, _P, _P, _P, _P, _P], ctypes.c_int),
                ("ttt_layer_norm_backward", [nc, _P, _I64, _P, _I64, _I64, _P, _P, _P, _P, _P, _P,
                                             _SZ, _P], ctypes.c_int)):
            f = getattr(L, name)
            f.argtypes, f.restype = args, res
        _typed = L
    return _typed


def _want(ok, what, why):
    if not ok:
        raise B.TTTError(B.TTT_ERR_INVALID_ARG, f"{what}: {why}")


def _token(precision):
    return torch.float32 if precision == B.PREC_FP32_CHECK else torch.bfloat16


def _device(what, t):
    """The index of the GPU a call's first tensor is on; every other tensor
    must be there too."""
    _want(isinstance(t, torch.Tensor) and t.is_cuda, what, "tensors must be on a GPU")
    return t.get_device()


def _check(what, dev, name, t, dtype, shape, rows=False):
    """The tensor's pointer.  `rows`: a matrix whose rows may lie apart.  One-token
    calls cost microseconds: the messages are put together only when one is due."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev:
        if t.is_contiguous():
            return t.data_ptr()
        if rows:
            _want(t.stride(1) == 1 or shape[1] <= 1, what, f"{name}: a row's values lie apart")
            _want(shape[0] <= 1 or t.stride(0) >= shape[1], what, f"{name}: rows overlap")
            return t.data_ptr()
    _want(t.get_device() == dev, what, f"{name} is on {t.device}, not on GPU {dev}")
    _want(t.dtype == dtype, what, f"{name} is {t.dtype}, not {dtype}")
    _want(t.shape == shape, what, f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    _want(False, what, f"{name} is not contiguous")


def _maybe(what, dev, name, t, dtype, shape):
    return None if t is None else _check(what, dev, name, t, dtype, shape)


def _out(what, dev, name, t, dtype, shape, like):
    """An output and its pointer; allocated if it is not given, from a tensor on
    the same device (`like`: of its type and shape, or at least its type)."""
    if t is None:
        t = torch.empty_like(like) if like.shape == shape and like.is_contiguous() \
            else like.new_empty(shape)
        return t, t.data_ptr()
    return t, _check(what, dev, name, t, dtype, shape)


def _space(what, dev, t, nbytes):
    if t is None:
        t = torch.empty(max(nbytes(), 1), dtype=torch.uint8, device=dev)
    _want(t.get_device() == dev and t.is_contiguous(), what,
          "workspace must be contiguous, on the tensors' device")
    return t, t.data_ptr(), t.numel() * t.element_size()


def _on(what, t, stream):
    """`stream` (a torch stream or a handle) as the current one.  What the call then
    allocates belongs to that stream: its memory is not another stream's again while
    the call's work may still use it."""
    dev = _device(what, t)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=dev) if stream else \
            torch.cuda.default_stream(dev)
    _want(stream.device.index == dev, what, f"stream is on {stream.device}, not on GPU {dev}")
    return torch.cuda.stream(stream)


def _run(what, dev, fn, args):
    """The library's call with the tensors' device current, on that device's
    current stream."""
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return _run(what, dev, fn, args)
    status = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if status != B.TTT_OK:
        raise B.TTTError(status, what)


def _ld(t):
    """Elements between rows (a single row's stride may be anything)."""
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


# ------------------------------------------------------------------ delta rule
def make_delta_config(heads: int, d: int, qk_heads: int | None = None, scale: float | None = None,
                      precision: int = B.PREC_BF16_TC) -> ttt_delta_config:
    """`scale` is the factor of the read; 1/sqrt(d) unless given."""
    return ttt_delta_config(heads, heads if qk_heads is None else qk_heads, d, precision,
                            d ** -0.5 if scale is None else scale)


def ttt_delta_workspace_bytes(cfg: ttt_delta_config, n: int, seqs: int = 1,
                              backward: bool = False) -> int:
    return int(_lib().ttt_delta_workspace_bytes(ctypes.byref(cfg), int(n), int(seqs),
                                                1 if backward else 0))


def alloc_delta_workspace(cfg: ttt_delta_config, n: int, seqs: int = 1, backward: bool = False,
                          device=None) -> torch.Tensor:
    nbytes = ttt_delta_workspace_bytes(cfg, n, seqs, backward)
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device or "cuda")


def _sequences(what, offsets):
    if offsets is None:
        return 1
    _want(offsets.dim() == 1 and offsets.shape[0] > 0, what, "offsets must be [seqs + 1]")
    return offsets.shape[0] - 1


def _delta_tokens(what, cfg, Q, K, V, log_decay, beta, offsets, seqs):
    """(device, tokens of the call as bytes, their number, token type)."""
    dev, tdt = _device(what, Q), _token(cfg.precision)
    n, heads, d = Q.shape[0], cfg.heads, cfg.d
    qk, per = (n, cfg.qk_heads * d), (n, heads)
    return dev, _pack_tokens(
        _check(what, dev, "Q", Q, tdt, qk, True), _check(what, dev, "K", K, tdt, qk, True),
        _check(what, dev, "V", V, tdt, (n, heads * d), True),
        _check(what, dev, "log_decay", log_decay, _F32, per),
        _check(what, dev, "beta", beta, _F32, per), _ld(Q), _ld(K), _ld(V), n,
        0 if offsets is None else _check(what, dev, "offsets", offsets, torch.int64, (seqs + 1,)),
        seqs), n, tdt


def ttt_delta_chunk(cfg: ttt_delta_config, Q, K, V, log_decay, beta, S=None, offsets=None,
                    S_out=None, O=None, workspace=None, stream=None):
    """The gated delta rule over packed sequences (offsets int64 [seqs + 1] on
    the device, or one sequence); returns (O, S_out).  S_out may be S."""
    what = "ttt_delta_chunk"
    if stream is not None:
        with _on(what, Q, stream):
            return ttt_delta_chunk(cfg, Q, K, V, log_decay, beta, S, offsets, S_out, O, workspace)
    seqs = _sequences(what, offsets)
    dev, t, n, tdt = _delta_tokens(what, cfg, Q, K, V, log_decay, beta, offsets, seqs)
    shape = (seqs, cfg.heads, cfg.d, cfg.d)
    pS = _maybe(what, dev, "S", S, _F32, shape)
    S_out, pSo = _out(what, dev, "S_out", S_out, _F32, shape, beta if S is None else S)
    O, pO = _out(what, dev, "O", O, tdt, (n, cfg.heads * cfg.d), V)
    workspace, pW, nbytes = _space(what, dev, workspace,
                                   lambda: ttt_delta_workspace_bytes(cfg, n, seqs))
    _run(what, dev, _lib().ttt_delta_chunk, (ctypes.byref(cfg), t, pS, pSo, pO, pW, nbytes))
    return O, S_out


def ttt_delta_step(cfg: ttt_delta_config, Q, K, V, log_decay, beta, S, slots=None, S_out=None,
                   O=None, stream=None):
    """One token for each request on a pool of states S [pool, heads, d, d]
    (slots: int32 [n], -1 for padding; without them request i has state i).
    The new states go to S_out, or into S where that is not given; returns O."""
    what = "ttt_delta_step"
    if stream is not None:
        with _on(what, Q, stream):
            return ttt_delta_step(cfg, Q, K, V, log_decay, beta, S, slots, S_out, O)
    dev, t, n, tdt = _delta_tokens(what, cfg, Q, K, V, log_decay, beta, None, Q.shape[0])
    _want(isinstance(S, torch.Tensor) and S.dim() == 4, what, "S must be [pool, heads, d, d]")
    pool = S.shape[0]
    shape = (pool, cfg.heads, cfg.d, cfg.d)
    pS = _check(what, dev, "S", S, _F32, shape)
    pSo = pS if S_out is None else _check(what, dev, "S_out", S_out, _F32, shape)
    pI = _maybe(what, dev, "slots", slots, torch.int32, (n,))
    O, pO = _out(what, dev, "O", O, tdt, (n, cfg.heads * cfg.d), V)
    _run(what, dev, _lib().ttt_delta_step, (ctypes.byref(cfg), t, pI, pool, pS, pSo, pO))
    return O


def ttt_delta_backward(cfg: ttt_delta_config, Q, K, V, log_decay, beta, dO, S=None, offsets=None,
                       dS_out=None, dQ=None, dK=None, dV=None, dlog_decay=None, dbeta=None,
                       dS=None, workspace=None, stream=None):
    """Gradients of sum(dO * O) + sum(dS_out * S_out) of ttt_delta_chunk:
    (dQ, dK, dV, dlog_decay, dbeta, dS).  dS may be dS_out."""
    what = "ttt_delta_backward"
    if stream is not None:
        with _on(what, Q, stream):
            return ttt_delta_backward(cfg, Q, K, V, log_decay, beta, dO, S, offsets, dS_out, dQ, dK, dV,
                                      dlog_decay, dbeta, dS, workspace)
    seqs = _sequences(what, offsets)
    dev, t, n, tdt = _delta_tokens(what, cfg, Q, K, V, log_decay, beta, offsets, seqs)
    qk, hv, per = (n, cfg.qk_heads * cfg.d), (n, cfg.heads * cfg.d), (n, cfg.heads)
    shape = (seqs, cfg.heads, cfg.d, cfg.d)
    pS = _maybe(what, dev, "S", S, _F32, shape)
    pG = _check(what, dev, "dO", dO, tdt, hv)
    pE = _maybe(what, dev, "dS_out", dS_out, _F32, shape)
    dQ, p1 = _out(what, dev, "dQ", dQ, tdt, qk, Q)
    dK, p2 = _out(what, dev, "dK", dK, tdt, qk, K)
    dV, p3 = _out(what, dev, "dV", dV, tdt, hv, dO)
    dlog_decay, p4 = _out(what, dev, "dlog_decay", dlog_decay, _F32, per, beta)
    dbeta, p5 = _out(what, dev, "dbeta", dbeta, _F32, per, beta)
    dS, p6 = _out(what, dev, "dS", dS, _F32, shape, beta if S is None else S)
    workspace, pW, nbytes = _space(what, dev, workspace,
                                   lambda: ttt_delta_workspace_bytes(cfg, n, seqs, True))
    _run(what, dev, _lib().ttt_delta_backward,
         (ctypes.byref(cfg), t, pS, pG, pE, p1, p2, p3, p4, p5, p6, pW, nbytes))
    return dQ, dK, dV, dlog_decay, dbeta, dS


# ------------------------------------------------------------------ rotary positions
def make_rope_config(d: int, rot, base=10000.0, layout: int = ROPE_HALF,
                     freq: int = ROPE_FREQ_AXIS, precision: int = B.PREC_BF16_TC) -> ttt_rope_config:
    """`rot`: values of a head rotated by (time, height, width), each even;
    `base`: one number, or one for each axis."""
    bases = tuple(base) if hasattr(base, "__len__") else (base,) * 3
    return ttt_rope_config(d, (_I32 * 3)(*rot), (ctypes.c_float * 3)(*bases), layout, freq,
                           precision)


def ttt_rope(cfg: ttt_rope_config, Q, K, positions, Q_out=None, K_out=None, inverse: bool = False,
             stream=None):
    """Rotate the heads of Q [n, q_heads*d] and K [n, k_heads*d] (or None) by
    positions float [n, 3]; returns (Q_out, K_out).  Q_out may be Q and K_out
    K.  inverse=True turns back: the gradient."""
    what = "ttt_rope"
    if stream is not None:
        with _on(what, Q, stream):
            return ttt_rope(cfg, Q, K, positions, Q_out, K_out, inverse)
    dev, tdt = _device(what, Q), _token(cfg.precision)
    n = Q.shape[0]

    def side(name, x, y):
        """(heads, input pointer and row distance, output, its pointer and distance)"""
        if x is None:
            _want(y is None, what, f"{name}_out without {name}")
            return 0, None, 0, None, None, 0
        _want(x.dim() == 2 and x.shape[1] % cfg.d == 0, what, f"{name} must be [n, heads * d]")
        w = x.shape[1]
        p = _check(what, dev, name, x, tdt, (n, w), True)
        if y is None:
            y = torch.empty_like(x) if x.is_contiguous() else x.new_empty((n, w))
            return w // cfg.d, p, _ld(x), y, y.data_ptr(), w
        return w // cfg.d, p, _ld(x), y, _check(what, dev, name + "_out", y, tdt, (n, w), True), _ld(y)

    hq, pQ, lq, Q_out, pQo, lqo = side("Q", Q, Q_out)
    hk, pK, lk, K_out, pKo, lko = side("K", K, K_out)
    pP = _check(what, dev, "positions", positions, _F32, (n, 3))
    _run(what, dev, _lib().ttt_rope, (ctypes.byref(cfg), pQ, lq, hq, pK, lk, hk, pP, n, pQo, lqo, pKo,
                                      lko, 1 if inverse else 0))
    return Q_out, K_out


# ------------------------------------------------------------------ layer norm
def make_norm_config(dim: int, eps: float = 1e-5,
                     precision: int = B.PREC_BF16_TC) -> ttt_norm_config:
    return ttt_norm_config(dim, eps, precision)


def ttt_norm_workspace_bytes(cfg: ttt_norm_config, rows: int) -> int:
    return int(_lib().ttt_norm_workspace_bytes(ctypes.byref(cfg), int(rows)))


def ttt_layer_norm(cfg: ttt_norm_config, X, weight=None, bias=None, Y=None, stats=None,
                   stream=None):
    """Layer norm of the rows of X [rows, dim]; returns (Y, stats), stats
    float [rows, 2] holding each row's mean and 1/sqrt(var + eps)."""
    what = "ttt_layer_norm"
    if stream is not None:
        with _on(what, X, stream):
            return ttt_layer_norm(cfg, X, weight, bias, Y, stats)
    dev, tdt = _device(what, X), _token(cfg.precision)
    dim = cfg.dim
    rows = X.shape[0]
    pX = _check(what, dev, "X", X, tdt, (rows, dim), True)
    pw = _maybe(what, dev, "weight", weight, _F32, (dim,))
    pb = _maybe(what, dev, "bias", bias, _F32, (dim,))
    Y, pY = _out(what, dev, "Y", Y, tdt, (rows, dim), X)
    if stats is None:
        stats = torch.empty((rows, 2), dtype=_F32, device=X.device)
    ps = _check(what, dev, "stats", stats, _F32, (rows, 2))
    _run(what, dev, _lib().ttt_layer_norm, (ctypes.byref(cfg), pX, _ld(X), rows, pw, pb, pY, ps))
    return Y, stats


def ttt_layer_norm_backward(cfg: ttt_norm_config, X, dY, stats, weight=None, dX=None,
                            dweight=None, dbias=None, workspace=None, stream=None):
    """(dX, dweight, dbias) from the forward call's X and stats."""
    what = "ttt_layer_norm_backward"
    if stream is not None:
        with _on(what, X, stream):
            return ttt_layer_norm_backward(cfg, X, dY, stats, weight, dX, dweight, dbias, workspace)
    dev, tdt = _device(what, X), _token(cfg.precision)
    dim = cfg.dim
    rows = X.shape[0]
    pX = _check(what, dev, "X", X, tdt, (rows, dim), True)
    pY = _check(what, dev, "dY", dY, tdt, (rows, dim), True)
    ps = _check(what, dev, "stats", stats, _F32, (rows, 2))
    pw = _maybe(what, dev, "weight", weight, _F32, (dim,))
    dX, p1 = _out(what, dev, "dX", dX, tdt, (rows, dim), X)
    dweight, p2 = _out(what, dev, "dweight", dweight, _F32, (dim,), stats if weight is None else weight)
    dbias, p3 = _out(what, dev, "dbias", dbias, _F32, (dim,), dweight)
    workspace, pW, nbytes = _space(what, dev, workspace, lambda: ttt_norm_workspace_bytes(cfg, rows))
    _run(what, dev, _lib().ttt_layer_norm_backward,
         (ctypes.byref(cfg), pX, _ld(X), pY, _ld(dY), rows, pw, ps, p1, p2, p3, pW, nbytes))
    return dX, dweight, dbias
