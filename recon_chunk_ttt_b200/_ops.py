"""ctypes binding of the operators around the layer (include/ttt.h): the gated
delta rule, rotary positions over three axes and layer norm.

Like the layer's binding this marshals arguments and allocates outputs that
are not given; types, shapes, strides and devices are checked here because the
C function sees plain pointers (TTTError with TTT_ERR_INVALID_ARG), the rest in
the library.  Work goes to the tensors' device, on `stream` or that device's
current stream.
"""
from __future__ import annotations

import ctypes

import torch

from . import _binding as B

_P, _I32, _I64, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t


class ttt_delta_config(ctypes.Structure):
    _fields_ = [("heads", _I32), ("qk_heads", _I32), ("d", _I32), ("precision", _I32),
                ("scale", ctypes.c_float)]


class ttt_delta_tokens(ctypes.Structure):
    _fields_ = [("Q", _P), ("K", _P), ("V", _P), ("log_decay", _P), ("beta", _P), ("ldq", _I64),
                ("ldk", _I64), ("ldv", _I64), ("n", _I64), ("offsets", _P), ("seqs", _I64)]


class ttt_rope_config(ctypes.Structure):
    _fields_ = [("d", _I32), ("rot", _I32 * 3), ("base", ctypes.c_float * 3), ("layout", _I32),
                ("freq", _I32), ("precision", _I32)]


class ttt_norm_config(ctypes.Structure):
    _fields_ = [("dim", _I64), ("eps", ctypes.c_float), ("precision", _I32)]


DEVICE_ERR_OFFSETS = 8  # TTT_DEVICE_ERR_OFFSETS
ROPE_HALF, ROPE_PAIRS = 0, 1
ROPE_FREQ_AXIS, ROPE_FREQ_HEAD = 0, 1

_typed = False


def _lib():
    global _typed
    L = B.lib()
    if not _typed:
        dc, dt = ctypes.POINTER(ttt_delta_config), ctypes.POINTER(ttt_delta_tokens)
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
        _typed = True
    return L


def _want(ok, what, why):
    if not ok:
        raise B.TTTError(B.TTT_ERR_INVALID_ARG, f"{what}: {why}")


def _token(precision):
    return torch.float32 if precision == B.PREC_FP32_CHECK else torch.bfloat16


class _Call:
    """One call's checks: every tensor on the first one's device, of its type
    and shape; the device is made current around the library's call."""

    def __init__(self, what, first):
        self.what = what
        _want(isinstance(first, torch.Tensor) and first.is_cuda, what, "tensors must be on a GPU")
        self.device = first.device

    def check(self, name, t, dtype, shape, optional=False, rows=False):
        """The tensor's pointer.  `rows`: a matrix whose rows may lie apart."""
        if t is None:
            _want(optional, self.what, f"{name} is missing")
            return None
        _want(t.device == self.device, self.what, f"{name} is on {t.device}, not {self.device}")
        _want(t.dtype == dtype, self.what, f"{name} is {t.dtype}, not {dtype}")
        _want(tuple(t.shape) == tuple(shape), self.what,
              f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
        if rows:
            _want(t.stride(1) == 1 or t.shape[1] <= 1, self.what, f"{name}: a row's values lie apart")
            _want(t.shape[0] <= 1 or t.stride(0) >= t.shape[1], self.what, f"{name}: rows overlap")
        else:
            _want(t.is_contiguous(), self.what, f"{name} is not contiguous")
        return t.data_ptr()

    def out(self, name, t, dtype, shape):
        if t is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        self.check(name, t, dtype, shape)
        return t

    def workspace(self, t, nbytes):
        if t is None:
            t = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=self.device)
        _want(t.device == self.device and t.is_contiguous(), self.what,
              "workspace must be contiguous, on the tensors' device")
        return t, t.numel() * t.element_size()

    def run(self, fn, args, stream):
        with torch.cuda.device(self.device):
            st = torch.cuda.current_stream().cuda_stream if stream is None else B._stream(stream)
            B._check(fn(*args, st), self.what)


def _ld(t):
    """Elements between rows (a single row's stride may be anything)."""
    return int(t.stride(0)) if t.shape[0] > 1 else max(int(t.shape[1]), 1)


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


def _delta_tokens(c, cfg, Q, K, V, log_decay, beta, offsets, seqs):
    n, tdt = int(Q.shape[0]), _token(cfg.precision)
    qk, hv = cfg.qk_heads * cfg.d, cfg.heads * cfg.d
    t = ttt_delta_tokens()
    t.Q = c.check("Q", Q, tdt, (n, qk), rows=True)
    t.K = c.check("K", K, tdt, (n, qk), rows=True)
    t.V = c.check("V", V, tdt, (n, hv), rows=True)
    t.log_decay = c.check("log_decay", log_decay, torch.float32, (n, cfg.heads))
    t.beta = c.check("beta", beta, torch.float32, (n, cfg.heads))
    t.ldq, t.ldk, t.ldv, t.n = _ld(Q), _ld(K), _ld(V), n
    if offsets is not None:
        t.offsets = c.check("offsets", offsets, torch.int64, (seqs + 1,))
    t.seqs = seqs
    return t


def ttt_delta_chunk(cfg: ttt_delta_config, Q, K, V, log_decay, beta, S=None, offsets=None,
                    S_out=None, O=None, workspace=None, stream=None):
    """The gated delta rule over packed sequences (offsets int64 [seqs + 1] on
    the device, or one sequence); returns (O, S_out).  S_out may be S."""
    c = _Call("ttt_delta_chunk", Q)
    seqs = 1 if offsets is None else int(offsets.shape[0]) - 1
    t = _delta_tokens(c, cfg, Q, K, V, log_decay, beta, offsets, seqs)
    shape = (seqs, cfg.heads, cfg.d, cfg.d)
    c.check("S", S, torch.float32, shape, optional=True)
    S_out = c.out("S_out", S_out, torch.float32, shape)
    O = c.out("O", O, _token(cfg.precision), (t.n, cfg.heads * cfg.d))
    ws, nbytes = c.workspace(workspace, ttt_delta_workspace_bytes(cfg, t.n, seqs)
                             if workspace is None else 0)
    c.run(_lib().ttt_delta_chunk, (ctypes.byref(cfg), ctypes.byref(t), B._ptr(S), B._ptr(S_out),
                                   B._ptr(O), B._ptr(ws), nbytes), stream)
    return O, S_out


def ttt_delta_step(cfg: ttt_delta_config, Q, K, V, log_decay, beta, S, slots=None, S_out=None,
                   O=None, stream=None):
    """One token for each request on a pool of states S [pool, heads, d, d]
    (slots: int32 [n], -1 for padding; without them request i has state i).
    The new states go to S_out, or into S where that is not given; returns O."""
    c = _Call("ttt_delta_step", Q)
    t = _delta_tokens(c, cfg, Q, K, V, log_decay, beta, None, int(Q.shape[0]))
    _want(isinstance(S, torch.Tensor) and S.dim() == 4, c.what, "S must be [pool, heads, d, d]")
    pool = int(S.shape[0])
    shape = (pool, cfg.heads, cfg.d, cfg.d)
    c.check("S", S, torch.float32, shape)
    S_out = S if S_out is None else c.out("S_out", S_out, torch.float32, shape)
    c.check("slots", slots, torch.int32, (t.n,), optional=True)
    O = c.out("O", O, _token(cfg.precision), (t.n, cfg.heads * cfg.d))
    c.run(_lib().ttt_delta_step, (ctypes.byref(cfg), ctypes.byref(t), B._ptr(slots), pool,
                                  B._ptr(S), B._ptr(S_out), B._ptr(O)), stream)
    return O


def ttt_delta_backward(cfg: ttt_delta_config, Q, K, V, log_decay, beta, dO, S=None, offsets=None,
                       dS_out=None, dQ=None, dK=None, dV=None, dlog_decay=None, dbeta=None,
                       dS=None, workspace=None, stream=None):
    """Gradients of sum(dO * O) + sum(dS_out * S_out) of ttt_delta_chunk:
    (dQ, dK, dV, dlog_decay, dbeta, dS).  dS may be dS_out."""
    c = _Call("ttt_delta_backward", Q)
    seqs = 1 if offsets is None else int(offsets.shape[0]) - 1
    t = _delta_tokens(c, cfg, Q, K, V, log_decay, beta, offsets, seqs)
    tdt, n = _token(cfg.precision), t.n
    shape = (seqs, cfg.heads, cfg.d, cfg.d)
    c.check("S", S, torch.float32, shape, optional=True)
    c.check("dO", dO, tdt, (n, cfg.heads * cfg.d))
    c.check("dS_out", dS_out, torch.float32, shape, optional=True)
    dQ = c.out("dQ", dQ, tdt, (n, cfg.qk_heads * cfg.d))
    dK = c.out("dK", dK, tdt, (n, cfg.qk_heads * cfg.d))
    dV = c.out("dV", dV, tdt, (n, cfg.heads * cfg.d))
    dlog_decay = c.out("dlog_decay", dlog_decay, torch.float32, (n, cfg.heads))
    dbeta = c.out("dbeta", dbeta, torch.float32, (n, cfg.heads))
    dS = c.out("dS", dS, torch.float32, shape)
    ws, nbytes = c.workspace(workspace, ttt_delta_workspace_bytes(cfg, n, seqs, True)
                             if workspace is None else 0)
    c.run(_lib().ttt_delta_backward,
          (ctypes.byref(cfg), ctypes.byref(t), B._ptr(S), B._ptr(dO), B._ptr(dS_out), B._ptr(dQ),
           B._ptr(dK), B._ptr(dV), B._ptr(dlog_decay), B._ptr(dbeta), B._ptr(dS), B._ptr(ws),
           nbytes), stream)
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
    c = _Call("ttt_rope", Q)
    n, tdt = int(Q.shape[0]), _token(cfg.precision)

    def side(name, x, y):
        if x is None:
            _want(y is None, c.what, f"{name}_out without {name}")
            return 0, None
        _want(x.dim() == 2 and x.shape[1] % cfg.d == 0, c.what, f"{name} must be [n, heads * d]")
        c.check(name, x, tdt, (n, int(x.shape[1])), rows=True)
        if y is None:
            y = torch.empty((n, int(x.shape[1])), dtype=tdt, device=c.device)
        else:
            c.check(name + "_out", y, tdt, (n, int(x.shape[1])), rows=True)
        return int(x.shape[1]) // cfg.d, y

    hq, Q_out = side("Q", Q, Q_out)
    hk, K_out = side("K", K, K_out)
    c.check("positions", positions, torch.float32, (n, 3))
    none = hk == 0
    c.run(_lib().ttt_rope,
          (ctypes.byref(cfg), B._ptr(Q), _ld(Q), hq, None if none else B._ptr(K),
           0 if none else _ld(K), hk, B._ptr(positions), n, B._ptr(Q_out), _ld(Q_out),
           None if none else B._ptr(K_out), 0 if none else _ld(K_out), 1 if inverse else 0), stream)
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
    c = _Call("ttt_layer_norm", X)
    rows, dim, tdt = int(X.shape[0]), int(cfg.dim), _token(cfg.precision)
    c.check("X", X, tdt, (rows, dim), rows=True)
    c.check("weight", weight, torch.float32, (dim,), optional=True)
    c.check("bias", bias, torch.float32, (dim,), optional=True)
    Y = c.out("Y", Y, tdt, (rows, dim))
    stats = c.out("stats", stats, torch.float32, (rows, 2))
    c.run(_lib().ttt_layer_norm, (ctypes.byref(cfg), B._ptr(X), _ld(X), rows, B._ptr(weight),
                                  B._ptr(bias), B._ptr(Y), B._ptr(stats)), stream)
    return Y, stats


def ttt_layer_norm_backward(cfg: ttt_norm_config, X, dY, stats, weight=None, dX=None,
                            dweight=None, dbias=None, workspace=None, stream=None):
    """(dX, dweight, dbias) from the forward call's X and stats."""
    c = _Call("ttt_layer_norm_backward", X)
    rows, dim, tdt = int(X.shape[0]), int(cfg.dim), _token(cfg.precision)
    c.check("X", X, tdt, (rows, dim), rows=True)
    c.check("dY", dY, tdt, (rows, dim), rows=True)
    c.check("stats", stats, torch.float32, (rows, 2))
    c.check("weight", weight, torch.float32, (dim,), optional=True)
    dX = c.out("dX", dX, tdt, (rows, dim))
    dweight = c.out("dweight", dweight, torch.float32, (dim,))
    dbias = c.out("dbias", dbias, torch.float32, (dim,))
    ws, nbytes = c.workspace(workspace, ttt_norm_workspace_bytes(cfg, rows)
                             if workspace is None else 0)
    c.run(_lib().ttt_layer_norm_backward,
          (ctypes.byref(cfg), B._ptr(X), _ld(X), B._ptr(dY), _ld(dY), rows, B._ptr(weight),
           B._ptr(stats), B._ptr(dX), B._ptr(dweight), B._ptr(dbias), B._ptr(ws), nbytes), stream)
    return dX, dweight, dbias
