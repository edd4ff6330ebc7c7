"""Argument checks of the operators around the layer (delta rule, rotary
positions, layer norm) through the C ABI: every refusal comes back as a status
before anything is enqueued, so no GPU is needed.  Pointers are plain numbers
here; nothing reads them."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import recon_chunk_ttt_b200 as R  # noqa: E402
from recon_chunk_ttt_b200 import _ops  # noqa: E402
from recon_chunk_ttt_b200 import build as _build  # noqa: E402

_build.build()
L = _ops._lib()
P = 1 << 20  # an aligned address that is never used


def _cfg(**kw):
    c = R.make_delta_config(4, 128, qk_heads=2)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _tok(n=10, seqs=1, **kw):
    t = R.ttt_delta_tokens()
    t.Q = t.K = t.V = t.log_decay = t.beta = P
    t.ldq = t.ldk = 256
    t.ldv = 512
    t.n, t.seqs = n, seqs
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def _chunk(cfg, tok, S_in=P, S_out=P, O=P, ws=P, nbytes=1 << 40):
    return L.ttt_delta_chunk(ctypes.byref(cfg), ctypes.byref(tok), S_in, S_out, O, ws, nbytes, None)


BAD_CFG = [(dict(heads=0), R.TTT_ERR_INVALID_ARG), (dict(qk_heads=3), R.TTT_ERR_INVALID_ARG),
           (dict(qk_heads=0), R.TTT_ERR_INVALID_ARG), (dict(d=96), R.TTT_ERR_UNSUPPORTED_SHAPE),
           (dict(precision=7), R.TTT_ERR_INVALID_ARG),
           (dict(scale=float("nan")), R.TTT_ERR_INVALID_ARG),
           (dict(scale=float("inf")), R.TTT_ERR_INVALID_ARG)]
BAD_TOK = [(dict(Q=None), R.TTT_ERR_INVALID_ARG), (dict(beta=None), R.TTT_ERR_INVALID_ARG),
           (dict(n=-1), R.TTT_ERR_INVALID_ARG), (dict(ldq=255), R.TTT_ERR_INVALID_ARG),
           (dict(ldq=257), R.TTT_ERR_ALIGNMENT), (dict(ldv=516), R.TTT_ERR_ALIGNMENT),
           (dict(K=P + 8), R.TTT_ERR_ALIGNMENT), (dict(log_decay=P + 2), R.TTT_ERR_ALIGNMENT),
           (dict(seqs=2), R.TTT_ERR_INVALID_ARG), (dict(seqs=-1), R.TTT_ERR_INVALID_ARG),
           (dict(offsets=P + 4), R.TTT_ERR_ALIGNMENT), (dict(seqs=70000), R.TTT_ERR_INVALID_ARG)]


@pytest.mark.parametrize("bad,want", BAD_CFG)
def test_delta_config_refused(bad, want):
    c = _cfg(**bad)
    assert _chunk(c, _tok()) == want
    assert R.ttt_delta_workspace_bytes(c, 10) == 0
    assert L.ttt_delta_backward(ctypes.byref(c), ctypes.byref(_tok()), *[P] * 10, 1 << 40, None) == want


@pytest.mark.parametrize("bad,want", BAD_TOK)
def test_delta_tokens_refused(bad, want):
    t = _tok(**bad)
    assert _chunk(_cfg(), t) == want
    assert L.ttt_delta_backward(ctypes.byref(_cfg()), ctypes.byref(t), *[P] * 10, 1 << 40, None) == want


def test_delta_outputs_and_workspace_refused():
    c, t = _cfg(), _tok()
    assert _chunk(c, t, O=None) == R.TTT_ERR_INVALID_ARG
    assert _chunk(c, t, S_in=P + 4) == R.TTT_ERR_ALIGNMENT
    assert _chunk(c, _tok(n=100), ws=None) == R.TTT_ERR_WORKSPACE
    t = _tok(n=100)
    need = R.ttt_delta_workspace_bytes(c, 100)
    assert need > 0 and _chunk(c, t, nbytes=need - 1) == R.TTT_ERR_WORKSPACE
    back = [P] * 10
    for i in (1, 3, 4, 5, 6, 7):  # dO, dQ, dK, dV, dlog_decay, dbeta
        a = list(back)
        a[i] = None
        assert L.ttt_delta_backward(ctypes.byref(c), ctypes.byref(t), *a, 1 << 40, None) == \
            R.TTT_ERR_INVALID_ARG
    need = R.ttt_delta_workspace_bytes(c, 100, 1, True)
    assert L.ttt_delta_backward(ctypes.byref(c), ctypes.byref(t), *back, need - 1, None) == \
        R.TTT_ERR_WORKSPACE


def test_delta_step_refused():
    def step(c=_cfg(), slots=P, pool=10, S=P, So=P, O=P, **kw):
        kw.setdefault("seqs", 10)
        return L.ttt_delta_step(ctypes.byref(c), ctypes.byref(_tok(**kw)), slots, pool, S, So, O, None)
    assert step(seqs=9) == R.TTT_ERR_INVALID_ARG
    assert step(offsets=P) == R.TTT_ERR_INVALID_ARG
    assert step(pool=-1) == R.TTT_ERR_INVALID_ARG
    assert step(slots=None, pool=9) == R.TTT_ERR_INVALID_ARG
    assert step(S=None) == R.TTT_ERR_INVALID_ARG
    assert step(O=None) == R.TTT_ERR_INVALID_ARG
    assert step(slots=P + 2) == R.TTT_ERR_ALIGNMENT
    assert step(S=P + 4) == R.TTT_ERR_ALIGNMENT
    assert step(n=0, seqs=0, O=None) == R.TTT_OK


def _rope(cfg, Q=P, ldq=256, hq=2, K=P, ldk=256, hk=2, pos=P, n=5, Qo=2 * P, ldqo=256, Ko=2 * P,
          ldko=256):
    return L.ttt_rope(ctypes.byref(cfg), Q, ldq, hq, K, ldk, hk, pos, n, Qo, ldqo, Ko, ldko, 0, None)


@pytest.mark.parametrize("bad,want", [
    (dict(rot=(31, 32, 32)), R.TTT_ERR_INVALID_ARG), (dict(rot=(0, 0, 0)), R.TTT_ERR_INVALID_ARG),
    (dict(rot=(64, 64, 2)), R.TTT_ERR_INVALID_ARG), (dict(rot=(-2, 64, 2)), R.TTT_ERR_INVALID_ARG),
    (dict(base=0.5), R.TTT_ERR_INVALID_ARG), (dict(base=float("inf")), R.TTT_ERR_INVALID_ARG),
    (dict(layout=2), R.TTT_ERR_INVALID_ARG), (dict(freq=-1), R.TTT_ERR_INVALID_ARG),
    (dict(d=80), R.TTT_ERR_UNSUPPORTED_SHAPE), (dict(precision=3), R.TTT_ERR_INVALID_ARG)])
def test_rope_config_refused(bad, want):
    kw = dict(d=128, rot=(32, 48, 48))
    kw.update(bad)
    assert _rope(R.make_rope_config(**kw)) == want


@pytest.mark.parametrize("bad,want", [
    (dict(n=-1), R.TTT_ERR_INVALID_ARG), (dict(hq=0), R.TTT_ERR_INVALID_ARG),
    (dict(Q=None), R.TTT_ERR_INVALID_ARG), (dict(pos=None), R.TTT_ERR_INVALID_ARG),
    (dict(hk=0), R.TTT_ERR_INVALID_ARG), (dict(K=None), R.TTT_ERR_INVALID_ARG),
    (dict(ldq=128), R.TTT_ERR_INVALID_ARG), (dict(ldko=128), R.TTT_ERR_INVALID_ARG),
    (dict(ldq=260), R.TTT_ERR_ALIGNMENT), (dict(Qo=2 * P + 8), R.TTT_ERR_ALIGNMENT),
    (dict(pos=P + 2), R.TTT_ERR_ALIGNMENT), (dict(Qo=P, ldqo=512), R.TTT_ERR_INVALID_ARG),
    (dict(n=0, Q=None), R.TTT_OK)])
def test_rope_arguments_refused(bad, want):
    assert _rope(R.make_rope_config(128, (32, 48, 48)), **bad) == want


def test_norm_refused():
    c = R.make_norm_config(64)
    fwd = lambda c, X=P, ldx=64, rows=3, w=P, b=P, Y=2 * P, st=P: L.ttt_layer_norm(  # noqa: E731
        ctypes.byref(c), X, ldx, rows, w, b, Y, st, None)
    assert fwd(R.make_norm_config(0)) == R.TTT_ERR_UNSUPPORTED_SHAPE
    assert fwd(R.make_norm_config(65537), ldx=70000) == R.TTT_ERR_UNSUPPORTED_SHAPE
    assert fwd(R.make_norm_config(64, eps=-1.0)) == R.TTT_ERR_INVALID_ARG
    assert fwd(R.make_norm_config(64, eps=float("nan"))) == R.TTT_ERR_INVALID_ARG
    assert fwd(R.make_norm_config(64, precision=9)) == R.TTT_ERR_INVALID_ARG
    assert fwd(c, X=None) == R.TTT_ERR_INVALID_ARG
    assert fwd(c, Y=None) == R.TTT_ERR_INVALID_ARG
    assert fwd(c, ldx=63) == R.TTT_ERR_INVALID_ARG
    assert fwd(c, rows=-1) == R.TTT_ERR_INVALID_ARG
    assert fwd(c, Y=P, ldx=128) == R.TTT_ERR_INVALID_ARG
    assert fwd(c, w=P + 4) == R.TTT_ERR_ALIGNMENT
    assert fwd(c, rows=0, X=None) == R.TTT_OK
    need = R.ttt_norm_workspace_bytes(c, 3)
    back = lambda X=P, ldx=64, dY=P, lddy=64, rows=3, w=P, st=P, dX=3 * P, dw=P, db=P, ws=P, \
        nb=need: L.ttt_layer_norm_backward(ctypes.byref(c), X, ldx, dY, lddy, rows, w, st,  # noqa: E731
                                           dX, dw, db, ws, nb, None)
    assert back(dX=None, dw=None, db=None) == R.TTT_ERR_INVALID_ARG
    assert back(st=None) == R.TTT_ERR_INVALID_ARG
    assert back(lddy=10) == R.TTT_ERR_INVALID_ARG
    assert back(dX=P, ldx=128) == R.TTT_ERR_INVALID_ARG
    assert back(ws=None) == R.TTT_ERR_WORKSPACE
    assert back(nb=need - 1) == R.TTT_ERR_WORKSPACE
    assert back(dY=P + 2) == R.TTT_ERR_ALIGNMENT


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    g = torch.zeros(4, 4)
    with pytest.raises(R.TTTError):
        R.ttt_delta_chunk(_cfg(), x, x, x, g, g)
    with pytest.raises(R.TTTError):
        R.ttt_layer_norm(R.make_norm_config(256), x)
