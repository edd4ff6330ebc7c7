"""Outputs left out: what the C interface allows to be NULL, against the call that wants everything."""
import ctypes

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import recon_chunk_ttt_b200 as R  # noqa: E402
from recon_chunk_ttt_b200 import _ops  # noqa: E402
from test_gpu_delta import BF, F32, _dtype, _inputs, _offsets  # noqa: E402

L = _ops._lib()


def _p(t):
    return None if t is None else t.data_ptr()


def _stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("prec", [BF, F32])
@pytest.mark.parametrize("dim", [8, 30, 64, 1000, 1024, 1153, 4096, 8190, 20000])
def test_norm_gradient_in_parts(dim, prec):
    """dX alone needs no workspace; each column sum alone; no statistics from the forward call."""
    rows, t = 3001 if dim < 5000 else 130, _dtype(prec)
    x, dy = (torch.randn(rows, dim, device="cuda").to(t) for _ in range(2))
    w, b = torch.randn(dim, device="cuda"), torch.randn(dim, device="cuda")
    cfg = R.make_norm_config(dim, precision=prec)
    Y, st = R.ttt_layer_norm(cfg, x, w, b)
    want = R.ttt_layer_norm_backward(cfg, x, dy, st, w)
    y = torch.empty_like(x)
    assert L.ttt_layer_norm(ctypes.byref(cfg), _p(x), dim, rows, _p(w), _p(b), _p(y), None, _stream()) == R.TTT_OK
    assert torch.equal(y, Y)
    n = R.ttt_norm_workspace_bytes(cfg, rows)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    for keep in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (0, 1, 1), (1, 0, 1)):
        out = [torch.full_like(o, 3.0) for o in want]
        ptr = [_p(o) if k else None for o, k in zip(out, keep)]
        space = (_p(ws), n) if keep[1] or keep[2] else (None, 0)
        assert L.ttt_layer_norm_backward(ctypes.byref(cfg), _p(x), dim, _p(dy), dim, rows, _p(w), _p(st), *ptr,
                                         *space, _stream()) == R.TTT_OK
        for o, full, k in zip(out, want, keep):
            assert torch.equal(o, full) if k else (o == 3).all()


@pytest.mark.parametrize("prec", [BF, F32])
@pytest.mark.parametrize("lens", [[150], [5], [1, 90, 0, 30], [2] * 40 + [100]])
def test_delta_without_last_states(lens, prec):
    """S_out or dS_in left out."""
    H, Hk, d, n = 4, 2, 128, sum(lens)
    x, S, dO, dSo = _inputs(n, n, H, Hk, d, prec, len(lens))
    cfg = R.make_delta_config(H, d, qk_heads=Hk, precision=prec)
    offs = _offsets(lens, 0) if len(lens) > 1 else None
    want, _ = R.ttt_delta_chunk(cfg, **x, S=S, offsets=offs)
    tok = R.ttt_delta_tokens(_p(x["Q"]), _p(x["K"]), _p(x["V"]), _p(x["log_decay"]), _p(x["beta"]),
                             Hk * d, Hk * d, H * d, n, _p(offs), len(lens))
    ws = R.alloc_delta_workspace(cfg, n, len(lens), backward=True)
    O = torch.empty_like(want)
    assert L.ttt_delta_chunk(ctypes.byref(cfg), ctypes.byref(tok), _p(S), None, _p(O), _p(ws), ws.numel(),
                             _stream()) == R.TTT_OK
    assert torch.equal(O, want)
    grads = R.ttt_delta_backward(cfg, **x, dO=dO, S=S, offsets=offs, dS_out=dSo)
    out = [torch.empty_like(g) for g in grads[:5]]
    assert L.ttt_delta_backward(ctypes.byref(cfg), ctypes.byref(tok), _p(S), _p(dO), _p(dSo), *map(_p, out), None,
                                _p(ws), ws.numel(), _stream()) == R.TTT_OK
    for a, b in zip(out, grads):
        assert torch.equal(a, b)
    R.ttt_check_device_error()
