"""Layer norm's gradient over the range of row scales: the result does not depend on the
rows' scale but for its own, so neither may its accuracy.  Tolerances as in test_gpu_rope_norm:
fp32 2e-6 of the row (here for each row), bf16 its rounding, 2^-8."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import recon_chunk_ttt_b200 as R  # noqa: E402
from test_gpu_rope_norm import BF, F32, _dtype  # noqa: E402


@pytest.mark.parametrize("prec", [BF, F32])
@pytest.mark.parametrize("dim", [48, 512, 1153, 6000, 20000])
@pytest.mark.parametrize("size", [1e-17, 1e-14, 1e-6, 1e6, 1e13, 1e15, 1e16])
def test_gradient_of_rows_of_any_size(dim, size, prec):
    """Rows of standard deviation `size`, eps = 0: rstd is 1 / size, up to 1e17."""
    rows, g = 21, torch.Generator(device="cuda").manual_seed(dim)
    x = (size * (torch.randn(rows, dim, generator=g, device="cuda") + 0.5)).to(_dtype(prec))
    dy = torch.randn(rows, dim, generator=g, device="cuda").to(_dtype(prec))
    w = torch.randn(dim, generator=g, device="cuda")
    cfg = R.make_norm_config(dim, eps=0.0, precision=prec)
    _, st = R.ttt_layer_norm(cfg, x, w)
    dX, dw, db = R.ttt_layer_norm_backward(cfg, x, dy, st, w)
    m, r = st.double()[:, :1], st.double()[:, 1:]
    xh, gw = (x.double() - m) * r, dy.double() * w.double()
    ref = r * (gw - gw.mean(1, True) - xh * (gw * xh).mean(1, True))
    assert torch.isfinite(ref).all() and torch.isfinite(dX).all()
    off = ((dX.double() - ref) / r).norm(dim=1) / (ref / r).norm(dim=1)
    assert (off <= (2.0 ** -8 if prec == BF else 2e-6)).all(), off.max().item()
    rw = (dy.double() * xh).sum(0)
    assert (dw.double() - rw).norm() <= 1e-5 * rw.norm()
    assert (db.double() - dy.double().sum(0)).norm() <= 1e-5 * db.double().norm()
