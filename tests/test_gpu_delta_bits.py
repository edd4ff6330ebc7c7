"""How many digits each output of the delta rule's bf16 path keeps: tolerances near what the operands'
parts allow, so that a part that gets lost shows.

A value rounded to bf16 is off by 2^-8 / m of itself at most, m in [1, 2) its mantissa, uniformly:
r = 2^-8 sqrt(mean(m^-2) / 3) = 0.41 * 2^-8 = 1.6e-3 on average.  Sums of products whose signs are mixed are off by
r for each operand that is a single bf16 part, as roots of sums of squares:
 - dV: its own rounding: r.
 - O: its own, and P's: sqrt(2) r.
 - dQ: its own, and one operand of each sum (S as it is kept; A and U have two parts): sqrt(2) r.
 - dK: its own, and up to two operands (dV and S; M, or E): sqrt(3) r.
Five hundredths are added for chance: 150,000 values and more, a few percent of them large.
A second part that is missing adds r or more in the products it belongs to.
States and dbeta are fp32 results: 4e-6, as in test_gpu_delta.  dlog_decay is a running sum of such results, which
may be far smaller than its terms: 4e-6 of the root of the sum of their squares (derived in
test_gpu_delta_decay_grad), over all tokens and heads."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import recon_chunk_ttt_b200 as R  # noqa: E402
from test_gpu_delta import BF, TOL_S, _inputs, _reference, _rel  # noqa: E402
from test_gpu_delta_decay_grad import _products  # noqa: E402

ROUND = 0.41 * 2.0 ** -8 * 1.05


@pytest.mark.parametrize("H,Hk,d,n", [(4, 4, 64, 640), (2, 1, 128, 640), (2, 2, 256, 400)])
def test_digits(H, Hk, d, n):
    x, S, dO, dSo = _inputs(7 * d, n, H, Hk, d, BF)
    cfg = R.make_delta_config(H, d, qk_heads=Hk)
    O, So = R.ttt_delta_chunk(cfg, **x, S=S)
    dQ, dK, dV, dg, db, dS = R.ttt_delta_backward(cfg, **x, dO=dO, S=S, dS_out=dSo)
    R.ttt_check_device_error()
    Or, Sr, v, S64 = _reference(x, S, [n], 0, H, Hk, d, d ** -0.5, leaves=True)
    ((Or * dO.double().cpu().view(n, H, d)).sum() + (Sr * dSo.double().cpu()).sum()).backward()
    again, size = _products(x, S[0], dO, dSo[0], H, Hk, d)
    assert (again - v["log_decay"].grad).norm() <= 1e-12 * again.norm()
    terms = size[..., 2].norm().item() / again.norm().item()
    off = {"O": (_rel(O.view(n, H, d), Or), 2 ** 0.5 * ROUND),
           "dQ": (_rel(dQ, v["Q"].grad), 2 ** 0.5 * ROUND), "dK": (_rel(dK, v["K"].grad), 3 ** 0.5 * ROUND),
           "dV": (_rel(dV, v["V"].grad), ROUND), "S": (_rel(So, Sr), TOL_S[BF]),
           "dS": (_rel(dS, S64.grad), TOL_S[BF]), "dbeta": (_rel(db, v["beta"].grad), TOL_S[BF]),
           "dlog_decay": (_rel(dg, v["log_decay"].grad), TOL_S[BF] * terms)}
    for k, (a, b) in off.items():
        assert a <= b, (k, a, b)
