"""The token gradients' kernel lays copies over shared memory that its threads wrote: equal chunks
in many blocks at once, and many times over, have to come out equal to the last bit."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import recon_chunk_ttt_b200 as R  # noqa: E402
from test_gpu_delta import BF, _inputs, _offsets  # noqa: E402


@pytest.mark.parametrize("H,Hk", [(4, 4), (4, 2)])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [64, 50])
def test_equal_chunks_have_equal_gradients(n, d, H, Hk):
    copies = 150
    x, S, dO, dSo = _inputs(n + d, n, H, Hk, d, BF)
    cfg = R.make_delta_config(H, d, qk_heads=Hk)
    one = R.ttt_delta_backward(cfg, **x, dO=dO, S=S, dS_out=dSo)
    many = {k: t.repeat(copies, 1) for k, t in x.items()}
    st = (copies, 1, 1, 1)
    for _ in range(10):
        got = R.ttt_delta_backward(cfg, **many, dO=dO.repeat(copies, 1), S=S.repeat(st),
                                   offsets=_offsets([n] * copies, 0), dS_out=dSo.repeat(st))
        for name, a, b in zip(("dQ", "dK", "dV", "dlog_decay", "dbeta", "dS"), got, one):
            a = a.view(copies, *b.shape) if name != "dS" else a.view(copies, *b.shape[1:])
            assert torch.equal(a, (b if name != "dS" else b[0]).expand_as(a)), name
    R.ttt_check_device_error()
