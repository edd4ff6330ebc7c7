"""Rotary positions where a block of the kernel takes several tokens (1,184 tokens of few heads
and more), over the pairs, layouts and types; a single rotated pair among them.  Tolerances as
in test_gpu_rope_norm: the result's own rounding, and 8 * 2^-24 of the row's largest value."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import recon_chunk_ttt_b200 as R  # noqa: E402
from test_gpu_rope_norm import (AXIS, BF, F32, HALF, HEAD, PAIRS, _check, _dtype,  # noqa: E402
                                _positions, _rope_ref)

BASE = (10000.0, 100.0, 500.0)


def _one(n, hq, hk, d, rot, layout, freq, prec):
    g = torch.Generator(device="cuda").manual_seed(n + d)
    Q = torch.randn(n, hq * d, generator=g, device="cuda").to(_dtype(prec))
    K = torch.randn(n, hk * d, generator=g, device="cuda").to(_dtype(prec)) if hk else None
    pos = _positions(n, d)
    cfg = R.make_rope_config(d, rot, base=BASE, layout=layout, freq=freq, precision=prec)
    for inverse in (False, True):
        Qo, Ko = R.ttt_rope(cfg, Q, K, pos, inverse=inverse)
        _check(Qo, _rope_ref(Q, pos, d, rot, BASE, layout, freq, inverse), Q, prec)
        if hk:
            _check(Ko, _rope_ref(K, pos, d, rot, BASE, layout, freq, inverse), K, prec)
    R.ttt_check_device_error()


@pytest.mark.parametrize("prec", [BF, F32])
@pytest.mark.parametrize("layout", [HALF, PAIRS])
@pytest.mark.parametrize("rot", [(2, 0, 0), (0, 2, 0), (0, 0, 2)])
@pytest.mark.parametrize("n,hq,hk,d", [(1184, 8, 0, 64), (1200, 1, 1, 128), (5000, 1, 0, 64),
                                       (5000, 3, 0, 256), (5001, 2, 1, 128)])
def test_one_pair(n, hq, hk, d, rot, layout, prec):
    _one(n, hq, hk, d, rot, layout, AXIS, prec)


@pytest.mark.parametrize("prec", [BF, F32])
@pytest.mark.parametrize("layout", [HALF, PAIRS])
@pytest.mark.parametrize("freq", [AXIS, HEAD])
@pytest.mark.parametrize("d,rot", [(64, (16, 24, 24)), (128, (0, 64, 64)), (256, (64, 96, 96)),
                                   (64, (2, 6, 2)), (128, (10, 14, 8)), (64, (2, 2, 0))])
@pytest.mark.parametrize("n,hq,hk", [(1200, 1, 0), (5000, 1, 0), (5000, 2, 1)])
def test_many_tokens_a_block(n, hq, hk, d, rot, freq, layout, prec):
    _one(n, hq, hk, d, rot, layout, freq, prec)
