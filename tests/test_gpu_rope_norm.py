"""Rotary positions over three axes and layer norm on the GPU against their
formulas in 64 bits, and the operators around the layer in a row.

Tolerances.  A bf16 result is off by its rounding, 2^-8 of the value, plus the
fp32 arithmetic; an fp32 rotation by a few roundings of values of its pair:
4 * 2^-24 of the pair's length.  Layer norm in fp32: the mean's error is
relative to the row's largest value (2^-24 a term of a tree of sums), so rows
whose mean is m standard deviations from zero are allowed (8 + 4 m) * 2^-24.
Column sums of n rows: n^(1/2) roundings of 2^-24, at most a few thousand rows
here: 1e-5.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import recon_chunk_ttt_b200 as R  # noqa: E402
from recon_chunk_ttt_b200 import build as _build  # noqa: E402

_build.build()

BF, F32 = R.PREC_BF16_TC, R.PREC_FP32_CHECK
HALF, PAIRS, AXIS, HEAD = R.ROPE_HALF, R.ROPE_PAIRS, R.ROPE_FREQ_AXIS, R.ROPE_FREQ_HEAD


def _dtype(prec):
    return torch.bfloat16 if prec == BF else torch.float32


def _rope_ref(x, pos, d, rot, base, layout, freq, inverse):
    x = x.double()
    n, total = x.shape[0], sum(rot)
    x = x.view(n, -1, d)
    y, j = x.clone(), 0
    for a in range(3):
        for i in range(rot[a] // 2):
            e = 2 * i / rot[a] if freq == AXIS else 2 * j / total
            ang = (pos[:, a].double() * float(torch.tensor(base[a])) ** -e)[:, None]
            ang = -ang if inverse else ang
            p, q = (2 * j, 2 * j + 1) if layout == PAIRS else (j, j + total // 2)
            y[..., p] = x[..., p] * ang.cos() - x[..., q] * ang.sin()
            y[..., q] = x[..., q] * ang.cos() + x[..., p] * ang.sin()
            j += 1
    return y.view(n, -1)


def _positions(n, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    p = torch.randint(-40, 2000, (n, 3), generator=g, device="cuda").float()
    p[:, 0] *= 500  # far
    p[::3, 1] += 0.5  # between the patches
    p[0] = 0
    return p


def _check(y, ref, x, prec):
    # a pair's length is at most sqrt(2) of its larger value: bound by the row's largest
    tol = (2.0 ** -8 if prec == BF else 0.0) * ref.abs() + 8 * 2.0 ** -24 * x.double().abs().amax(1, True)
    bad = (y.double() - ref).abs() > tol
    assert not bad.any(), ((y.double() - ref).abs() / tol).max().item()


@pytest.mark.parametrize("prec", [BF, F32])
@pytest.mark.parametrize("d,rot", [(64, (16, 24, 24)), (128, (32, 48, 48)), (128, (0, 64, 64)),
                                   (256, (64, 96, 96)), (64, (2, 6, 2)), (128, (10, 14, 8)),
                                   (256, (2, 0, 0)), (64, (0, 0, 64))])
@pytest.mark.parametrize("layout", [HALF, PAIRS])
@pytest.mark.parametrize("freq", [AXIS, HEAD])
def test_rope(d, rot, layout, freq, prec):
    n, hq, hk, base = 77, 3, 2, (10000.0, 100.0, 500.0)
    g = torch.Generator(device="cuda").manual_seed(d)
    Q = torch.randn(n, hq * d, generator=g, device="cuda").to(_dtype(prec))
    K = torch.randn(n, hk * d, generator=g, device="cuda").to(_dtype(prec))
    pos = _positions(n)
    cfg = R.make_rope_config(d, rot, base=base, layout=layout, freq=freq, precision=prec)
    for inverse in (False, True):
        Qo, Ko = R.ttt_rope(cfg, Q, K, pos, inverse=inverse)
        _check(Qo, _rope_ref(Q, pos, d, rot, base, layout, freq, inverse), Q, prec)
        _check(Ko, _rope_ref(K, pos, d, rot, base, layout, freq, inverse), K, prec)
        q3, total = Qo.view(n, hq, d), sum(rot)
        assert torch.equal(q3[..., total:], Q.view(n, hq, d)[..., total:])  # what is not rotated
    assert torch.equal(Qo[0], Q[0])  # position 0


@pytest.mark.parametrize("layout", [HALF, PAIRS])
@pytest.mark.parametrize("n", [1, 2, 9, 1374, 5000])
def test_rope_sizes_strides_in_place(n, layout):
    """Heads of one projection's output, in place and into another's columns;
    only q; there and back."""
    d, hq, hk, rot = 128, 4, 1, (32, 48, 48)
    cfg = R.make_rope_config(d, rot, layout=layout)
    both = torch.randn(n, (hq + 2 * hk) * d, device="cuda", dtype=torch.bfloat16)
    Q, K, V = both.split([hq * d, hk * d, hk * d], 1)
    pos = _positions(n, 3)
    Qd, Kd = R.ttt_rope(cfg, Q, K, pos)
    wide = torch.full((n, 2 * hq * d), 3.0, device="cuda", dtype=torch.bfloat16)
    R.ttt_rope(cfg, Q, None, pos, Q_out=wide[:, hq * d:])
    assert torch.equal(wide[:, hq * d:], Qd) and (wide[:, :hq * d] == 3).all()
    keep = V.clone()
    R.ttt_rope(cfg, Q, K, pos, Q_out=Q, K_out=K)
    assert torch.equal(Q, Qd) and torch.equal(K, Kd) and torch.equal(V, keep)
    # there and back: turning back leaves each value off by 2^-8 of itself, and turning that
    # error again makes at most sqrt(2) 2^-8 of the row's largest value of it
    back, _ = R.ttt_rope(cfg, Kd, None, pos, inverse=True)
    again = _rope_ref(back, pos, d, rot, (1e4,) * 3, layout, AXIS, False)
    assert ((again - Kd.double()).abs() <= 1.5 * 2.0 ** -8 * Kd.double().abs().amax(1, True)).all()


@pytest.mark.parametrize("hq,hk,layout", [(4096, 4096, PAIRS), (4096, 4, HALF)])
def test_rope_as_many_heads_as_there_may_be(hq, hk, layout):
    """A token whose heads are more than 2^16 vectors; every head as the first."""
    d, rot = 128, (32, 48, 48)
    cfg = R.make_rope_config(d, rot, layout=layout)
    x = torch.randn(2, d, device="cuda", dtype=torch.bfloat16)
    pos = _positions(2, 5)
    want, _ = R.ttt_rope(cfg, x, None, pos)
    Q, K = R.ttt_rope(cfg, x.repeat(1, hq), x.repeat(1, hk), pos)
    assert torch.equal(Q, want.repeat(1, hq)) and torch.equal(K, want.repeat(1, hk))


def test_rope_values_pass_and_positions_that_are_no_numbers():
    """NaN and infinity in the part that is not rotated stay where they are; a
    position of NaN reaches its own token's axis only."""
    d, rot = 64, (8, 8, 8)
    cfg = R.make_rope_config(d, rot, precision=F32)
    x = torch.randn(5, d, device="cuda")
    x[:, 24:] = float("nan")
    x[2, 30] = float("inf")
    pos = _positions(5)
    pos[3, 1] = float("nan")
    y, _ = R.ttt_rope(cfg, x, None, pos)
    assert torch.equal(torch.isnan(y[:, 24:]), torch.isnan(x[:, 24:])) and torch.isinf(y[2, 30])
    bad = torch.isnan(y[:, :24])
    assert bad[3, 4:8].all() and bad[3, 16:20].all() and bad.sum() == 8
    with pytest.raises(R.TTTError):
        R.ttt_rope(cfg, x[:, :60], None, pos)
    with pytest.raises(R.TTTError):
        R.ttt_rope(cfg, x, None, pos.double())
    with pytest.raises(R.TTTError):
        R.ttt_rope(cfg, x, None, pos[:4])


DIMS = [1, 3, 64, 100, 128, 1000, 1024, 1153, 2048, 4096, 4097, 8192, 16384, 20000]


def _norm_ref(x, w, b, eps):
    x = x.double()
    m = x.mean(1, keepdim=True)
    r = ((x - m).square().mean(1, keepdim=True) + eps).rsqrt()
    y = (x - m) * r
    if w is not None:
        y = y * w.double()
    if b is not None:
        y = y + b.double()
    return y, torch.cat([m, r], 1)


@pytest.mark.parametrize("prec", [BF, F32])
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("affine", [0, 1, 2])
def test_norm(dim, affine, prec):
    rows = 37
    g = torch.Generator(device="cuda").manual_seed(dim)
    x = (torch.randn(rows, dim, generator=g, device="cuda") + 3).to(_dtype(prec))
    w = torch.randn(dim, generator=g, device="cuda") if affine else None
    b = torch.randn(dim, generator=g, device="cuda") if affine == 2 else None
    cfg = R.make_norm_config(dim, eps=1e-5, precision=prec)
    Y, st = R.ttt_layer_norm(cfg, x, w, b)
    ref, sr = _norm_ref(x, w, b, 1e-5)
    # values and mean of up to 8 standard deviations; dim 1: y is the bias exactly
    scale = ref.abs() + (1 if w is None else w.double().abs()) * 8
    tol = (2.0 ** -8 if prec == BF else 0) * ref.abs() + 24 * 2.0 ** -24 * scale
    assert ((Y.double() - ref).abs() <= tol).all()
    assert ((st[:, 0].double() - sr[:, 0]).abs() <= 8 * 2.0 ** -24 * 8).all()
    assert ((st[:, 1].double() / sr[:, 1] - 1).abs() <= 24 * 2.0 ** -24).all()


def _norm_grads(x, dy, w, eps):
    x = x.double().requires_grad_(True)
    w = (torch.ones(x.shape[1], device="cuda") if w is None else w).double().requires_grad_(True)
    b = torch.zeros(x.shape[1], device="cuda", dtype=torch.float64, requires_grad=True)
    y, _ = _norm_ref(x, w, b, eps)
    y.backward(dy.double())
    return x.grad, w.grad, b.grad


@pytest.mark.parametrize("prec", [BF, F32])
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("rows", [1, 50, 3001])
def test_norm_backward(dim, rows, prec):
    if dim * rows > 40_000_000:
        rows = 700
    g = torch.Generator(device="cuda").manual_seed(dim + rows)
    x = (torch.randn(rows, dim, generator=g, device="cuda") + 1).to(_dtype(prec))
    dy = torch.randn(rows, dim, generator=g, device="cuda").to(_dtype(prec))
    w = torch.randn(dim, generator=g, device="cuda") if rows != 50 else None
    cfg = R.make_norm_config(dim, eps=1e-5, precision=prec)
    _, st = R.ttt_layer_norm(cfg, x, w, None)
    dX, dw, db = R.ttt_layer_norm_backward(cfg, x, dy, st, w)
    rx, rw, rb = _norm_grads(x, dy, w, 1e-5)
    if dim > 1:  # a row of one value has no gradient: what is left is rounding of dy times rstd
        assert (dX.double() - rx).norm() <= (2.0 ** -8 if prec == BF else 2e-6) * rx.norm()
        assert (dw.double() - rw).norm() <= 1e-5 * rw.norm()
    assert (db.double() - rb).norm() <= 1e-5 * rb.norm()
    again = R.ttt_layer_norm_backward(cfg, x, dy, st, w)
    assert torch.equal(again[0], dX) and torch.equal(again[1], dw) and torch.equal(again[2], db)


@pytest.mark.parametrize("prec", [BF, F32])
@pytest.mark.parametrize("dim", [96, 257, 1024, 6000, 17000])
def test_norm_strides_in_place_and_parts(dim, prec):
    rows, t = 65, _dtype(prec)
    wide = torch.randn(rows, dim + 24, device="cuda").to(t)
    x, dyw = wide[:, :dim], torch.randn(rows, dim + 9, device="cuda").to(t)
    dy = dyw[:, :dim]
    w, b = torch.randn(dim, device="cuda"), torch.randn(dim, device="cuda")
    cfg = R.make_norm_config(dim, precision=prec)
    xd, dyd = x.contiguous(), dy.contiguous()
    Y, st = R.ttt_layer_norm(cfg, xd, w, b)
    # rows apart may be read value by value, in another order of the sums
    near = lambda a, c: (a.double() - c.double()).norm() <= (2.0 ** -8 if prec == BF else 1e-5) * c.double().norm()  # noqa: E731
    Ys, sts = R.ttt_layer_norm(cfg, x, w, b)
    assert near(Ys, Y) and near(sts, st)
    z = xd.clone()
    R.ttt_layer_norm(cfg, z, w, b, Y=z)
    assert torch.equal(z, Y)
    full = R.ttt_layer_norm_backward(cfg, xd, dyd, st, w)
    for a, c in zip(R.ttt_layer_norm_backward(cfg, x, dy, st, w), full):
        assert near(a, c)
    z = dyd.clone()
    got = R.ttt_layer_norm_backward(cfg, xd, z, st, w, dX=z)
    for a, c in zip(got, full):
        assert torch.equal(a, c)
    z = xd.clone()
    got = R.ttt_layer_norm_backward(cfg, z, dyd, st, w, dX=z)
    for a, c in zip(got, full):
        assert torch.equal(a, c)


def test_norm_rows_that_are_special():
    """A constant row gives the bias; a row of NaN or infinity stays alone; no
    rows give zero sums; a mean far from zero keeps its spread."""
    dim = 512
    cfg = R.make_norm_config(dim, precision=F32)
    x = torch.randn(6, dim, device="cuda")
    x[1] = 7.0
    x[2, 5] = float("nan")
    x[3, 9] = float("inf")
    x[4] = 1e4 + torch.randn(dim, device="cuda")
    w, b = torch.randn(dim, device="cuda"), torch.randn(dim, device="cuda")
    Y, st = R.ttt_layer_norm(cfg, x, w, b)
    assert torch.allclose(Y[1], b, atol=1e-6)
    assert torch.isnan(Y[2]).all() and torch.isnan(Y[3]).all()
    assert torch.isfinite(Y[[0, 1, 4, 5]]).all()
    ref, _ = _norm_ref(x[4:5], w, b, 1e-5)
    # the mean is off by half a step of 1e4 (5e-4) at most, the values are exact
    assert ((Y[4].double() - ref[0]).abs() <= 1.1e-3 * (w.double().abs() + 0.01)).all()
    e = torch.empty(0, dim, device="cuda")
    dX, dw, db = R.ttt_layer_norm_backward(cfg, e, e, torch.empty(0, 2, device="cuda"), w)
    assert dX.shape == (0, dim) and (dw == 0).all() and (db == 0).all()


def test_norm_against_differences():
    """Central differences of the forward call, fp32, summed in 64 bits."""
    rows, dim, h = 7, 96, 2.0 ** -6
    cfg = R.make_norm_config(dim, precision=F32)
    x, w = torch.randn(rows, dim, device="cuda"), torch.randn(dim, device="cuda")
    b, dy = torch.randn(dim, device="cuda"), torch.randn(rows, dim, device="cuda")
    loss = lambda x, w, b: (R.ttt_layer_norm(cfg, x, w, b)[0].double() * dy.double()).sum().item()  # noqa: E731
    _, st = R.ttt_layer_norm(cfg, x, w, b)
    grads = R.ttt_layer_norm_backward(cfg, x, dy, st, w)
    for i, t in enumerate((x, w, b)):
        z = torch.randn_like(t)
        args = [[x, w, b], [x, w, b]]
        args[0][i], args[1][i] = t + h * z, t - h * z
        diff = (loss(*args[0]) - loss(*args[1])) / (2 * h)
        along = (grads[i].double() * z.double()).sum().item()
        assert abs(diff - along) <= 1e-3 * grads[i].double().norm().item() * z.double().norm().item()


def test_norm_rope_captured():
    """Captured and replayed on new data, on a stream of its own."""
    n, d, H = 300, 64, 4
    x = torch.randn(n, H * d, device="cuda", dtype=torch.bfloat16)
    y = torch.randn_like(x)
    w = torch.randn(H * d, device="cuda")
    pos = _positions(n)
    nc, rc = R.make_norm_config(H * d), R.make_rope_config(d, (16, 24, 24))

    def run(x):
        z, st = R.ttt_layer_norm(nc, x, w)
        q, _ = R.ttt_rope(rc, z, None, pos)
        return (q,) + R.ttt_layer_norm_backward(nc, x, q, st, w)

    want, buf = run(y), x.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run(buf)
    buf.copy_(y)
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_all_in_a_row():
    """What a block does with its tokens: norm, projections, positions, delta
    rule, and the gradients of it all, against the same in 64 bits; then the
    last tokens one at a time.  Each of the four stages rounds its bf16 result
    (2^-8) and hands on the last one's: 4 * 4 * 2^-8 of each gradient."""
    n, C, H, Hk, d = 200, 256, 4, 2, 64
    g = torch.Generator(device="cuda").manual_seed(8)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = rnd(n, C).bfloat16()
    lw, lb = 1 + 0.1 * rnd(C), 0.1 * rnd(C)
    W = (rnd((2 * Hk + H) * d, C) / math.sqrt(C) / 8).bfloat16()
    gate, beta = -0.1 * torch.rand(n, H, generator=g, device="cuda"), torch.sigmoid(rnd(n, H))
    i = torch.arange(n, device="cuda")
    pos = torch.stack([i // 100, i % 100 // 10, i % 10], 1).float()
    dO = rnd(n, H * d).bfloat16()
    rot = (16, 24, 24)
    nc, rc = R.make_norm_config(C), R.make_rope_config(d, rot)
    dc = R.make_delta_config(H, d, qk_heads=Hk)

    z, st = R.ttt_layer_norm(nc, x, lw, lb)
    p = z @ W.t()
    Q, K, V = p.split([Hk * d, Hk * d, H * d], 1)
    Qr, Kr = R.ttt_rope(rc, Q, K, pos)
    O, S = R.ttt_delta_chunk(dc, Qr, Kr, V, gate, beta)
    dQr, dKr, dV, dg, db, _ = R.ttt_delta_backward(dc, Qr, Kr, V, gate, beta, dO)
    dQ, dK = R.ttt_rope(rc, dQr, dKr, pos, inverse=True)
    dp = torch.cat([dQ, dK, dV], 1)
    dz = dp @ W
    dx, dlw, dlb = R.ttt_layer_norm_backward(nc, x, dz, st, lw)
    R.ttt_check_device_error()

    v = {k: t.double().cpu().requires_grad_(True)
         for k, t in dict(x=x, lw=lw, lb=lb, W=W, gate=gate, beta=beta).items()}
    zz, _ = _norm_ref(v["x"], v["lw"], v["lb"], 1e-5)
    pp = zz @ v["W"].t()
    q, k, val = pp.split([Hk * d, Hk * d, H * d], 1)
    ang, j = [], 0
    for a in range(3):
        for c in range(rot[a] // 2):
            ang.append(pos[:, a].double().cpu() * 10000.0 ** (-2 * c / rot[a]))
    ang = torch.stack(ang, 1)[:, None]

    def turn(t, h):
        t = t.view(n, h, d)
        lo, hi = t[..., :d // 2], t[..., d // 2:]
        return torch.cat([lo * ang.cos() - hi * ang.sin(), hi * ang.cos() + lo * ang.sin()], -1)

    q, k = (turn(t, Hk).repeat_interleave(H // Hk, 1) for t in (q, k))
    val, s, rows = val.view(n, H, d), torch.zeros(H, d, d, dtype=torch.float64), []
    for t in range(n):
        s = s * torch.exp(v["gate"][t])[:, None, None]
        u = v["beta"][t][:, None] * (val[t] - torch.einsum("hij,hj->hi", s, k[t]))
        s = s + u[:, :, None] * k[t][:, None, :]
        rows.append(d ** -0.5 * torch.einsum("hij,hj->hi", s, q[t]))
    out = torch.stack(rows).view(n, H * d)
    (out * dO.double().cpu()).sum().backward()
    tol = 16 * 2.0 ** -8
    rel = lambda a, b: ((a.double().cpu() - b).norm() / b.norm()).item()  # noqa: E731
    for name, a, b in (("O", O, out.detach()), ("dx", dx, v["x"].grad), ("dlw", dlw, v["lw"].grad),
                       ("dlb", dlb, v["lb"].grad), ("dW", dp.float().t() @ z.float(), v["W"].grad),
                       ("dgate", dg, v["gate"].grad), ("dbeta", db, v["beta"].grad)):
        assert rel(a, b) <= tol, (name, rel(a, b))

    # serving: the first 150 tokens at once, the rest one by one
    m = 150
    _, st = R.ttt_delta_chunk(dc, Qr[:m], Kr[:m], V[:m], gate[:m], beta[:m])
    for t in range(m, n):
        zt, _ = R.ttt_layer_norm(nc, x[t:t + 1], lw, lb)
        qt, kt, vt = (zt @ W.t()).split([Hk * d, Hk * d, H * d], 1)
        qt, kt = R.ttt_rope(rc, qt, kt, pos[t:t + 1])
        o = R.ttt_delta_step(dc, qt, kt, vt, gate[t:t + 1], beta[t:t + 1], st)
        assert rel(o, out[t:t + 1].detach()) <= tol
    assert rel(st, S.double().cpu()) <= tol


@pytest.mark.parametrize("dim", [6, 34, 66, 258, 1154, 4098, 8190, 16386])
def test_norm_rows_of_pairs(dim):
    """bf16 rows that are even but no whole 16-byte vectors; rows that are, apart
    by an even distance."""
    test_norm(dim, 2, BF)
    test_norm_backward(dim, 50, BF)
    test_norm_backward(dim, 3001, BF)
    rows, whole = 65, dim // 8 * 8 + 8
    x = torch.randn(rows, whole + 2, device="cuda", dtype=torch.bfloat16)[:, :whole]
    dy = torch.randn(rows, whole + 6, device="cuda", dtype=torch.bfloat16)[:, :whole]
    w = torch.randn(whole, device="cuda")
    cfg = R.make_norm_config(whole)
    Y, st = R.ttt_layer_norm(cfg, x, w)
    Yd, _ = R.ttt_layer_norm(cfg, x.contiguous(), w)
    assert (Y.double() - Yd.double()).norm() <= 2.0 ** -8 * Yd.double().norm()
    got = R.ttt_layer_norm_backward(cfg, x, dy, st, w)
    for a, c in zip(got, _norm_grads(x, dy, w, 1e-5)):
        assert (a.double() - c).norm() <= (2.0 ** -8 if a.dtype == torch.bfloat16 else 1e-5) * c.norm()
