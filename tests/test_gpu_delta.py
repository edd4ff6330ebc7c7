"""The gated delta rule on the GPU against its definition in 64 bits, token
after token: S' = e^g S, u = b (v - S' k), S = S' + u k^T, o = scale S q.

Tolerances (relative Frobenius, per sequence and head).  A bf16 value is off
by at most 2^-8 of itself.  O: its own rounding, and that of the in-chunk
weights P, whose products can be larger than their sum: 4 * 2^-8.  Gradients
of bf16 tokens: their own rounding and up to two bf16 operands in each of three
sums: 6 * 2^-8.  FP32 results (states, and the gradients of log_decay and beta)
come from operands kept to 2^-24 and sums of up to 16 products a step cut at
2^-23: 16 * 2^-23 = 2e-6 a sum, two sums deep: 4e-6; in FP32_CHECK one rounding
of 2^-24 a token, at most 300 tokens: 2e-5.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import recon_chunk_ttt_b200 as R  # noqa: E402
from recon_chunk_ttt_b200 import build as _build  # noqa: E402

_build.build()

BF, F32 = R.PREC_BF16_TC, R.PREC_FP32_CHECK
TOL_O = {BF: 4 * 2.0 ** -8, F32: 2e-5}
TOL_G = {BF: 6 * 2.0 ** -8, F32: 2e-5}
TOL_S = {BF: 4e-6, F32: 2e-5}


def _dtype(prec):
    return torch.bfloat16 if prec == BF else torch.float32


def _inputs(seed, n, H, Hk, d, prec, seqs=1, decay=0.3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    unit = lambda h: torch.nn.functional.normalize(  # noqa: E731
        rnd(n, h, d) + 0.2 * rnd(1, h, d), dim=-1).reshape(n, h * d).to(_dtype(prec))
    x = dict(Q=unit(Hk), K=unit(Hk), V=(0.5 * rnd(n, H * d)).to(_dtype(prec)),
             log_decay=-decay * torch.rand(n, H, generator=g, device="cuda"),
             beta=torch.sigmoid(rnd(n, H)))
    return x, 0.1 * rnd(seqs, H, d, d), rnd(n, H * d).to(_dtype(prec)), 0.1 * rnd(seqs, H, d, d)


def _reference(x, S, lens, first, H, Hk, d, scale, leaves=False):
    """(O rows, states) in 64 bits; with leaves=True the inputs are float64
    leaves that require gradients, returned too."""
    v = {k: t.double().cpu() for k, t in x.items()}
    S = S.double().cpu()
    if leaves:
        v = {k: t.requires_grad_(True) for k, t in v.items()}
        S = S.requires_grad_(True)
    n = v["Q"].shape[0]
    q = v["Q"].view(n, Hk, d).repeat_interleave(H // Hk, 1)
    k = v["K"].view(n, Hk, d).repeat_interleave(H // Hk, 1)
    val = v["V"].view(n, H, d)
    rows, states, t = [], [], first
    for i, m in enumerate(lens):
        s = S[i]
        for _ in range(m):
            s = s * torch.exp(v["log_decay"][t])[:, None, None]
            u = v["beta"][t][:, None] * (val[t] - torch.einsum("hij,hj->hi", s, k[t]))
            s = s + u[:, :, None] * k[t][:, None, :]
            rows.append(scale * torch.einsum("hij,hj->hi", s, q[t]))
            t += 1
        states.append(s)
    O = torch.stack(rows) if rows else val.new_zeros(0, H, d)
    out = (O, torch.stack(states))
    return out + (v, S) if leaves else out


def _rel(a, b):
    a, b = a.double().cpu(), b.detach().double().cpu()
    assert torch.isfinite(a).all()
    nb = b.norm().item()
    return (a - b).norm().item() / nb if nb else a.norm().item()


def _close(a, b, tol, what, heads_dim):
    """Over the whole and over every head."""
    assert _rel(a, b) <= tol, (what, _rel(a, b), tol)
    for h in range(a.shape[heads_dim]):
        r = _rel(a.select(heads_dim, h), b.select(heads_dim, h))
        assert r <= 2 * tol, (what, "head", h, r, tol)


def _offsets(lens, first):
    return torch.tensor([first] + list(lens), device="cuda").cumsum(0)


CASES = [  # lens, H, Hk, d, precision
    ([1], 1, 1, 64, BF), ([1], 4, 2, 256, BF), ([63], 2, 1, 128, BF), ([64], 2, 2, 128, BF),
    ([65], 3, 3, 64, BF), ([129], 4, 1, 256, BF), ([300], 2, 1, 128, BF), ([193], 6, 3, 64, BF),
    ([5, 0, 64, 0, 130, 1, 63], 2, 1, 128, BF), ([0], 2, 2, 256, BF), ([0, 0, 7], 1, 1, 256, BF),
    ([70] * 23, 16, 8, 128, BF), ([70] * 11, 16, 4, 64, BF), ([40] * 5, 8, 8, 256, BF),
    ([1], 2, 1, 64, F32), ([100], 2, 2, 128, F32), ([33, 0, 17], 4, 2, 256, F32),
]


@pytest.mark.parametrize("lens,H,Hk,d,prec", CASES)
@pytest.mark.parametrize("packed", [False, True])
def test_chunk(lens, H, Hk, d, prec, packed):
    """One sequence without offsets; packed sequences with rows before the
    first and behind the last, which stay as they are and hold NaN."""
    if not packed and len(lens) > 1:
        pytest.skip("needs offsets")
    first, behind = (3, 70) if packed else (0, 0)
    n = first + sum(lens) + behind
    x, S, _, _ = _inputs(n + d, n, H, Hk, d, prec, len(lens))
    used = slice(first, first + sum(lens))
    clean = {k: t.clone() for k, t in x.items()}
    if packed:
        for t in x.values():
            t[:first] = float("nan")
            t[first + sum(lens):] = float("inf")
    cfg = R.make_delta_config(H, d, qk_heads=Hk, precision=prec)
    O = torch.full((n, H * d), 7.0, dtype=_dtype(prec), device="cuda")
    O, So = R.ttt_delta_chunk(cfg, **x, S=S, offsets=_offsets(lens, first) if packed else None, O=O)
    R.ttt_check_device_error()
    Or, Sr = _reference(clean, S, lens, first, H, Hk, d, d ** -0.5)
    assert (O[:first] == 7).all() and (O[used.stop:] == 7).all()
    if sum(lens):
        _close(O[used].view(-1, H, d), Or, TOL_O[prec], "O", 1)
    _close(So, Sr, TOL_S[prec], "S", 1)


@pytest.mark.parametrize("prec", [BF, F32])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_chunk_strides_scale_in_place_no_state(d, prec):
    """Q, K, V as columns of one projection's output; a scale of its own; the
    state in place; no state at all."""
    H, Hk, n = 4, 2, 150
    x, S, _, _ = _inputs(5, n, H, Hk, d, prec)
    both = torch.cat([x["Q"], x["K"], x["V"]], 1).contiguous()
    q, k = both[:, :Hk * d], both[:, Hk * d:2 * Hk * d]
    v = both[:, 2 * Hk * d:]
    cfg = R.make_delta_config(H, d, qk_heads=Hk, precision=prec, scale=-0.7)
    st = S.clone()
    O, So = R.ttt_delta_chunk(cfg, q, k, v, x["log_decay"], x["beta"], S=st, S_out=st)
    assert So.data_ptr() == st.data_ptr()
    Or, Sr = _reference(x, S, [n], 0, H, Hk, d, cfg.scale)
    _close(O.view(n, H, d), Or, TOL_O[prec], "O", 1)
    _close(st, Sr, TOL_S[prec], "S", 1)
    O0, S0 = R.ttt_delta_chunk(cfg, q, k, v, x["log_decay"], x["beta"])
    Or, Sr = _reference(x, torch.zeros_like(S), [n], 0, H, Hk, d, cfg.scale)
    _close(O0.view(n, H, d), Or, TOL_O[prec], "O", 1)
    _close(S0, Sr, TOL_S[prec], "S", 1)
    R.ttt_check_device_error()


@pytest.mark.parametrize("prec", [BF, F32])
def test_chunk_gates_at_their_ends(prec):
    """log_decay 0, -inf (forgets all), -80; beta 0, 1, 2; a value of infinity
    ahead in another sequence."""
    H, d, lens = 4, 64, [100, 90]
    n = sum(lens)
    x, S, _, _ = _inputs(9, n, H, H, d, prec, 2)
    x["log_decay"][:, 0] = 0
    x["log_decay"][40, 1] = float("-inf")
    x["log_decay"][64, 1] = float("-inf")
    x["log_decay"][:, 2] = -80.0
    x["beta"][::3, 0] = 0
    x["beta"][:, 1] = 1
    x["beta"][::2, 3] = 2
    cfg = R.make_delta_config(H, d, precision=prec)
    clean = {k: t.clone() for k, t in x.items()}
    x["V"][lens[0]:] = float("inf")
    O, So = R.ttt_delta_chunk(cfg, **x, S=S, offsets=_offsets(lens, 0))
    Or, Sr = _reference(clean, S, lens, 0, H, H, d, d ** -0.5)
    _close(O[:100].view(-1, H, d), Or[:100], TOL_O[prec], "O", 1)
    _close(So[:1], Sr[:1], TOL_S[prec], "S", 1)
    R.ttt_check_device_error()


def test_chunk_long_equals_pieces():
    """A long sequence in one call, and in pieces with the state handed on."""
    H, d, n = 2, 128, 5000
    x, S, _, _ = _inputs(11, n, H, H, d, BF, decay=0.01)
    cfg = R.make_delta_config(H, d)
    O, So = R.ttt_delta_chunk(cfg, **x, S=S)
    st, parts = S.clone(), []
    for a, b in ((0, 64), (64, 1000), (1000, 1001), (1001, 5000)):
        o, st = R.ttt_delta_chunk(cfg, **{k: t[a:b].contiguous() for k, t in x.items()}, S=st)
        parts.append(o)
    # both are within TOL_S of the exact state
    assert _rel(st, So) <= 2 * TOL_S[BF]
    assert _rel(torch.cat(parts), O) <= 2 * TOL_O[BF]
    again, Sa = R.ttt_delta_chunk(cfg, **x, S=S)
    assert torch.equal(again, O) and torch.equal(Sa, So)  # the same from run to run


@pytest.mark.parametrize("prec", [BF, F32])
@pytest.mark.parametrize("d,H,Hk", [(64, 3, 1), (128, 4, 2), (256, 2, 2)])
def test_step(d, H, Hk, prec):
    """Slots in any order, one twice and one three times, padding, a slot
    outside the pool; the other states stay bit for bit."""
    slots = [4, -1, 0, 4, 6, 9, 2, 6, 6, 100, 1]
    n, pool = len(slots), 8
    x, S, _, _ = _inputs(21, n, H, Hk, d, prec, pool)
    cfg = R.make_delta_config(H, d, qk_heads=Hk, precision=prec)
    sl = torch.tensor(slots, dtype=torch.int32, device="cuda")
    for place in ("in", "out"):
        st = S.clone()
        So = torch.full_like(S, 5.0) if place == "out" else st
        O = R.ttt_delta_step(cfg, **x, S=st, slots=sl, S_out=So)
        ref, rows = S.double().cpu().clone(), []
        for i, s in enumerate(slots):
            if not 0 <= s < pool:
                rows.append(torch.zeros(1, H, d, dtype=torch.float64))
                continue
            o, sn = _reference({k: t[i:i + 1] for k, t in x.items()}, ref[s:s + 1], [1], 0, H, Hk, d,
                               d ** -0.5)
            ref[s] = sn[0]
            rows.append(o)
        _close(O.view(n, H, d), torch.cat(rows), TOL_O[prec], "O", 1)
        for s in range(pool):
            if s in slots:
                assert _rel(So[s], ref[s]) <= 4e-6
            elif place == "in":
                assert torch.equal(So[s], S[s])
            else:
                assert (So[s] == 5).all() and torch.equal(st, S)


@pytest.mark.parametrize("prec", [BF, F32])
def test_steps_equal_chunk(prec):
    """Serving: a prompt in one call, then token by token, against all tokens
    in one call."""
    H, d, n, cut = 4, 128, 90, 70
    x, S, _, _ = _inputs(31, n, H, H, d, prec)
    cfg = R.make_delta_config(H, d, precision=prec)
    O, So = R.ttt_delta_chunk(cfg, **x, S=S)
    o, st = R.ttt_delta_chunk(cfg, **{k: t[:cut].contiguous() for k, t in x.items()}, S=S)
    rows = [o]
    for t in range(cut, n):
        rows.append(R.ttt_delta_step(cfg, **{k: v[t:t + 1] for k, v in x.items()}, S=st))
    assert _rel(torch.cat(rows), O) <= 2 * TOL_O[prec]
    assert _rel(st, So) <= 2 * TOL_S[prec]


GRADS = [
    ([1], 1, 1, 64, BF), ([64], 2, 1, 128, BF), ([65], 2, 2, 256, BF), ([150], 4, 2, 64, BF),
    ([5, 0, 64, 0, 130, 1, 63], 2, 1, 128, BF), ([130], 4, 1, 256, BF), ([0], 1, 1, 64, BF),
    ([600], 2, 2, 64, BF), ([30, 40], 8, 2, 256, BF), ([200] * 3, 2, 2, 128, BF),
    ([1], 2, 1, 64, F32), ([50, 0, 23], 4, 2, 128, F32), ([37], 2, 2, 256, F32),
]


@pytest.mark.parametrize("lens,H,Hk,d,prec", GRADS)
@pytest.mark.parametrize("full", [False, True])
def test_backward(lens, H, Hk, d, prec, full):
    """Against the definition's gradient in 64 bits; `full`: with a first state
    and a gradient of the last, packed between rows that stay as they are."""
    first, behind = (2, 5) if full else (0, 0)
    n = first + sum(lens) + behind
    x, S, dO, dSo = _inputs(n + 3 * d, n, H, Hk, d, prec, len(lens))
    clean = {k: t.clone() for k, t in x.items()}
    if full:
        for t in list(x.values()) + [dO]:
            t[:first] = float("nan")
            t[n - behind:] = float("nan")
    cfg = R.make_delta_config(H, d, qk_heads=Hk, precision=prec)
    tdt = _dtype(prec)
    mk = lambda w, dt: torch.full((n, w), 7.0, dtype=dt, device="cuda")  # noqa: E731
    outs = dict(dQ=mk(Hk * d, tdt), dK=mk(Hk * d, tdt), dV=mk(H * d, tdt),
                dlog_decay=mk(H, torch.float32), dbeta=mk(H, torch.float32))
    offs = _offsets(lens, first) if full or len(lens) > 1 else None
    got = R.ttt_delta_backward(cfg, **x, dO=dO, S=S if full else None, offsets=offs,
                               dS_out=dSo if full else None, **outs)
    R.ttt_check_device_error()
    Or, Sr, v, S64 = _reference(clean, S if full else torch.zeros_like(S), lens, first, H, Hk, d,
                                d ** -0.5, leaves=True)
    used = slice(first, first + sum(lens))
    loss = (Or * dO[used].double().cpu().view(-1, H, d)).sum()
    if full:
        loss = loss + (Sr * dSo.double().cpu()).sum()
    if sum(lens) or full:  # else nothing depends on anything
        loss.backward()
    for name, key, h, tol in (("dQ", "Q", Hk, TOL_G[prec]), ("dK", "K", Hk, TOL_G[prec]),
                              ("dV", "V", H, TOL_G[prec]), ("dlog_decay", "log_decay", H, TOL_S[prec]),
                              ("dbeta", "beta", H, TOL_S[prec])):
        t = outs[name]
        assert (t[:first] == 7).all() and (t[n - behind:] == 7).all(), name
        if sum(lens) == 0:
            continue
        g = v[key].grad[used]
        if name == "dlog_decay":  # a head that forgets fast has next to nothing: over all heads
            assert _rel(t[used], g) <= tol, (name, _rel(t[used], g))
            continue
        _close(t[used].view(sum(lens), h, -1), g.view(sum(lens), h, -1), tol, name, 1)
    gs = S64.grad if S64.grad is not None else torch.zeros_like(S64)
    assert _rel(got[5], gs) <= TOL_S[prec], ("dS", _rel(got[5], gs))


@pytest.mark.parametrize("prec", [BF, F32])
def test_backward_gates_at_their_ends(prec):
    """beta 0 (its gradient is not 0), 1, 2; log_decay 0, -inf, -60; dS in place."""
    H, d, n = 4, 64, 140
    x, S, dO, dSo = _inputs(77, n, H, H, d, prec)
    x["log_decay"][:, 0] = 0
    x["log_decay"][50, 1] = float("-inf")
    x["log_decay"][:, 2] = -60.0
    x["beta"][::2, 0] = 0
    x["beta"][:, 3] = 2
    cfg = R.make_delta_config(H, d, precision=prec)
    Or, Sr, v, S64 = _reference(x, S, [n], 0, H, H, d, d ** -0.5, leaves=True)
    ((Or * dO.double().cpu().view(n, H, d)).sum() + (Sr * dSo.double().cpu()).sum()).backward()
    ds = dSo.clone()
    dQ, dK, dV, dg, db, dS = R.ttt_delta_backward(cfg, **x, dO=dO, S=S, dS_out=ds, dS=ds)
    R.ttt_check_device_error()
    assert dS.data_ptr() == ds.data_ptr()
    for a, key, tol in ((dQ, "Q", TOL_G), (dK, "K", TOL_G), (dV, "V", TOL_G), (db, "beta", TOL_S)):
        _close(a.view(n, H, -1), v[key].grad.view(n, H, -1), tol[prec], key, 1)
    g = v["log_decay"].grad
    g[~torch.isfinite(x["log_decay"].cpu())] = 0  # 0 * e^-inf in the reference
    assert _rel(dg, g) <= TOL_S[prec]
    assert _rel(dS, S64.grad) <= TOL_S[prec]


def test_backward_against_differences():
    """fp32: the gradient along random directions against central differences
    of the forward call summed in 64 bits (error of the difference: h^2 and
    2^-24 / h; h = 2^-6 leaves about 3e-4)."""
    H, d, n, h = 2, 64, 40, 2.0 ** -6
    x, S, dO, dSo = _inputs(55, n, H, 1, d, F32)
    cfg = R.make_delta_config(H, d, qk_heads=1, precision=F32)

    def loss(x, S):
        O, So = R.ttt_delta_chunk(cfg, **x, S=S)
        return (O.double() * dO.double()).sum().item() + (So.double() * dSo.double()).sum().item()

    g = R.ttt_delta_backward(cfg, **x, dO=dO, S=S, dS_out=dSo)
    gen = torch.Generator(device="cuda").manual_seed(1)
    for i, key in enumerate(["Q", "K", "V", "log_decay", "beta", "S"]):
        t = S if key == "S" else x[key]
        z = torch.randn(t.shape, generator=gen, device="cuda") * (0.1 if key in ("log_decay", "beta") else 1)
        z = z / z.norm() * t.norm() / 4
        vals = []
        for sgn in (1, -1):
            moved = t + sgn * h * z
            vals.append(loss(x, moved) if key == "S" else loss({**x, key: moved}, S))
        diff = (vals[0] - vals[1]) / (2 * h)
        along = (g[i].double() * z.double()).sum().item()
        bound = 1e-3 * g[i].double().norm().item() * z.double().norm().item()
        assert abs(diff - along) <= bound, (key, diff, along, bound)


def test_bad_offsets_are_reported():
    """Offsets that decrease or leave 0..n stay inside the arrays and set the
    device error word; the next call is unharmed."""
    H, d, n = 2, 64, 100
    x, S, dO, _ = _inputs(3, n, H, H, d, BF, 3)
    cfg = R.make_delta_config(H, d)
    for offs in ([0, 60, 40, 100], [-5, 10, 20, 30], [0, 10, 20, 101]):
        R.ttt_delta_chunk(cfg, **x, S=S, offsets=torch.tensor(offs, device="cuda"))
        with pytest.raises(R.TTTError):
            R.ttt_check_device_error()
    offs = torch.tensor([0, 10, 20, 100], device="cuda")
    a, _ = R.ttt_delta_chunk(cfg, **x, S=S, offsets=offs)
    R.ttt_check_device_error()
    b, _ = R.ttt_delta_chunk(cfg, **x, S=S, offsets=offs)
    assert torch.equal(a, b)


@pytest.mark.parametrize("prec", [BF, F32])
def test_graphs_and_streams(prec):
    """Captured calls that share a workspace, replayed on new data; calls on
    another stream."""
    H, d, n = 2, 128, 130
    x, S, dO, dSo = _inputs(41, n, H, H, d, prec)
    y, _, _, _ = _inputs(42, n, H, H, d, prec)
    cfg = R.make_delta_config(H, d, precision=prec)
    ws = R.alloc_delta_workspace(cfg, n, backward=True)
    want_x = R.ttt_delta_chunk(cfg, **x, S=S)
    want_y = R.ttt_delta_chunk(cfg, **y, S=S)
    want_g = R.ttt_delta_backward(cfg, **y, dO=dO, S=S, dS_out=dSo)
    buf = {k: t.clone() for k, t in x.items()}
    O, So = torch.empty_like(want_x[0]), torch.empty_like(want_x[1])
    outs = [torch.empty_like(t) for t in want_g]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        R.ttt_delta_chunk(cfg, **buf, S=S, S_out=So, O=O, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(O, want_x[0]) and torch.equal(So, want_x[1])
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        R.ttt_delta_chunk(cfg, **buf, S=S, S_out=So, O=O, workspace=ws)
    with torch.cuda.graph(g2):
        R.ttt_delta_backward(cfg, **buf, dO=dO, S=S, dS_out=dSo, dQ=outs[0], dK=outs[1], dV=outs[2],
                             dlog_decay=outs[3], dbeta=outs[4], dS=outs[5], workspace=ws)
    for k in buf:
        buf[k].copy_(y[k])
    for _ in range(2):
        g2.replay()
        g1.replay()
    torch.cuda.synchronize()
    assert torch.equal(O, want_y[0]) and torch.equal(So, want_y[1])
    for a, b in zip(outs, want_g):
        assert torch.equal(a, b)
    R.ttt_check_device_error()


def test_binding_refusals():
    H, d, n = 2, 64, 100
    x, S, dO, _ = _inputs(1, n, H, H, d, BF)
    cfg = R.make_delta_config(H, d)
    bad = [dict(Q=x["Q"].float()), dict(V=x["V"][:5]), dict(beta=x["beta"].t()),
           dict(K=x["K"].t().contiguous().t()), dict(log_decay=x["log_decay"].cpu()),
           dict(S=S.double()), dict(S=S[:, :1]), dict(offsets=torch.tensor([0, 100]))]
    for b in bad:
        with pytest.raises(R.TTTError):
            R.ttt_delta_chunk(cfg, **{**x, **b})
    with pytest.raises(R.TTTError):
        R.ttt_delta_chunk(cfg, **x, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(R.TTTError):
        R.ttt_delta_step(cfg, **x, S=S)  # 100 requests, one state
    assert np.isfinite(R.ttt_delta_chunk(cfg, **x, S=S)[0].float().cpu().numpy()).all()


@pytest.mark.parametrize("lens,H,Hk,d", [
    ([1] * 30 + [300] + [0] * 5 + [17, 16, 64] + [4] * 25, 4, 2, 128),  # ranked by length
    ([1] * 300 + [100] + [0] * 220 + [40], 2, 2, 64),                   # too many to be ranked
    ([9] * 30, 2, 1, 256),                                              # short ones alone
])
def test_short_and_long_together(lens, H, Hk, d):
    """Single tokens and long sequences in one call, states in place."""
    n = sum(lens)
    x, S, _, _ = _inputs(n, n, H, Hk, d, BF, len(lens))
    cfg = R.make_delta_config(H, d, qk_heads=Hk)
    Or, Sr = _reference(x, S, lens, 0, H, Hk, d, d ** -0.5)
    O, So = R.ttt_delta_chunk(cfg, **x, S=S, offsets=_offsets(lens, 0), S_out=S)
    assert So is S and R.ttt_check_device_error() == 0
    _close(O.view(-1, H, d), Or, TOL_O[BF], "O", 1)
    _close(S, Sr, TOL_S[BF], "S", 1)


@pytest.mark.parametrize("handle", [False, True])
def test_stream_argument(handle):
    """A call on a stream that is behind the current one: the workspace and the
    outputs it allocates are not the current stream's to use."""
    H, d, n = 4, 128, 700
    x, S, dO, dSo = _inputs(43, n, H, H, d, BF)
    cfg = R.make_delta_config(H, d)
    want = R.ttt_delta_chunk(cfg, **x, S=S)
    grad = R.ttt_delta_backward(cfg, **x, dO=dO, S=S, dS_out=dSo)
    sizes = [R.ttt_delta_workspace_bytes(cfg, n, backward=b) for b in (False, True)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    s = side.cuda_stream if handle else side
    got = R.ttt_delta_chunk(cfg, **x, S=S, stream=s)
    ggot = R.ttt_delta_backward(cfg, **x, dO=dO, S=S, dS_out=dSo, stream=s)
    for b in sizes:
        for _ in range(4):
            torch.empty(b, dtype=torch.uint8, device="cuda").fill_(255)
    torch.cuda.synchronize()
    for a, b in zip(got + ggot, want + grad):
        assert torch.equal(a, b)
    assert torch.equal(R.ttt_delta_chunk(cfg, **x, S=S, stream=0)[0], want[0])


def test_offsets_without_an_entry():
    x, _, _, _ = _inputs(1, 20, 1, 1, 64, BF)
    cfg = R.make_delta_config(1, 64)
    for bad in (torch.empty(0, dtype=torch.int64, device="cuda"),
                torch.tensor([[0, 20]], device="cuda")):
        with pytest.raises(R.TTTError):
            R.ttt_delta_chunk(cfg, **x, offsets=bad)


@pytest.mark.parametrize("lens,H,Hk,d", [([70] * 11, 8, 4, 64), ([3] * 515 + [90], 2, 1, 64),
                                         ([1, 700, 64], 8, 8, 128)])
def test_backward_of_many_chains(lens, H, Hk, d):
    """More chains than SMs; more sequences than are ranked; heads of their own."""
    test_backward(lens, H, Hk, d, BF, True)


def test_two_calls_at_once():
    """Forward and gradient on two streams at a time, each with its workspace."""
    H, d, n = 4, 128, 900
    cfg = R.make_delta_config(H, d)
    data = [_inputs(50 + i, n, H, H, d, BF) for i in range(4)]
    off = _offsets([400, 0, 500], 0)
    S = [torch.stack([y[0] for _ in range(3)]) for _, y, _, _ in data]
    want = [(R.ttt_delta_chunk(cfg, **x, S=s, offsets=off)
             + R.ttt_delta_backward(cfg, **x, dO=dO, S=s, offsets=off))
            for (x, _, dO, _), s in zip(data, S)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in data]
    for _ in range(3):
        got = [(R.ttt_delta_chunk(cfg, **x, S=s, offsets=off, stream=st)
                + R.ttt_delta_backward(cfg, **x, dO=dO, S=s, offsets=off, stream=st))
               for (x, _, dO, _), s, st in zip(data, S, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))
    R.ttt_check_device_error()
