"""The gradient of the delta rule's log decays, head by head, where heads forget fast or a token
resets the state: it is e^g times a product of the states on both sides of the token, and may not
drown in the rounding of what other tokens or heads have.

Tolerances.  From e^-6 on the bf16 path takes a running sum from the sequence's end: <E, S> of the last states,
then dO . O - dV . V of each token.  The sum may be far smaller than its terms, so its error is measured against
these: O and dV are fp32 results as the states are (4e-6, as in test_gpu_delta), and so are their products; they add
up as the root of the sum of their squares from the token to the end.  Heads that forget next to nothing within a
token keep test_gpu_delta's 4e-6 of the whole head.  FP32_CHECK forms the gradient directly from fp32 states,
one rounding of 2^-24 a token as there: 2e-5.

Below e^-6 the bf16 path forms it from the state S before the chunk and the gradient E behind it, kept in
bf16.  Their products may cancel, so the rounding is measured against the products, token by token: the value is
linear in S and in E, with derivatives e^(G_t) A_t and e^(G_end - G_t) S'_t (A_t, S'_t: gradient and faded
state at the token, G the sum of the chunk's log decays).  A value rounded to bf16 is off by 2^-8 / m of itself at
most, m in [1, 2) its mantissa, uniformly: 2^-8 sqrt(mean(m^-2) / 3) = 0.41 * 2^-8 on average.  So the sum is off
by 0.41 * 2^-8 times the root of the sum of the squared products, of S and of E together; five times that is
allowed.  What lies between two tokens of the chunk has U and dV in two parts, each off by 2^-17 at most, in one
factor of (dO . U), in both of (dV . U): 2 * 2^-17 of the root of the sum of the squared products of A_t and
S'_t, five times for what their errors share: 10 * 2^-17."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import recon_chunk_ttt_b200 as R  # noqa: E402
from test_gpu_delta import BF, F32, TOL_S, _inputs, _offsets, _reference, _rel  # noqa: E402


def _products(x, S, dO, dSo, H, Hk, d):
    """For one sequence (S, dSo: its states) in 64 bits: dlog_decay [n, H], and for each token and head
    the root of the sum of the squared products of its value with the state before its chunk and the
    gradient behind it, of those of its own state and gradient, and of those of the running sum."""
    n, grp = x["Q"].shape[0], H // Hk
    v = {k: t.double().cpu() for k, t in x.items()}
    q = v["Q"].view(n, Hk, d).repeat_interleave(grp, 1)
    k = v["K"].view(n, Hk, d).repeat_interleave(grp, 1)
    val, g, b = v["V"].view(n, H, d), v["log_decay"], v["beta"]
    do = dO.double().cpu().view(n, H, d) * d ** -0.5
    s, faded = S.double().cpu(), []
    before, o = [], []  # the state before each chunk
    for t in range(n):
        if t % 64 == 0:
            before.append(s)
        f = s * torch.exp(g[t])[:, None, None]
        faded.append(f)
        u = b[t][:, None] * (val[t] - torch.einsum("hij,hj->hi", f, k[t]))
        s = f + u[:, :, None] * k[t][:, None, :]
        o.append(torch.einsum("hij,hj->hi", s, q[t]))
    A, dg, size = dSo.double().cpu(), torch.zeros(n, H, dtype=torch.float64), torch.zeros(n, H, 3)
    terms = (A * s).square().sum((-1, -2))
    for t in reversed(range(n)):
        c = t // 64 * 64
        if t == n - 1 or t % 64 == 63:
            E, end = A, t
        A = A + do[t][:, :, None] * q[t][:, None, :]
        dv = b[t][:, None] * torch.einsum("hij,hj->hi", A, k[t])
        A = A - dv[:, :, None] * k[t][:, None, :]
        terms = terms + (do[t] * o[t]).square().sum(-1) + (dv * val[t]).square().sum(-1)
        size[t, :, 2] = terms.sqrt()
        dg[t] = (A * faded[t]).sum((-1, -2))
        to, on = torch.exp(g[c:t + 1].sum(0)), torch.exp(g[t + 1:end + 1].sum(0))
        p1 = to[:, None, None] * A * before[c // 64]
        p2 = on[:, None, None] * faded[t] * E
        size[t, :, 0] = (p1.square().sum((-1, -2)) + p2.square().sum((-1, -2))).sqrt()
        size[t, :, 1] = (A * faded[t]).square().sum((-1, -2)).sqrt()
        A = A * torch.exp(g[t])[:, None, None]
    return dg, size


def _gradient(x, S, dO, dSo, lens, H, Hk, d, prec):
    n = sum(lens)
    cfg = R.make_delta_config(H, d, qk_heads=Hk, precision=prec)
    offs = _offsets(lens, 0) if len(lens) > 1 else None
    got = R.ttt_delta_backward(cfg, **x, dO=dO, S=S, offsets=offs, dS_out=dSo)
    R.ttt_check_device_error()
    Or, Sr, v, _ = _reference(x, S, lens, 0, H, Hk, d, d ** -0.5, leaves=True)
    ((Or * dO.double().cpu().view(n, H, d)).sum() + (Sr * dSo.double().cpu()).sum()).backward()
    return got[3], v["log_decay"].grad


def _fades(got, ref, size, what, alone=True):
    """Tokens below e^-6 (alone), or of the running sum."""
    tol = 5 * 0.41 * 2.0 ** -8 * size[..., 0] + 10 * 2.0 ** -17 * size[..., 1] if alone else 4e-6 * size[..., 2]
    off = (got.double().cpu() - ref).abs()
    assert (off <= tol).all(), (what, (off / tol).max())


RATES = [-0.05, -6.0, -7.9, -8.1, -12.0, -16.0, -20.0, -60.0]


FADE = -6.0


@pytest.mark.parametrize("prec", [BF, F32])
@pytest.mark.parametrize("lens,d,Hk", [([150], 64, 8), ([5, 0, 64, 130, 1], 128, 4), ([100], 256, 8),
                                       ([600], 64, 2)])
def test_heads_that_forget_fast(lens, d, Hk, prec, rates=RATES):
    """Each head at a rate of its own, checked by itself."""
    H, n = len(rates), sum(lens)
    x, S, dO, dSo = _inputs(n + d, n, H, Hk, d, prec, len(lens))
    rate = torch.tensor(rates, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(n + d)
    x["log_decay"] = rate * (1 + 0.01 * torch.rand(n, H, generator=gen, device="cuda"))
    got, ref = _gradient(x, S, dO, dSo, lens, H, Hk, d, prec)
    size, t = [], 0
    for i, m in enumerate(lens if prec == BF else []):
        one = {k: v[t:t + m] for k, v in x.items()}
        size.append(_products(one, S[i], dO[t:t + m], dSo[i], H, Hk, d)[1] if m else torch.zeros(0, H, 3))
        t += m
    for h, g in enumerate(rates):
        if prec == BF and g < -1:
            alone = bool(x["log_decay"][:, h].max() < FADE)
            _fades(got[:, h], ref[:, h], torch.cat(size)[:, h], g, alone)
        else:
            assert _rel(got[:, h], ref[:, h]) <= TOL_S[prec], g


@pytest.mark.parametrize("d", [64, 128, 256])
def test_heads_on_both_sides_of_the_rule(d):
    test_heads_that_forget_fast([200, 31], d, 4, BF, [-3.0, -5.0, -5.9, -6.1])


@pytest.mark.parametrize("prec", [BF, F32])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_tokens_that_reset(d, prec):
    """Slow heads in which some tokens forget almost everything, or all: those tokens by
    themselves, and exactly 0 where nothing is left."""
    H, n = 4, 700
    x, S, dO, dSo = _inputs(d, n, H, 2, d, prec, decay=0.05)
    at = {0: [0, 63, 64, 130, 600], 1: [65, 66, 67], 2: [511, 512, 699], 3: [1, 320, 448]}
    for h, ts in at.items():
        x["log_decay"][ts, h] = -18.0
    x["log_decay"][448, 3] = float("-inf")
    x["log_decay"][66, 1] = -1e30
    got, ref = _gradient(x, S, dO, dSo, [n], H, 2, d, prec)
    assert got[448, 3] == 0 and got[66, 1] == 0
    again, size = _products(x, S[0], dO, dSo[0], H, 2, d)
    assert (again - ref).norm() <= 1e-12 * ref.norm()
    for h, ts in at.items():
        ts = [t for t in ts if x["log_decay"][t, h] > -100]
        if prec == F32:
            assert _rel(got[ts, h], ref[ts, h]) <= TOL_S[F32], h
        else:
            _fades(got[ts, h], ref[ts, h], size[ts, h], h)
        slow = [t for t in range(n) if x["log_decay"][t, h] > FADE]
        assert _rel(got[slow, h], ref[slow, h]) <= 2 * TOL_S[prec], h


@pytest.mark.parametrize("first", [0, 3])
def test_rows_around_stay(first):
    """Fast heads in packed sequences between rows that hold NaN; no first state."""
    H, d, lens = 2, 64, [70, 30]
    n = first + sum(lens) + 9
    x, S, dO, dSo = _inputs(5, n, H, 2, d, BF, 2)
    x["log_decay"][:] = -15.0
    used = slice(first, first + sum(lens))
    clean = {k: t[used].clone() for k, t in x.items()}
    for t in list(x.values()) + [dO]:
        t[:first] = float("nan")
        t[used.stop:] = float("nan")
    cfg = R.make_delta_config(H, d)
    dg = torch.full((n, H), 7.0, device="cuda")
    R.ttt_delta_backward(cfg, **x, dO=dO, offsets=_offsets(lens, first), dlog_decay=dg)
    R.ttt_check_device_error()
    Or, _, v, _ = _reference(clean, torch.zeros_like(S), lens, 0, H, 2, d, d ** -0.5, leaves=True)
    (Or * dO[used].double().cpu().view(-1, H, d)).sum().backward()
    assert (dg[:first] == 7).all() and (dg[used.stop:] == 7).all()
    assert (dg[used][[0, 70]] == 0).all()  # no state before a sequence's first token
    ref, zero = v["log_decay"].grad, torch.zeros_like(S[0])
    for a, b in ((0, 70), (70, 100)):
        part = {k: t[a:b] for k, t in clean.items()}
        again, size = _products(part, zero, dO[used][a:b], zero, H, 2, d)
        assert (again - ref[a:b]).norm() <= 1e-12 * ref[a:b].norm()
        _fades(dg[used][a:b], ref[a:b], size, a)


def test_bad_offsets_with_tokens_that_forget():
    """Offsets that decrease or leave 0..n: reported, nothing outside the arrays, and the next call unharmed."""
    H, d, n = 2, 64, 200
    x, S, dO, dSo = _inputs(3, n, H, H, d, BF, 3)
    x["log_decay"][::5] = -12.0
    cfg = R.make_delta_config(H, d)
    good = torch.tensor([0, 10, 90, 200], device="cuda")
    want = R.ttt_delta_backward(cfg, **x, dO=dO, S=S, offsets=good, dS_out=dSo)
    for offs in ([0, 160, 40, 200], [-70, 10, 20, 130], [0, 10, 70, 264], [200, 130, 70, 0]):
        R.ttt_delta_backward(cfg, **x, dO=dO, S=S, offsets=torch.tensor(offs, device="cuda"), dS_out=dSo)
        with pytest.raises(R.TTTError):
            R.ttt_check_device_error()
    again = R.ttt_delta_backward(cfg, **x, dO=dO, S=S, offsets=good, dS_out=dSo)
    R.ttt_check_device_error()
    for a, b in zip(again, want):
        assert torch.equal(a, b)
