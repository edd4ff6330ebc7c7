"""The gated delta rule, rotary positions over three axes and layer norm: what is measured of them.

`run` computes a case either in its plain form (elementary torch operations in 32 bits, 64 where 32
would lose what matters, rounded once at the end) or, with `own`, by this package's entry points.
`exact` computes the same outputs in 64 bits straight from the definitions: token after token for
the delta rule.  Sizes are those of this repository's workloads (1,374-token frames, 4 heads of 256,
100 frames) and generic serving and training shapes.
"""
from __future__ import annotations

import math
import random

import torch

own = False

CHUNK = 64
FRAME = 1374  # 37 x 37 patches + 5 special tokens


# ------------------------------------------------------------------------------------ cases
def _delta(name, op, n, heads, d, qk_heads=None, seqs=1, dtype="bf16", state=True):
    return {"name": name, "op": op, "n": n, "heads": heads, "qk_heads": qk_heads or heads, "d": d,
            "seqs": seqs, "dtype": dtype, "state": state}


def _rope(name, n, heads, k_heads, d, rot, inverse, layout="half", freq="axis", dtype="bf16"):
    return {"name": name, "op": "rope", "n": n, "heads": heads, "k_heads": k_heads, "d": d,
            "rot_t": rot[0], "rot_h": rot[1], "rot_w": rot[2], "inverse": inverse,
            "layout": layout, "freq": freq, "dtype": dtype}


def _norm(name, op, rows, dim, dtype="bf16", affine=True):
    return {"name": name, "op": op, "rows": rows, "dim": dim, "dtype": dtype, "affine": affine}


def listed():
    return [
        # one frame of the streaming workload carried through a head state, in order
        _delta("chunk_frame", "chunk", FRAME, 4, 256),
        # a packed batch of prompts of uneven lengths, two value heads to a key head
        _delta("chunk_packed", "chunk", 16411, 16, 128, qk_heads=8, seqs=13),
        # the 100-frame scene as one sequence: few heads, a long recurrence
        _delta("chunk_scene100", "chunk", 100 * FRAME, 4, 256, state=False),
        # one new token of one request: latency
        _delta("step_one", "step", 1, 4, 256),
        # one new token for each of 96 requests: the states' traffic
        _delta("step_batch", "step", 96, 32, 128, qk_heads=16, seqs=96),
        # training: gradients of one frame, and of a packed batch
        _delta("delta_grad_frame", "grad", FRAME, 4, 256),
        _delta("delta_grad_packed", "grad", 16384, 16, 128, qk_heads=8, seqs=7),
        # q and k of one frame, every axis with its own frequencies
        _rope("rope_frame", FRAME, 4, 4, 256, (64, 96, 96), False),
        # gradients of q and k of 100 frames, heads' frequencies shared over the axes
        _rope("rope_grad_scene100", 100 * FRAME, 8, 2, 128, (32, 48, 48), True, layout="pairs",
              freq="head"),
        # the norm before a frame's projections (the layer's 1024 channels)
        _norm("norm_frame", "norm", FRAME, 1024),
        # an odd width in 32 bits
        _norm("norm_odd_f32", "norm", 20011, 1153, dtype="f32"),
        # its gradients over 100 frames
        _norm("norm_grad_scene100", "norm_grad", 100 * FRAME, 1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "step", "grad", "rope", "norm", "norm_grad"])
    if op in ("chunk", "step", "grad"):
        d = rng.choice([64, 128, 256])
        heads = rng.choice([1, 2, 4, 6, 8, 16])
        group = rng.choice([g for g in (1, 2, 4) if heads % g == 0])
        dtype = "bf16"
        if op == "step":
            n = _log(rng, 1, 256)
            seqs = n
            dtype = rng.choice(["bf16", "bf16", "f32"])
        else:
            # at most the work of the largest listed case of the kind
            most = (100 * FRAME * 4 * 256 if op == "chunk" else 16384 * 16 * 128) // (heads * d)
            dtype = rng.choice(["bf16"] * 5 + ["f32"]) if op == "chunk" else "bf16"
            n = _log(rng, 1, min(most, 300 if dtype == "f32" else 40000))
            seqs = min(rng.choice([1, 1, 2, 5, 17]), n)
        return {"op": op, "n": n, "heads": heads, "qk_heads": heads // group, "d": d, "seqs": seqs,
                "dtype": dtype, "state": rng.random() < 0.7}
    if op == "rope":
        d = rng.choice([64, 128, 256])
        parts = [2 * rng.randint(0, d // 6) for _ in range(3)]
        if sum(parts) == 0:
            parts[0] = 2
        heads = rng.choice([1, 2, 4, 8, 16])
        return {"op": op, "n": _log(rng, 1, 100 * FRAME * 10 * 128 // (2 * heads * d)),
                "heads": heads, "k_heads": rng.choice([k for k in (0, 1, 2, heads) if k <= heads]),
                "d": d, "rot_t": parts[0], "rot_h": parts[1], "rot_w": parts[2],
                "inverse": rng.random() < 0.5, "layout": rng.choice(["half", "pairs"]),
                "freq": rng.choice(["axis", "head"]), "dtype": rng.choice(["bf16", "bf16", "f32"])}
    dim = rng.choice([64, 256, 1024, 2048, 4096, 8192, _log(rng, 1, 8192)])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    most = 100 * FRAME * 1024 // dim // (2 if dtype == "f32" else 1)
    return {"op": op, "rows": _log(rng, 1, min(most, 200000)), "dim": dim, "dtype": dtype,
            "affine": rng.random() < 0.8}


def _lengths(case):
    """Lengths of the packed sequences: uneven, one of them empty where there are many."""
    n, seqs = case["n"], case["seqs"]
    if seqs == 1 or case["op"] == "step":
        return [n] if seqs == 1 else [1] * n
    r = random.Random(n * 131 + seqs)
    cuts = sorted(r.randint(0, n) for _ in range(seqs - 1))
    if seqs > 4:
        cuts[2] = cuts[1]
    return [b - a for a, b in zip([0] + cuts, cuts + [n])]


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _size(case):
    return 2 if case["dtype"] == "bf16" else 4


# ------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    t, op = _type(case), case["op"]
    s = {"case": case}
    if op in ("chunk", "step", "grad"):
        n, H, Hk, d = case["n"], case["heads"], case["qk_heads"], case["d"]
        lens = _lengths(case)
        N = len(lens)

        def unit(h):  # normalised per token and head, with a direction that the tokens share
            x = normal(n, h, d) + 0.2 * normal(1, h, d)
            return (x / x.square().sum(-1, keepdim=True).sqrt()).to(t).reshape(n, h * d)

        s["Q"], s["K"] = unit(Hk), unit(Hk)
        s["V"] = (0.5 * normal(n, H * d)).to(t)
        # decay: one rate for each head, from slow to fast, times a softplus of the token
        rate = torch.exp(torch.linspace(-6.0, 0.5, H, device="cuda"))
        s["log_decay"] = -rate * torch.log1p(torch.exp(normal(n, H)))
        s["beta"] = torch.sigmoid(normal(n, H))
        s["S"] = 0.1 * normal(N, H, d, d) if case["state"] or op == "step" else None
        s["lengths"] = lens
        s["offsets"] = None
        if op != "step" and N > 1:
            s["offsets"] = torch.tensor([0] + lens, device="cuda").cumsum(0)
        if op == "step":  # the requests' places in the pool of states, in no order
            s["slots"] = torch.randperm(N, generator=gen, device="cuda").to(torch.int32)
            s["S_out"] = torch.empty_like(s["S"])
        if op == "grad":
            s["dO"] = normal(n, H * d).to(t)
            s["dS_out"] = 0.1 * normal(N, H, d, d) if case["state"] else None
    elif op == "rope":
        n, d = case["n"], case["d"]
        s["Q"] = normal(n, case["heads"] * d).to(t)
        s["K"] = normal(n, case["k_heads"] * d).to(t) if case["k_heads"] else None
        i = torch.arange(n, device="cuda")
        frame, place = i // FRAME, (i % FRAME - 5).clamp(min=0)  # 5 special tokens at the origin
        s["positions"] = torch.stack([frame, place // 37, place % 37], 1).float()
        s["positions"][:, 0] += int(seed) % 1000 * 37  # far on in a video
    else:
        rows, dim = case["rows"], case["dim"]
        s["X"] = (normal(rows, dim) * torch.exp(0.5 * normal(rows, 1)) + 0.3 * normal(rows, 1)).to(t)
        s["weight"] = 1 + 0.2 * normal(dim) if case["affine"] else None
        s["bias"] = 0.2 * normal(dim) if case["affine"] else None
        if op == "norm_grad":  # what the forward pass left
            s["dY"] = normal(rows, dim).to(t)
            x = s["X"].double()
            m = x.mean(-1)
            v = (x - m[:, None]).square().mean(-1)
            s["stats"] = torch.stack([m, (v + 1e-5).rsqrt()], 1).float()
    if own:
        import recon_chunk_ttt_b200 as R

        p = R.PREC_BF16_TC if case["dtype"] == "bf16" else R.PREC_FP32_CHECK
        if op in ("chunk", "step", "grad"):
            s["cfg"] = R.make_delta_config(case["heads"], case["d"], qk_heads=case["qk_heads"], precision=p)
            if op == "chunk":
                s["workspace"] = R.alloc_delta_workspace(s["cfg"], case["n"], len(s["lengths"]))
            elif op == "grad":
                s["workspace"] = R.alloc_delta_workspace(s["cfg"], case["n"], len(s["lengths"]), backward=True)
        elif op == "rope":
            s["cfg"] = R.make_rope_config(
                case["d"], (case["rot_t"], case["rot_h"], case["rot_w"]),
                layout=R.ROPE_HALF if case["layout"] == "half" else R.ROPE_PAIRS,
                freq=R.ROPE_FREQ_AXIS if case["freq"] == "axis" else R.ROPE_FREQ_HEAD, precision=p)
        else:
            s["cfg"] = R.make_norm_config(case["dim"], eps=1e-5, precision=p)
    return s


# ------------------------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    return {"chunk": _plain_chunk, "step": _plain_step, "grad": _plain_grad, "rope": _plain_rope,
            "norm": _plain_norm, "norm_grad": _plain_norm_grad}[op](state)


def _own(s, op):
    import recon_chunk_ttt_b200 as R

    if op == "chunk":
        O, S = R.ttt_delta_chunk(s["cfg"], s["Q"], s["K"], s["V"], s["log_decay"], s["beta"],
                                 S=s["S"], offsets=s["offsets"], workspace=s["workspace"])
        return {"O": O, "S": S}
    if op == "step":
        O = R.ttt_delta_step(s["cfg"], s["Q"], s["K"], s["V"], s["log_decay"], s["beta"], s["S"],
                             slots=s["slots"], S_out=s["S_out"])
        return {"O": O, "S": s["S_out"]}
    if op == "grad":
        g = R.ttt_delta_backward(s["cfg"], s["Q"], s["K"], s["V"], s["log_decay"], s["beta"], s["dO"],
                                 S=s["S"], offsets=s["offsets"], dS_out=s["dS_out"],
                                 workspace=s["workspace"])
        return dict(zip(("dQ", "dK", "dV", "dlog_decay", "dbeta", "dS"), g))
    if op == "rope":
        Q, K = R.ttt_rope(s["cfg"], s["Q"], s["K"], s["positions"], inverse=s["case"]["inverse"])
        return {"Q": Q} if K is None else {"Q": Q, "K": K}
    if op == "norm":
        Y, stats = R.ttt_layer_norm(s["cfg"], s["X"], s["weight"], s["bias"])
        return {"Y": Y, "stats": stats}
    dX, dw, db = R.ttt_layer_norm_backward(s["cfg"], s["X"], s["dY"], s["stats"], s["weight"])
    return {"dX": dX, "dweight": dw, "dbias": db}


# ------------------------------------------------------------------------------------ plain forms
# The delta rule in chunks of 64 tokens: inside a chunk the updates U solve (I + L) U = beta (V -
# gamma K S^T) with L the strictly lower part of beta Gamma (K K^T); only the states go in order.
def _chunks(s):
    """Inputs as [sequence, head, chunk, token, ...], padded with tokens that change nothing."""
    case = s["case"]
    H, Hk, d, C = case["heads"], case["qk_heads"], case["d"], CHUNK
    lens = torch.tensor(s["lengths"], device="cuda")
    start = lens.cumsum(0) - lens
    nc = max(1, -(-max(s["lengths"]) // C))
    at = torch.arange(nc * C, device="cuda")
    mask = at[None] < lens[:, None]
    idx = torch.where(mask, start[:, None] + at[None], 0)

    def take(x, h, w):
        x = torch.where(mask[..., None], x[idx].float(), 0.0).view(len(lens), nc, C, h, w)
        return x.permute(0, 3, 1, 2, 4)

    f = {"Q": take(s["Q"], Hk, d).repeat_interleave(H // Hk, 1), "V": take(s["V"], H, d),
         "K": take(s["K"], Hk, d).repeat_interleave(H // Hk, 1), "b": take(s["beta"], H, 1)}
    G = take(s["log_decay"], H, 1)[..., 0].double().cumsum(-1)
    f["Gamma"] = torch.exp((G[..., :, None] - G[..., None, :]).clamp(max=0.0)).float().tril()
    f["gamma"] = torch.exp(G).float()[..., None]
    f["rest"] = torch.exp(G[..., -1:] - G).float()[..., None]
    f["KK"] = f["Gamma"] * (f["K"] @ f["K"].mT)
    f["P"] = d ** -0.5 * f["Gamma"] * (f["Q"] @ f["K"].mT)
    f["L"] = (f["b"] * f["KK"]).tril(-1)
    M = -f["L"].double()  # (I + L)^-1 = (I + M)(I + M^2)(I + M^4) ...
    eye = torch.eye(C, device="cuda", dtype=torch.float64)
    M2 = M @ M
    M4 = M2 @ M2
    M8 = M4 @ M4
    M16 = M8 @ M8
    T = (eye + M) @ (eye + M2) @ (eye + M4) @ (eye + M8) @ (eye + M16) @ (eye + M16 @ M16)
    f["T"] = T.float()
    f["mask"], f["idx"] = mask, idx
    return f


def _back(s, f, x, h, w):
    """[sequence, head, chunk, token, w] to the packed tokens' rows."""
    x = x.permute(0, 2, 3, 1, 4).reshape(len(s["lengths"]), -1, h * w)
    return x[f["mask"]]  # sequences follow one another: the rows are in the tokens' order


def _start(s, f):
    N, H, d = len(s["lengths"]), s["case"]["heads"], s["case"]["d"]
    return s["S"] if s["S"] is not None else torch.zeros(N, H, d, d, device="cuda")


def _forward(s, f):
    """U [.., token, d] of all chunks, the states before each chunk, and the last states."""
    S = _start(s, f)
    W = f["T"] @ (f["b"] * f["gamma"] * f["K"])
    U0 = f["T"] @ (f["b"] * f["V"])
    Kr = f["rest"] * f["K"]
    states, us = [], []
    for c in range(W.shape[2]):
        states.append(S)
        U = U0[:, :, c] - W[:, :, c] @ S.mT
        us.append(U)
        S = f["gamma"][:, :, c, -1:] * S + U.mT @ Kr[:, :, c]
    return torch.stack(us, 2), torch.stack(states, 2), S


def _plain_chunk(s):
    case, t = s["case"], _type(s["case"])
    f = _chunks(s)
    U, S0, S = _forward(s, f)
    O = case["d"] ** -0.5 * f["gamma"] * (f["Q"] @ S0.mT) + f["P"] @ U
    return {"O": _back(s, f, O, case["heads"], case["d"]).to(t), "S": S}


def _plain_step(s):
    case = s["case"]
    n, H, Hk, d = case["n"], case["heads"], case["qk_heads"], case["d"]
    at = s["slots"].long()
    q = s["Q"].float().view(n, Hk, d, 1).repeat_interleave(H // Hk, 1)
    k = s["K"].float().view(n, Hk, d, 1).repeat_interleave(H // Hk, 1)
    v = s["V"].float().view(n, H, d, 1)
    S = torch.exp(s["log_decay"])[..., None, None] * s["S"][at]
    S = S + (s["beta"][..., None, None] * (v - S @ k)) @ k.mT
    s["S_out"][at] = S
    return {"O": (d ** -0.5 * (S @ q)).view(n, H * d).to(_type(case)), "S": s["S_out"]}


def _plain_grad(s):
    case, t = s["case"], _type(s["case"])
    N, H, Hk, d = len(s["lengths"]), case["heads"], case["qk_heads"], case["d"]
    f = _chunks(s)
    U, S0, _ = _forward(s, f)
    Q, K, V, b, gamma, rest, P, T = (f[k] for k in ("Q", "K", "V", "b", "gamma", "rest", "P", "T"))
    nc = U.shape[2]
    rows = torch.where(f["mask"][..., None], s["dO"][f["idx"]].float(), 0.0)
    D = rows.view(N, nc, CHUNK, H, d).permute(0, 3, 1, 2, 4)
    scale = d ** -0.5
    TD = T.mT @ (P.mT @ D)          # the part of X = T^T dU that needs no state
    TK = T.mT @ (rest * K)
    SQ = scale * D.mT @ (gamma * Q)
    bgK = b * gamma * K
    dS = s["dS_out"] if s["dS_out"] is not None else torch.zeros_like(_start(s, f))
    xs, ds = [None] * nc, [None] * nc
    for c in reversed(range(nc)):
        ds[c] = dS
        X = TD[:, :, c] + TK[:, :, c] @ dS.mT
        xs[c] = X
        dS = gamma[:, :, c, -1:] * dS + SQ[:, :, c] - X.mT @ bgK[:, :, c]
    X, E = torch.stack(xs, 2), torch.stack(ds, 2)
    dP, dL = (D @ U.mT).tril(), -(X @ U.mT).tril(-1)
    DS, XS, UE = D @ S0, X @ S0, U @ E
    A = dP * scale * f["Gamma"]
    M = dL * b * f["Gamma"]
    xk = (XS * K).sum(-1, keepdim=True)
    dQ = scale * gamma * DS + A @ K
    dK = A.mT @ Q + M @ K + M.mT @ K + rest * UE - b * gamma * XS
    db = (X * V).sum(-1, keepdim=True) - gamma * xk + (dL * f["KK"]).sum(-1, keepdim=True)
    Z = dP * P + dL * f["L"]
    dG = Z.sum(-1, keepdim=True) - Z.sum(-2)[..., None]
    dG = dG + scale * gamma * (DS * Q).sum(-1, keepdim=True) - b * gamma * xk
    uk = rest * (UE * K).sum(-1, keepdim=True)
    end = uk.sum(-2) + gamma[:, :, :, -1] * (E * S0).sum((-1, -2))[..., None]
    dg = (dG - uk).flip(-2).cumsum(-2).flip(-2) + end[..., None, :]

    def shared(x):  # key heads get the sum over the value heads that read them
        return x.view(N, Hk, H // Hk, nc, CHUNK, d).sum(2)

    return {"dQ": _back(s, f, shared(dQ), Hk, d).to(t), "dK": _back(s, f, shared(dK), Hk, d).to(t),
            "dV": _back(s, f, b * X, H, d).to(t), "dlog_decay": _back(s, f, dg, H, 1),
            "dbeta": _back(s, f, db, H, 1), "dS": dS}


def _angles(case, positions):
    """[tokens, d / 2] angles in 64 bits: pairs of the first axis, the second, the third, the rest still."""
    parts = [case["rot_t"], case["rot_h"], case["rot_w"]]
    pairs, total = case["d"] // 2, sum(parts)
    j = torch.arange(pairs, device="cuda", dtype=torch.float64)
    axis = (j >= parts[0] // 2).long() + (j >= (parts[0] + parts[1]) // 2)
    size = torch.tensor(parts, device="cuda", dtype=torch.float64)[axis]
    first = (torch.tensor([0, parts[0], parts[0] + parts[1]], device="cuda", dtype=torch.float64) / 2)[axis]
    e = 2 * (j - first) / size if case["freq"] == "axis" else 2 * j / total
    freq = torch.where(j < total // 2, torch.exp(-math.log(10000.0) * e), 0.0)
    return positions.double()[:, axis] * freq


def _plain_rope(s):
    case, d = s["case"], s["case"]["d"]
    a = _angles(case, s["positions"])[:, None]
    cos, sin = torch.cos(a).float(), torch.sin(a).float()
    sin = -sin if case["inverse"] else sin
    half = (case["rot_t"] + case["rot_h"] + case["rot_w"]) // 2

    def turn(x):
        x = x.float().view(x.shape[0], -1, d)
        if case["layout"] == "pairs":
            p, q = x[..., 0::2], x[..., 1::2]
            y = torch.stack([p * cos - q * sin, q * cos + p * sin], -1)
        else:  # the halves of the rotated part are paired
            c, n = cos[..., :half], sin[..., :half]
            p, q = x[..., :half], x[..., half:2 * half]
            y = torch.cat([p * c - q * n, q * c + p * n, x[..., 2 * half:]], -1)
        return y.reshape(x.shape[0], -1).to(_type(case))

    return {"Q": turn(s["Q"])} if s["K"] is None else {"Q": turn(s["Q"]), "K": turn(s["K"])}


def _plain_norm(s):
    x = s["X"].float()
    m = x.mean(-1, keepdim=True)
    c = x - m
    r = (c.square().mean(-1, keepdim=True) + 1e-5).rsqrt()
    y = c * r
    if s["weight"] is not None:
        y = y * s["weight"] + s["bias"]
    return {"Y": y.to(s["X"].dtype), "stats": torch.cat([m, r], 1)}


def _plain_norm_grad(s):
    m, r = s["stats"][:, :1], s["stats"][:, 1:]
    y = (s["X"].float() - m) * r
    g = s["dY"].float()
    w = g if s["weight"] is None else g * s["weight"]
    dx = r * (w - w.mean(-1, keepdim=True) - y * (w * y).mean(-1, keepdim=True))
    return {"dX": dx.to(s["X"].dtype), "dweight": (g * y).sum(0), "dbias": g.sum(0)}


# ------------------------------------------------------------------------------------ the work
def work(case):
    z, op = _size(case), case["op"]
    if op in ("chunk", "step", "grad"):
        n, H, Hk, d = case["n"], case["heads"], case["qk_heads"], case["d"]
        tokens = n * (2 * Hk + 2 * H) * d * z + 8 * n * H
        states = len(_lengths(case)) * H * d * d * 4
        if op == "grad":  # and dO, the gradients; per token the state is read and changed thrice over
            tokens += n * (2 * Hk + H) * d * z + 8 * n * H
            return {"bytes": tokens + (4 if case["state"] else 1) * states, "flops": 20 * n * H * d * d}
        return {"bytes": tokens + (2 if case["state"] or op == "step" else 1) * states,
                "flops": 6 * n * H * d * d}
    if op == "rope":
        x = case["n"] * (case["heads"] + case["k_heads"]) * case["d"]
        return {"bytes": 2 * z * x + 12 * case["n"], "flops": 3 * x}
    x = case["rows"] * case["dim"]
    p = 8 * case["dim"]
    if op == "norm":
        return {"bytes": 2 * z * x + 8 * case["rows"] + (p if case["affine"] else 0), "flops": 7 * x}
    return {"bytes": 3 * z * x + 8 * case["rows"] + p * (1.5 if case["affine"] else 1), "flops": 12 * x}


# ------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op in ("chunk", "step"):
        return _exact_tokens(case, s)
    if op == "grad":
        return _exact_grad(case, s)
    if op == "rope":
        return _exact_rope(case, s)
    x = s["X"].double()
    w = 1.0 if s["weight"] is None else s["weight"].double()
    if op == "norm":
        m, v = x.mean(1), x.var(1, unbiased=False)
        y = (x - m[:, None]) / (v[:, None] + 1e-5).sqrt() * w + (0.0 if s["bias"] is None else s["bias"].double())
        return {"Y": y, "stats": torch.stack([m, 1 / (v + 1e-5).sqrt()], 1)}
    mean, rstd = s["stats"].double().unbind(1)
    y = (x - mean[:, None]) * rstd[:, None]
    g = s["dY"].double()
    dy = g * w
    dx = (dy - dy.mean(1)[:, None] - y * (dy * y).mean(1)[:, None]) * rstd[:, None]
    return {"dX": dx, "dweight": torch.einsum("rc,rc->c", g, y), "dbias": g.sum(0)}


def _by_time(s, x, h, w):
    """Packed rows as [time, sequence, h, w] in 64 bits; sequences that have ended have zeros."""
    lens = s["lengths"]
    out = torch.zeros(max(lens), len(lens), h, w, device="cuda", dtype=torch.float64)
    o = 0
    for i, n in enumerate(lens):
        out[:n, i] = x[o:o + n].double().view(n, h, w)
        o += n
    return out


def _to_rows(s, x):
    return torch.cat([x[:n, i].flatten(1) for i, n in enumerate(s["lengths"])])


def _token(S, q, k, v, g, b):
    S = S * torch.exp(g)[..., None]
    u = b * (v - torch.einsum("nhij,nhj->nhi", S, k))
    return S + u[..., :, None] * k[..., None, :], u


def _sequences(case, s):
    H, Hk, d = case["heads"], case["qk_heads"], case["d"]
    q = _by_time(s, s["Q"], Hk, d).repeat_interleave(H // Hk, 2)
    k = _by_time(s, s["K"], Hk, d).repeat_interleave(H // Hk, 2)
    v, g, b = _by_time(s, s["V"], H, d), _by_time(s, s["log_decay"], H, 1), _by_time(s, s["beta"], H, 1)
    S = torch.zeros(len(s["lengths"]), H, d, d, device="cuda", dtype=torch.float64)
    if s["S"] is not None:
        S += s["S"].double()[s["slots"].long()] if case["op"] == "step" else s["S"].double()
    return q, k, v, g, b, S


def _exact_tokens(case, s):
    q, k, v, g, b, S = _sequences(case, s)
    o = torch.zeros_like(v)
    for t in range(v.shape[0]):
        S, _ = _token(S, q[t], k[t], v[t], g[t], b[t])
        o[t] = torch.einsum("nhij,nhj->nhi", S, q[t]) / math.sqrt(case["d"])
    if case["op"] == "step":
        S = torch.empty_like(S).index_copy_(0, s["slots"].long(), S)
    return {"O": _to_rows(s, o), "S": S}


def _exact_grad(case, s):
    H, Hk, d, every = case["heads"], case["qk_heads"], case["d"], 128
    q, k, v, g, b, S = _sequences(case, s)
    do = _by_time(s, s["dO"], H, d) / math.sqrt(d)
    kept = []
    for t in range(v.shape[0]):
        if t % every == 0:
            kept.append(S)
        S, _ = _token(S, q[t], k[t], v[t], g[t], b[t])
    A = torch.zeros_like(S) if s["dS_out"] is None else s["dS_out"].double()
    dq, dk, dv, dg, db = (torch.zeros_like(x) for x in (q, k, v, g, b))
    for first in reversed(range(0, v.shape[0], every)):
        S, before = kept[first // every], []
        for t in range(first, min(first + every, v.shape[0])):
            before.append(S)
            S, _ = _token(S, q[t], k[t], v[t], g[t], b[t])
        for t in reversed(range(first, min(first + every, v.shape[0]))):
            after, u = _token(before[t - first], q[t], k[t], v[t], g[t], b[t])
            faded = before[t - first] * torch.exp(g[t])[..., None]
            dq[t] = torch.einsum("nhij,nhi->nhj", after, do[t])
            A = A + do[t][..., :, None] * q[t][..., None, :]
            du = torch.einsum("nhij,nhj->nhi", A, k[t])
            dv[t] = b[t] * du
            db[t] = (du * (v[t] - torch.einsum("nhij,nhj->nhi", faded, k[t]))).sum(-1, keepdim=True)
            dk[t] = torch.einsum("nhij,nhi->nhj", A, u) - torch.einsum("nhij,nhi->nhj", faded, dv[t])
            A = A - dv[t][..., :, None] * k[t][..., None, :]
            dg[t] = (A * faded).sum((-1, -2))[..., None]
            A = A * torch.exp(g[t])[..., None]

    def shared(x):
        return x.unflatten(2, (Hk, H // Hk)).sum(3)

    return {"dQ": _to_rows(s, shared(dq)), "dK": _to_rows(s, shared(dk)), "dV": _to_rows(s, dv),
            "dlog_decay": _to_rows(s, dg), "dbeta": _to_rows(s, db), "dS": A}


def _exact_rope(case, s):
    d, pos = case["d"], s["positions"].double()
    parts = (case["rot_t"], case["rot_h"], case["rot_w"])
    total = sum(parts)
    out = {}
    for name in ("Q", "K"):
        if s[name] is None:
            continue
        x = s[name].double().view(case["n"], -1, d)
        y = x.clone()
        j = 0
        for axis in range(3):
            for i in range(parts[axis] // 2):
                e = i / (parts[axis] / 2) if case["freq"] == "axis" else j / (total / 2)
                a = (pos[:, axis] * 10000.0 ** -e)[:, None] * (-1 if case["inverse"] else 1)
                lo, hi = (2 * j, 2 * j + 1) if case["layout"] == "pairs" else (j, j + total // 2)
                y[..., lo] = x[..., lo] * torch.cos(a) - x[..., hi] * torch.sin(a)
                y[..., hi] = x[..., hi] * torch.cos(a) + x[..., lo] * torch.sin(a)
                j += 1
        out[name] = y.view(case["n"], -1)
    return out
