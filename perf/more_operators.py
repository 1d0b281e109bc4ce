"""Cases of the sequence encoder's block without attention: group norm, gated recurrence and gated linear units.

An encoder of long series mixes along time by a gated linear recurrence where attention over the whole series would
cost too much, mixes its features by gated linear units, and normalises groups of channels in front of either.
``run`` makes one call of one of these operators, forward or forward and backward, either in plain torch operations
(``own`` false) or through this package's entry points (``own`` true).
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # the newest sample of 16 streams, normalised by itself: latency alone
        dict(name="group_norm_token", op="norm", train=False, dtype="bf16", wdtype="bf16", B=16, S=1, G=8, cg=64,
             activation="silu", ragged=False),
        # a training step on the loss's own batch: 32 padded series of up to 512 samples, 64 features
        dict(name="group_norm_batch", op="norm", train=True, dtype="fp32", wdtype="fp32", B=32, S=512, G=8, cg=8,
             activation="gelu", ragged=True),
        # a training step over long series in mixed precision, weights kept in fp32
        dict(name="group_norm_long", op="norm", train=True, dtype="bf16", wdtype="fp32", B=16, S=4096, G=32, cg=16,
             activation="silu", ragged=False),
        # the newest sample of 16 streams, each with its state
        dict(name="recurrence_token", op="recurrence", train=False, dtype="bf16", B=16, N=1, C=1024, state=True,
             ragged=False, reverse=False, tied=True),
        # a training step on the loss's own batch, backwards in time, as the second half of a bidirectional encoder
        dict(name="recurrence_batch", op="recurrence", train=True, dtype="fp32", B=32, N=512, C=64, state=False,
             ragged=True, reverse=True, tied=True),
        # encoding two long series of an odd length before their first answer, the input with a gate of its own
        dict(name="recurrence_prompt", op="recurrence", train=False, dtype="fp16", B=2, N=16383, C=264, state=True,
             ragged=False, reverse=False, tied=False),
        # a training step over long series
        dict(name="recurrence_long", op="recurrence", train=True, dtype="bf16", B=4, N=8192, C=1024, state=True,
             ragged=False, reverse=False, tied=True),
        # the newest sample of 16 streams: the weights are read once
        dict(name="gated_token", op="gated", train=False, dtype="bf16", rows=16, K=1024, F=4096, bias=False,
             activation="silu"),
        # a training step on the loss's own feature batch in full precision
        dict(name="gated_batch", op="gated", train=True, dtype="fp32", rows=16384, K=64, F=256, bias=True,
             activation="gelu"),
        # odd sizes everywhere: a series of 1021 samples, sizes that are no multiple of anything
        dict(name="gated_odd", op="gated", train=True, dtype="fp16", rows=1021, K=250, F=683, bias=True,
             activation="sigmoid"),
        # encoding four long series before their first answer
        dict(name="gated_prompt", op="gated", train=False, dtype="bf16", rows=16384, K=1024, F=2736, bias=False,
             activation="gelu"),
        # a training step of a wide encoder
        dict(name="gated_wide", op="gated", train=True, dtype="bf16", rows=16384, K=1024, F=4096, bias=False,
             activation="silu"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "recurrence", "gated"])
    dtype = rng.choice(["fp32", "bf16", "bf16", "fp16"])
    train = rng.random() < 0.6
    if op == "norm":
        cg = rng.choice([1, 2, 3, 4, 5, 8, 16, 24, 32, 64, 128])
        G = _log(rng, 1, min(512, 4096 // cg))
        B = _log(rng, 1, 64) if rng.random() < 0.7 else _log(rng, 64, 4096)
        S = _log(rng, 1, max(1, min(8192, (1 << 25) // (B * G * cg))))
        return dict(op=op, train=train, dtype=dtype, wdtype=rng.choice(["fp32", dtype]), B=B, S=S, G=G, cg=cg,
                    activation=rng.choice(["none", "silu", "gelu", "relu"]), ragged=rng.random() < 0.4)
    if op == "recurrence":
        B, C = _log(rng, 1, 32), _log(rng, 8, 4096)
        if rng.random() < 0.6:
            C = (C + 7) // 8 * 8
        N = rng.randint(1, 8) if rng.random() < 0.2 else _log(rng, 1, min(16384, (1 << 25) // (B * C)))
        return dict(op=op, train=train, dtype=dtype, B=B, N=N, C=C, state=rng.random() < 0.5, ragged=rng.random() < 0.4,
                    reverse=rng.random() < 0.4, tied=rng.random() < 0.7)
    K, F = _log(rng, 8, 2048), _log(rng, 8, 4096)
    if rng.random() < 0.6:
        K, F = (K + 7) // 8 * 8, (F + 7) // 8 * 8
    most = (1 << 30 if dtype == "fp32" else 1 << 36) // (K * F)
    rows = rng.randint(1, 32) if rng.random() < 0.25 else _log(rng, 1, max(1, min(16384, most)))
    return dict(op=op, train=train, dtype=dtype, rows=rows, K=K, F=F, bias=rng.random() < 0.5,
                activation=rng.choice(["silu", "gelu", "relu", "sigmoid"]))


def _lengths(case, limit):
    """Lengths of a padded batch: full, down to half, and an idle slot (0) where there are enough."""
    got = [max(1, limit - (b * 7919 + 3) % (limit // 2 + 1)) for b in range(case["B"])]
    if case["B"] >= 4:
        got[1] = 0
    return got


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype, train = DTYPES[case["dtype"]], case["train"]

    def normal(*shape, mean=0.0, std=1.0, dtype=dtype, grad=train):
        t = (torch.randn(*shape, generator=gen, device="cuda") * std + mean).to(dtype)
        return t.requires_grad_() if grad else t

    s = {"case": case}
    if case["op"] == "norm":
        B, S, C = case["B"], case["S"], case["G"] * case["cg"]
        w = DTYPES[case["wdtype"]]
        s["x"] = normal(B, S, C, mean=0.3, std=1.5)
        s["weight"] = normal(C, mean=1.0, std=0.2, dtype=w)
        s["bias"] = normal(C, std=0.2, dtype=w)
        s["dy"] = normal(B, S, C, std=1e-2, grad=False) if train else None
        s["lengths"] = torch.tensor(_lengths(case, S), dtype=torch.int32, device="cuda") if case["ragged"] else None
        return s
    if case["op"] == "recurrence":
        B, N, C = case["B"], case["N"], case["C"]
        s["x"] = normal(B, N, C)
        # gates of a trained encoder: memories of one sample to some thousands
        s["gate"] = normal(B, N, C, mean=2.0, std=2.0)
        s["state"] = normal(B, C, dtype=torch.float32) if case["state"] else None
        s["dh"] = normal(B, N, C, std=1e-2, grad=False) if train else None
        s["dlast"] = normal(B, C, std=1e-2, dtype=torch.float32, grad=False) if train and case["state"] else None
        s["lengths"] = torch.tensor(_lengths(case, N), dtype=torch.int32, device="cuda") if case["ragged"] else None
        return s
    R, K, F = case["rows"], case["K"], case["F"]
    s["x"] = normal(R, K)
    s["wg"], s["wu"] = normal(F, K, std=K ** -0.5), normal(F, K, std=K ** -0.5)
    s["bg"], s["bu"] = (normal(F, std=0.2), normal(F, std=0.2)) if case["bias"] else (None, None)
    s["dh"] = normal(R, F, std=1e-2, grad=False) if train else None
    return s


def _ops():
    import differentiable_series_alignment_gb300 as package
    return package


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "recurrence": _own_recurrence, "gated": _own_gated}[op](state)
    with torch.no_grad():
        return {"norm": _plain_norm, "recurrence": _plain_recurrence, "gated": _plain_gated}[op](state)


def _own_norm(s):
    case = s["case"]
    y = _ops().group_norm(s["x"], case["G"], s["weight"], s["bias"],
                          activation=None if case["activation"] == "none" else case["activation"], lengths=s["lengths"])
    if not case["train"]:
        return y
    return y.detach(), *torch.autograd.grad(y, (s["x"], s["weight"], s["bias"]), s["dy"])


def _own_recurrence(s):
    case = s["case"]
    h, last = _ops().gated_recurrence(s["x"], s["gate"], s["state"], lengths=s["lengths"], reverse=case["reverse"],
                                      tied=case["tied"], return_state=True)
    if not case["train"]:
        return h, last
    if case["state"]:
        return h.detach(), last.detach(), *torch.autograd.grad((h, last), (s["x"], s["gate"], s["state"]),
                                                               (s["dh"], s["dlast"]))
    return h.detach(), last.detach(), *torch.autograd.grad(h, (s["x"], s["gate"]), s["dh"])


def _own_gated(s):
    case = s["case"]
    h = _ops().gated_linear(s["x"], s["wg"], s["wu"], s["bg"], s["bu"], activation=case["activation"])
    if not case["train"]:
        return h
    leaves = (s["x"], s["wg"], s["wu"]) + ((s["bg"], s["bu"]) if case["bias"] else ())
    return h.detach(), *torch.autograd.grad(h, leaves, s["dh"])


# ---- plain forms, in fp32

def _act(name, z):
    """The activation and its derivative."""
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return z * s, s * (1 + z * (1 - s))
    if name == "gelu":
        c = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return z * c, c + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if name == "relu":
        on = (z > 0).to(z.dtype)
        return z * on, on
    if name == "sigmoid":
        s = 1 / (1 + torch.exp(-z))
        return s, s * (1 - s)
    return z, torch.ones_like(z)


def _plain_norm(s):
    case = s["case"]
    B, S, G, cg = (case[k] for k in ("B", "S", "G", "cg"))
    split = lambda t: t.float().view(-1, S if t.dim() == 3 else 1, G, cg)  # noqa: E731
    x, w, b = split(s["x"]), split(s["weight"]), split(s["bias"])
    if case["ragged"]:
        valid = (torch.arange(S, device="cuda") < s["lengths"][:, None])[:, :, None, None].float()
        n = (s["lengths"].clamp(min=1) * cg).float()[:, None, None, None]
    else:
        valid, n = 1.0, float(S * cg)
    total = lambda t: t.sum((1, 3), keepdim=True)  # noqa: E731
    xc = (x - total(x * valid) / n) * valid
    r = torch.rsqrt(total(xc * xc) / n + 1e-5)
    xh = xc * r
    y, slope = _act(case["activation"], xh * w + b)
    y = (y * valid).to(s["x"].dtype).view_as(s["x"])
    if not case["train"]:
        return y
    dz = split(s["dy"]) * slope * valid
    g = dz * w
    dx = r * (g - total(g) / n - xh * (total(g * xh) / n)) * valid
    return (y, dx.to(s["x"].dtype).view_as(s["x"]), (dz * xh).sum((0, 1)).flatten().to(s["weight"].dtype),
            dz.sum((0, 1)).flatten().to(s["bias"].dtype))


def _scan(a, u):
    """h_t = a_t h_{t-1} + u_t over dimension 1 from 0, in steps that double; (h, products of a up to t)."""
    h, p, d = u, a, 1
    while d < u.shape[1]:
        h = torch.cat([h[:, :d], h[:, d:] + p[:, d:] * h[:, :-d]], dim=1)
        p = torch.cat([p[:, :d], p[:, d:] * p[:, :-d]], dim=1)
        d *= 2
    return h, p


def _plain_recurrence(s):
    case, dtype = s["case"], s["x"].dtype
    B, N, C = case["B"], case["N"], case["C"]
    at = torch.arange(N, device="cuda")
    if case["ragged"]:
        valid = (at < s["lengths"][:, None])[..., None]
    else:
        valid = torch.ones(1, 1, 1, dtype=torch.bool, device="cuda")
    turn = (lambda t: t.flip(1)) if case["reverse"] else (lambda t: t)
    zero = torch.zeros((), device="cuda")
    x, g = s["x"].float(), s["gate"].float()
    # behind a sequence's end the state stays as it is
    a = turn(torch.where(valid, 1 / (1 + torch.exp(-g)), zero + 1))
    b = turn(torch.where(valid, 1 / (1 + torch.exp(g)), zero))          # 1 - a
    x = turn(torch.where(valid, x, zero))
    first = s["state"] if case["state"] else torch.zeros(B, C, device="cuda")
    h, p = _scan(a, b * x if case["tied"] else x)
    h = h + p * first[:, None]
    last = h[:, -1]
    out = torch.where(valid, turn(h), zero).to(dtype)
    if not case["train"]:
        return out, last
    e = turn(torch.where(valid, s["dh"].float(), zero))
    if case["state"]:
        e = torch.cat([e[:, :-1], e[:, -1:] + s["dlast"][:, None]], dim=1)
    # e_t = dh_t + a_{t+1} e_{t+1}: the same scan, backwards
    follow = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], dim=1)
    e = _scan(follow.flip(1), e.flip(1))[0].flip(1)
    before = torch.cat([first[:, None], h[:, :-1]], dim=1)
    dx = e * b if case["tied"] else e
    dg = e * (before - x if case["tied"] else before) * a * b
    back = lambda t: torch.where(valid, turn(t), zero).to(dtype)  # noqa: E731
    if case["state"]:
        return out, last, back(dx), back(dg), a[:, 0] * e[:, 0]
    return out, last, back(dx), back(dg)


def _plain_gated(s):
    case, dtype = s["case"], s["x"].dtype
    x, wg, wu = s["x"].float(), s["wg"].float(), s["wu"].float()
    g, u = x @ wg.T, x @ wu.T
    if case["bias"]:
        g, u = g + s["bg"].float(), u + s["bu"].float()
    v, slope = _act(case["activation"], g)
    h = (v * u).to(dtype)
    if not case["train"]:
        return h
    dh = s["dh"].float()
    dg, du = dh * u * slope, dh * v
    out = (h, dg @ wg + du @ wu, dg.T @ x, du.T @ x) + ((dg.sum(0), du.sum(0)) if case["bias"] else ())
    return tuple(t.to(dtype) for t in out)


def work(case):
    size, train = (4 if case["dtype"] == "fp32" else 2), case["train"]
    if case["op"] == "norm":
        C = case["G"] * case["cg"]
        rows = sum(_lengths(case, case["S"])) if case["ragged"] else case["B"] * case["S"]
        w = (4 if case["wdtype"] == "fp32" else 2) * C
        # x in, y out, the padding's zeros too; a training pass also takes dy and gives dx and the weights' gradients
        moved = (rows + case["B"] * case["S"]) * C * size
        return {"bytes": moved * (2 if train else 1) + w * (4 if train else 2), "flops": rows * C * (32 if train else 12)}
    if case["op"] == "recurrence":
        C = case["C"]
        rows = sum(_lengths(case, case["N"])) if case["ragged"] else case["B"] * case["N"]
        states = case["B"] * C * 4 * ((2 if case["state"] else 1) * (2 if train and case["state"] else 1))
        moved = (2 * rows + case["B"] * case["N"]) * C * size           # x, gate in, h out
        if train:
            moved += (rows + 2 * case["B"] * case["N"]) * C * size      # dh in, dx, dgate out
        return {"bytes": moved + states, "flops": rows * C * (20 if train else 8)}
    R, K, F = case["rows"], case["K"], case["F"]
    e, w = R * (K + F) * size, 2 * F * K * size
    b = 2 * F * size if case["bias"] else 0
    return {"bytes": (e + w + b) * (2 if train else 1), "flops": R * K * F * (12 if train else 4)}


# ---- the definitions in 64 bits; gradients by differentiating them

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "recurrence":
        with torch.no_grad():
            return _exact_recurrence(s)
    wide = {k: t.detach().double().requires_grad_() for k, t in s.items()
            if torch.is_tensor(t) and t.is_floating_point()}
    if case["op"] == "norm":
        y = _exact_norm(case, wide, s["lengths"])
        leaves, upstream = [wide[k] for k in ("x", "weight", "bias")], s["dy"]
    else:
        y = _exact_gated(case, wide)
        leaves, upstream = [wide[k] for k in ("x", "wg", "wu", "bg", "bu") if k in wide], s["dh"]
    if not case["train"]:
        return y.detach()
    return y.detach(), *torch.autograd.grad(y, leaves, upstream.double())


def _exact_act(name, z):
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if name == "relu":
        return torch.clamp(z, min=0)
    if name == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    return z


def _exact_norm(case, wide, lengths):
    B, S, G, cg = (case[k] for k in ("B", "S", "G", "cg"))
    w, b = wide["weight"].view(G, cg), wide["bias"].view(G, cg)
    if not case["ragged"]:
        t = wide["x"].view(B, S, G, cg).transpose(1, 2).reshape(B, G, S * cg)
        var, mean = torch.var_mean(t, dim=2, unbiased=False, keepdim=True)
        t = ((t - mean) / torch.sqrt(var + 1e-5)).view(B, G, S, cg).transpose(1, 2)
        return _exact_act(case["activation"], t * w + b).reshape(B, S, G * cg)
    rows = []
    for i, n in enumerate(lengths.tolist()):
        out = torch.zeros(S - n, G * cg, dtype=torch.float64, device="cuda")
        if n > 0:
            t = wide["x"][i, :n].view(n, G, cg)
            var, mean = torch.var_mean(t, dim=(0, 2), unbiased=False, keepdim=True)
            t = (t - mean) / torch.sqrt(var + 1e-5)
            out = torch.cat([_exact_act(case["activation"], t * w + b).view(n, G * cg), out])
        rows.append(out)
    return torch.stack(rows)


def _exact_gated(case, wide):
    g, u = wide["x"] @ wide["wg"].T, wide["x"] @ wide["wu"].T
    if case["bias"]:
        g, u = g + wide["bg"], u + wide["bu"]
    return _exact_act(case["activation"], g) * u


def _exact_recurrence(s):
    """Step by step."""
    case = s["case"]
    B, N, C = case["B"], case["N"], case["C"]
    n = s["lengths"] if case["ragged"] else torch.full((B,), N, device="cuda")
    live = (torch.arange(N, device="cuda")[:, None] < n)[..., None].double()       # (N, B, 1)
    x, a = s["x"].double().transpose(0, 1), torch.sigmoid(s["gate"].double()).transpose(0, 1)
    b = torch.sigmoid(-s["gate"].double()).transpose(0, 1)
    order = range(N - 1, -1, -1) if case["reverse"] else range(N)
    keep, take = a * live + (1 - live), live * (b * x if case["tied"] else x)
    h = s["state"].double() if case["state"] else torch.zeros(B, C, dtype=torch.float64, device="cuda")
    out, before = torch.empty_like(x), torch.empty_like(x)
    for t in order:
        before[t] = h
        h = torch.addcmul(take[t], keep[t], h)
        out[t] = h
    last = h
    out = (out * live).transpose(0, 1).contiguous()
    if not case["train"]:
        return out, last
    dh = s["dh"].double().transpose(0, 1) * live
    e = s["dlast"].double() if case["state"] else torch.zeros(B, C, dtype=torch.float64, device="cuda")
    es = torch.empty_like(x)
    for t in reversed(order):
        e = e + dh[t]
        es[t] = e
        e = e * keep[t]
    dx = es * live * b if case["tied"] else es * live
    dg = es * live * (before - x if case["tied"] else before) * a * b
    got = (out, last, dx.transpose(0, 1).contiguous(), dg.transpose(0, 1).contiguous())
    return (*got, e) if case["state"] else got
