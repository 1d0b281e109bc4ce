"""Cases of the sequence-encoder operators next to the Soft-DTW loss: layer norm, rotary positions and attention.

A model trained on the Soft-DTW loss turns raw series into the feature sequences that the loss aligns. Its blocks
normalise their input, turn queries and keys by their positions and attend over the sequence. ``run`` makes one call
of one of these operators, forward or forward and backward, either in plain torch operations (``own`` false) or
through this package's entry points (``own`` true).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # the newest sample of 16 streams through a normalisation: latency alone
        dict(name="norm_token", op="norm", train=False, dtype="bf16", wdtype="bf16", rows=16, C=512),
        # a training step on the loss's own feature batch, 32 sequences of 512 samples, 64 features
        dict(name="norm_features", op="norm", train=True, dtype="fp32", wdtype="fp32", rows=16384, C=64),
        # a training step of a wide encoder in mixed precision, weights kept in fp32
        dict(name="norm_wide", op="norm", train=True, dtype="bf16", wdtype="fp32", rows=65535, C=1024),
        # the newest sample of 16 streams, each at its own position; a quarter of a head turns, neighbours paired
        dict(name="rotary_token", op="rotary", train=False, dtype="bf16", B=16, N=1, Hq=8, Hkv=2, D=128, R=32,
             interleaved=True, length=8192, own_positions=True),
        # a training step over long sequences with shared key heads, whole heads turn, halves paired
        dict(name="rotary_train", op="rotary", train=True, dtype="bf16", B=4, N=4096, Hq=16, Hkv=4, D=128, R=128,
             interleaved=False, length=4096, own_positions=False),
        # the newest sample of 2 small fp32 streams over what they have seen so far: the smallest call
        dict(name="attention_stream", op="attention", train=False, dtype="fp32", B=2, N=1, M=777, Hq=4, Hkv=4, D=64,
             causal=True, window=0, ragged=False),
        # the newest sample of 16 streams over their caches, of different fill, one slot of the batch idle
        dict(name="attention_token", op="attention", train=False, dtype="bf16", B=16, N=1, M=8192, Hq=32, Hkv=8, D=128,
             causal=True, window=0, ragged=True),
        # encoding 4 long series before their first answer
        dict(name="attention_prompt", op="attention", train=False, dtype="bf16", B=4, N=4096, M=4096, Hq=16, Hkv=4,
             D=128, causal=True, window=0, ragged=False),
        # a training step on the loss's own batch, padded to 512 samples, both directions visible
        dict(name="attention_batch", op="attention", train=True, dtype="bf16", B=32, N=512, M=512, Hq=8, Hkv=8, D=64,
             causal=False, window=0, ragged=True),
        # a training step over long causal sequences with shared key heads
        dict(name="attention_long", op="attention", train=True, dtype="bf16", B=2, N=4096, M=4096, Hq=16, Hkv=4,
             D=128, causal=True, window=0, ragged=False),
        # cross attention of two series of unequal odd length inside a band, as alignment constrains it
        dict(name="attention_band", op="attention", train=True, dtype="fp16", B=3, N=1021, M=2039, Hq=6, Hkv=6, D=80,
             causal=False, window=256, ragged=False),
        # a training step in full precision, where the loss's gradients are compared against its own tolerance
        dict(name="attention_fp32", op="attention", train=True, dtype="fp32", B=8, N=512, M=512, Hq=4, Hkv=4, D=64,
             causal=False, window=0, ragged=False),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "rotary", "attention", "attention"])
    dtype = rng.choice(["fp32", "bf16", "bf16", "fp16"])
    train = rng.random() < 0.6
    if op == "norm":
        C = _log(rng, 8, 8192)
        rows = _log(rng, 1, min(65535, (1 << 26) // C))
        return dict(op=op, train=train, dtype=dtype, wdtype=rng.choice(["fp32", dtype]), rows=rows, C=C)
    Hkv = rng.randint(1, 8)
    Hq = Hkv * rng.choice([1, 1, 2, 3, 4])
    if op == "rotary":
        D = 2 * rng.randint(8, 64)
        R = rng.choice([D, 2 * rng.randint(1, D // 2)])
        B = _log(rng, 1, 16)
        N = _log(rng, 1, max(1, min(8192, (1 << 24) // (B * (Hq + Hkv) * D))))
        return dict(op=op, train=train, dtype=dtype, B=B, N=N, Hq=Hq, Hkv=Hkv, D=D, R=R,
                    interleaved=rng.random() < 0.5, length=rng.randint(N, 16384), own_positions=rng.random() < 0.5)
    B = _log(rng, 1, 32)
    D = rng.randint(4, 128) if dtype == "fp32" else 8 * rng.randint(4, 16)
    most = (3e10 if dtype == "fp32" else 2e11) / (4 * D * Hq * B)       # visible pairs of one head, at the most
    if not train and rng.random() < 0.4:                               # a few new samples over a cache
        N = rng.randint(1, 8)
        M = _log(rng, N, min(16384, (1 << 28) // (B * Hkv * D)))
        causal, ragged, window = True, rng.random() < 0.5, rng.choice([0, 0, 512])
    else:
        N = _log(rng, 1, min(4096, math.sqrt(most)))
        M = N if rng.random() < 0.6 else _log(rng, 1, min(4096, math.sqrt(most)))
        causal, ragged, window = rng.random() < 0.5, rng.random() < 0.5, rng.choice([0, 0, 64, 300])
    return dict(op=op, train=train, dtype=dtype, B=B, N=N, M=M, Hq=Hq, Hkv=Hkv, D=D, causal=causal, window=window,
                ragged=ragged)


def _lengths(case, limit, salt):
    """Lengths of a padded batch: full, down to half, and idle slots (0) where nothing is trained on."""
    got = [max(1, limit - (b * 7919 + salt) % (limit // 2 + 1)) for b in range(case["B"])]
    if not case["train"] and case["B"] >= 4:
        got[1] = 0
    return got


def _both_lengths(case):
    if not case["ragged"]:
        return [case["N"]] * case["B"], [case["M"]] * case["B"]
    keys = _lengths(case, case["M"], 3)
    if case["N"] == case["M"]:
        return keys, keys
    return [case["N"]] * case["B"], keys


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype, train = DTYPES[case["dtype"]], case["train"]

    def normal(*shape, mean=0.0, std=1.0, dtype=dtype, grad=train):
        t = (torch.randn(*shape, generator=gen, device="cuda") * std + mean).to(dtype)
        return t.requires_grad_() if grad else t

    state = {"case": case}
    if case["op"] == "norm":
        rows, C = case["rows"], case["C"]
        w = DTYPES[case["wdtype"]]
        state["x"] = normal(rows, C, mean=0.3, std=1.5)
        state["weight"] = normal(C, mean=1.0, std=0.2, dtype=w)
        state["bias"] = normal(C, std=0.2, dtype=w)
        state["dy"] = normal(rows, C, std=1e-2, grad=False) if train else None
        return state
    B, N, Hq, Hkv, D = (case[k] for k in ("B", "N", "Hq", "Hkv", "D"))
    if case["op"] == "rotary":
        # (cos, sin) of every position: what a program makes once
        angle = torch.arange(case["length"], device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(0, case["R"], 2, device="cuda", dtype=torch.float64) / case["R"])
        state["table"] = torch.stack([angle.cos(), angle.sin()], dim=-1).to(torch.float32)
        state["positions"] = torch.randint(0, case["length"], (B, N), generator=gen, device="cuda",
                                           dtype=torch.int32) if case["own_positions"] else None
        state["q"], state["k"] = normal(B, N, Hq, D), normal(B, N, Hkv, D)
        state["dq"], state["dk"] = (normal(B, N, H, D, std=1e-2, grad=False) if train else None for H in (Hq, Hkv))
        return state
    M = case["M"]
    state["q"], state["k"] = normal(B, N, Hq, D, std=1.5), normal(B, M, Hkv, D, std=1.5)
    state["v"] = normal(B, M, Hkv, D)
    state["do"] = normal(B, N, Hq, D, std=1e-2, grad=False) if train else None
    state["q_lengths"], state["k_lengths"] = (torch.tensor(n, dtype=torch.int32, device="cuda") if case["ragged"]
                                              else None for n in _both_lengths(case))
    return state


def _ops():
    import differentiable_series_alignment_gb300 as package
    return package


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "rotary": _own_rotary, "attention": _own_attention}[op](state)
    with torch.no_grad():
        return {"norm": _plain_norm, "rotary": _plain_rotary, "attention": _plain_attention}[op](state)


def _own_norm(s):
    y = _ops().layer_norm(s["x"], s["weight"], s["bias"])
    if not s["case"]["train"]:
        return y
    return y.detach(), *torch.autograd.grad(y, (s["x"], s["weight"], s["bias"]), s["dy"])


def _own_rotary(s):
    q, k = _ops().rotary(s["q"], s["k"], table=s["table"], positions=s["positions"],
                         interleaved=s["case"]["interleaved"])
    if not s["case"]["train"]:
        return q, k
    return q.detach(), k.detach(), *torch.autograd.grad((q, k), (s["q"], s["k"]), (s["dq"], s["dk"]))


def _own_attention(s):
    case = s["case"]
    out = _ops().attention(s["q"], s["k"], s["v"], causal=case["causal"], window=case["window"] or None,
                           q_lengths=s["q_lengths"], k_lengths=s["k_lengths"])
    if not case["train"]:
        return out
    return out.detach(), *torch.autograd.grad(out, (s["q"], s["k"], s["v"]), s["do"])


def _plain_norm(s):
    x, w, b = s["x"].float(), s["weight"].float(), s["bias"].float()
    xc = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((xc * xc).mean(-1, keepdim=True) + 1e-5)
    xh = xc * r
    y = (xh * w + b).to(s["x"].dtype)
    if not s["case"]["train"]:
        return y
    dy = s["dy"].float()
    dh = dy * w
    dx = r * (dh - dh.mean(-1, keepdim=True) - xh * (dh * xh).mean(-1, keepdim=True))
    return (y, dx.to(s["x"].dtype), (dy * xh).sum(0).to(s["weight"].dtype), dy.sum(0).to(s["bias"].dtype))


def _turn(x, c, s, R, interleaved, dtype):
    """x with its first R features turned in pairs by the angles whose cosines and sines are c and s."""
    t, rest = x[..., :R].to(dtype), x[..., R:].to(dtype)
    if interleaved:
        a, b = t[..., 0::2], t[..., 1::2]
        t = torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)
    else:
        a, b = t[..., :R // 2], t[..., R // 2:]
        t = torch.cat([a * c - b * s, b * c + a * s], dim=-1)
    return torch.cat([t, rest], dim=-1)


def _plain_rotary(s):
    case = s["case"]
    rows = s["table"][:case["N"]] if s["positions"] is None else s["table"][s["positions"].long()]
    c, n = rows[..., None, :, 0], rows[..., None, :, 1]
    turn = lambda x, n: _turn(x, c, n, case["R"], case["interleaved"], torch.float32).to(x.dtype)  # noqa: E731
    if not case["train"]:
        return turn(s["q"], n), turn(s["k"], n)
    return turn(s["q"], n), turn(s["k"], n), turn(s["dq"], -n), turn(s["dk"], -n)


def _visible(case, N, M, q_lengths, k_lengths):
    """(B, N, M): which keys a row sees; the last row of a sequence stands at its last key."""
    i = torch.arange(N, device="cuda")[None, :, None]
    j = torch.arange(M, device="cuda")[None, None, :]
    n = torch.tensor(q_lengths, device="cuda")[:, None, None]
    m = torch.tensor(k_lengths, device="cuda")[:, None, None]
    see = (i < n) & (j < m)
    at = i + (m - n)
    if case["causal"]:
        see = see & (j <= at)
    if case["window"]:
        see = see & (j > at - case["window"])
        if not case["causal"]:
            see = see & (j < at + case["window"])
    return see


def _plain_mask(s):
    """(B or 1, 1, 1, N, M) truth values, on the device throughout; None where every row sees every key."""
    case = s["case"]
    N, M = case["N"], case["M"]
    if not (case["causal"] or case["window"] or case["ragged"]):
        return None
    i = torch.arange(N, device="cuda", dtype=torch.int32)[:, None]
    j = torch.arange(M, device="cuda", dtype=torch.int32)
    n = s["q_lengths"][:, None, None] if case["ragged"] else N
    m = s["k_lengths"][:, None, None] if case["ragged"] else M
    at = i + (m - n)
    see = (i < n) & (j < m)
    if case["causal"]:
        see = see & (j <= at)
    if case["window"]:
        see = see & (j > at - case["window"])
        if not case["causal"]:
            see = see & (j < at + case["window"])
    return see.view(-1, 1, 1, N, M)


def _plain_attention(s):
    case = s["case"]
    B, N, M, Hq, Hkv, D = (case[k] for k in ("B", "N", "M", "Hq", "Hkv", "D"))
    G, scale, dtype = Hq // Hkv, D ** -0.5, s["q"].dtype
    heads = lambda x: x.float().view(B, -1, Hkv, x.shape[2] // Hkv, D).permute(0, 2, 3, 1, 4)  # noqa: E731
    back = lambda x: x.permute(0, 3, 1, 2, 4).reshape(B, x.shape[3], -1, D).to(dtype)  # noqa: E731
    q, k, v = heads(s["q"]), heads(s["k"]), heads(s["v"])                       # (B, Hkv, G or 1, length, D)
    score = (q * scale) @ k.transpose(-1, -2)                                   # (B, Hkv, G, N, M)
    mask = _plain_mask(s)
    if mask is not None:
        score = score.masked_fill_(~mask, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    o = p @ v
    if not case["train"]:
        return back(o)
    do = heads(s["do"])
    dp = do @ v.transpose(-1, -2)
    ds = p * (dp - (do * o).sum(-1, keepdim=True))
    dq = ds @ k * scale
    dk = (ds.transpose(-1, -2) @ q).sum(2, keepdim=True) * scale
    dv = (p.transpose(-1, -2) @ do).sum(2, keepdim=True)
    return back(o), back(dq), back(dk), back(dv)


def _pairs(case):
    """Visible (row, key) pairs of one head, over the batch."""
    total = 0
    for n, m in zip(*_both_lengths(case)):
        at = np.arange(n, dtype=np.int64) + (m - n)
        high = np.minimum(m, at + 1) if case["causal"] else np.full(n, m)
        low = np.zeros(n, dtype=np.int64)
        if case["window"]:
            low = np.maximum(0, at - case["window"] + 1)
            if not case["causal"]:
                high = np.minimum(m, at + case["window"])
        total += int(np.maximum(0, high - low).sum())
    return total


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "norm":
        e, w = case["rows"] * case["C"], (4 if case["wdtype"] == "fp32" else 2) * case["C"]
        # forward: x in, y out; a training pass also takes dy and gives dx and the weights' gradients
        return {"bytes": e * size * (4 if case["train"] else 2) + w * (4 if case["train"] else 2),
                "flops": e * (18 if case["train"] else 8)}
    B, N, Hq, Hkv, D = (case[k] for k in ("B", "N", "Hq", "Hkv", "D"))
    if case["op"] == "rotary":
        turns = 2 if case["train"] else 1
        table = (B * N if case["own_positions"] else N) * case["R"] * 4
        return {"bytes": turns * 2 * B * N * (Hq + Hkv) * D * size + table,
                "flops": turns * 3 * B * N * (Hq + Hkv) * case["R"]}
    rows, keys = (sum(n) for n in _both_lengths(case))
    passes = 2 if case["train"] else 1           # q, k, v in and o out; then do in and dq, dk, dv out
    return {"bytes": passes * (B * N * Hq + rows * Hq + 2 * (keys if passes == 1 else B * case["M"]) * Hkv) * D * size,
            "flops": _pairs(case) * Hq * D * (14 if case["train"] else 4)}


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if case["op"] == "norm":
            return _exact_norm(s)
        if case["op"] == "rotary":
            return _exact_rotary(s)
        if work(case)["flops"] > 4e12:
            return None
        return _exact_attention(s)


def _exact_norm(s):
    x, w, b = s["x"].double(), s["weight"].double(), s["bias"].double()
    var, mean = torch.var_mean(x, dim=1, unbiased=False, keepdim=True)
    std = torch.sqrt(var + 1e-5)
    y = (x - mean) / std * w + b
    if not s["case"]["train"]:
        return y
    dy, C = s["dy"].double(), x.shape[1]
    u = (x - mean) / std
    g = dy * w
    dx = (C * g - g.sum(1, keepdim=True) - u * (g * u).sum(1, keepdim=True)) / (C * std)
    return y, dx, torch.einsum("rc,rc->c", dy, u), dy.sum(0)


def _exact_rotary(s):
    case = s["case"]
    R, N = case["R"], case["N"]
    rows = s["table"][:N].expand(case["B"], N, R // 2, 2) if s["positions"] is None else s["table"][s["positions"].long()]
    turn = torch.view_as_complex(rows.double().contiguous())[:, :, None]

    def turned(x, by):
        x = x.double()
        pairs = x[..., :R].unflatten(-1, (R // 2, 2) if case["interleaved"] else (2, R // 2))
        if not case["interleaved"]:
            pairs = pairs.transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * by)
        z = z if case["interleaved"] else z.transpose(-1, -2)
        return torch.cat([z.flatten(-2), x[..., R:]], dim=-1)

    if not case["train"]:
        return turned(s["q"], turn), turned(s["k"], turn)
    return (turned(s["q"], turn), turned(s["k"], turn), turned(s["dq"], turn.conj()), turned(s["dk"], turn.conj()))


def _exact_attention(s):
    case = s["case"]
    B, N, M, Hq, Hkv, D = (case[k] for k in ("B", "N", "M", "Hq", "Hkv", "D"))
    see = _visible(case, N, M, *_both_lengths(case))
    shared = Hq // Hkv
    o = torch.zeros(B, N, Hq, D, dtype=torch.float64, device="cuda")
    dq, dk, dv = (torch.zeros(B, L, H, D, dtype=torch.float64, device="cuda")
                  for L, H in ((N, Hq), (M, Hkv), (M, Hkv)))
    for b in range(B):
        for h in range(Hq):
            q, k, v = s["q"][b, :, h].double(), s["k"][b, :, h // shared].double(), s["v"][b, :, h // shared].double()
            z = (q @ k.T / math.sqrt(D)).masked_fill(~see[b], -math.inf)
            p = torch.nan_to_num(torch.softmax(z, dim=1), nan=0.0)      # a row that sees nothing
            o[b, :, h] = p @ v
            if case["train"]:
                g = s["do"][b, :, h].double()
                dz = g @ v.T
                dz = p * (dz - (p * dz).sum(1, keepdim=True))
                dq[b, :, h] = dz @ k / math.sqrt(D)
                dk[b, :, h // shared] += dz.T @ q / math.sqrt(D)
                dv[b, :, h // shared] += p.T @ g
    return (o, dq, dk, dv) if case["train"] else o
