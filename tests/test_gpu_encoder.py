"""Layer norm, rotary positions and attention on the GPU against their definitions in 64 bits.

Tolerances are bounds, element by element, of what the arithmetic of the operators can be off by
(first order in the unit roundoffs), evaluated in 64 bits beside each result:

  u32 = 2^-24 (fp32), ut = 2^-24 / 2^-8 / 2^-11 (one rounding to fp32 / bf16 / fp16, to nearest or not)
  a sum of n terms in fp32, in any order, truncating or rounding: n * 2 * u32 * sum |terms|
  ex2: 2^-22 relative; its argument, a sum of D products less a maximum of their size, adds
  (2 D + 6) u32 * (scale sum |q||k| + its maximum over the row) to the relative error of a probability

and a 16-bit result, or a probability rounded to 16 bits before the product that consumes it, adds ut of
itself. fp16 adds its smallest step (2^-24) to every rounding that can be subnormal.
"""
import importlib.util
import math
import os

import pytest

from helpers import ensure_built

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U32 = 2.0 ** -24
UT = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}
TINY = {F32: 2.0 ** -126, BF16: 2.0 ** -126, F16: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def package():
    ensure_built()
    import differentiable_series_alignment_gb300 as p
    p.load()
    return p


def randn(gen, *shape, dtype=F32, std=1.0, mean=0.0):
    return (torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float64) * std + mean).to(dtype)


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def within(got, want, bound, what):
    got, bound = got.double(), bound.expand_as(want)
    assert got.shape == want.shape, what
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - want).abs() / bound
    k = int(over.argmax())
    assert float(over.max()) <= 1.0, (f"{what}: off by {float(over.max()):.3g} of its bound at {k}: "
                                     f"{float(got.flatten()[k])!r}, not {float(want.flatten()[k])!r}")


# --- layer norm ---------------------------------------------------------------------------------

NORM_SHAPES = [(1, 1), (3, 2), (5, 7), (16, 64), (33, 100), (9, 128), (257, 256), (4, 1000), (31, 1003), (700, 1024),
               (3, 1536), (2, 4096), (5, 8192), (3, 8200), (2, 20011)]


def norm_reference(x, w, b, dy, eps, dtype, wdtype):
    """(y, dx, dw, db) and their bounds."""
    x, dy = x.double(), dy.double()
    C, R = x.shape[1], x.shape[0]
    w = torch.ones(C, device="cuda", dtype=torch.float64) if w is None else w.double()
    b = torch.zeros(C, device="cuda", dtype=torch.float64) if b is None else b.double()
    mu = x.mean(1, keepdim=True)
    var = ((x - mu) ** 2).mean(1, keepdim=True)
    r = (var + eps) ** -0.5
    xh = (x - mu) * r
    # relative to the spread of the row: the mean's error, that of the centred value, and the root's
    dmu = (2 * C + 2) * U32 * x.abs().mean(1, keepdim=True)
    dr = r * ((2 * C + 8) * U32 + r * dmu)                  # through the variance: 2 r^2 (dev) dmu <= r dmu, halved
    dxh = (dmu + 2 * U32 * (x.abs() + mu.abs())) * r + (x - mu).abs() * dr
    y = xh * w + b
    by = dxh * w.abs() + 3 * U32 * ((xh * w).abs() + b.abs()) + UT[dtype] * y.abs() + TINY[dtype]
    g = dy * w
    m1, m2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = r * (g - m1 - xh * m2)
    dm1 = (2 * C + 2) * U32 * g.abs().mean(1, keepdim=True)
    dm2 = (2 * C + 4) * U32 * (g * xh).abs().mean(1, keepdim=True) + (g.abs() * dxh).mean(1, keepdim=True)
    bdx = (r * (dm1 + xh.abs() * dm2 + dxh * m2.abs() + 6 * U32 * (g.abs() + m1.abs() + (xh * m2).abs()))
           + dr * (dx / r).abs() + UT[dtype] * dx.abs() + TINY[dtype])
    dw, db = (dy * xh).sum(0), dy.sum(0)
    bdw = (2 * R + 4) * U32 * (dy * xh).abs().sum(0) + (dy.abs() * dxh).sum(0) + UT[wdtype] * dw.abs() + TINY[wdtype]
    bdb = (2 * R + 2) * U32 * dy.abs().sum(0) + UT[wdtype] * db.abs() + TINY[wdtype]
    return (y, by), (dx, bdx), (dw, bdw), (db, bdb)


@pytest.mark.parametrize("dtype,wdtype", [(F32, F32), (BF16, F32), (BF16, BF16), (F16, F16)])
@pytest.mark.parametrize("rows,C", NORM_SHAPES)
def test_norm_and_its_gradients(package, rows, C, dtype, wdtype):
    gen = generator(rows * 31 + C)
    x = randn(gen, rows, C, dtype=dtype, std=1.7, mean=0.6).requires_grad_()
    w = randn(gen, C, dtype=wdtype, std=0.3, mean=1.0).requires_grad_()
    b = randn(gen, C, dtype=wdtype, std=0.3).requires_grad_()
    dy = randn(gen, rows, C, dtype=dtype, std=0.1)
    with torch.no_grad():
        alone = package.layer_norm(x, w, b, 1e-3)
    y = package.layer_norm(x, w, b, 1e-3)
    assert torch.equal(y, alone)
    got = (y, *torch.autograd.grad(y, (x, w, b), dy))
    for name, g, (want, bound) in zip(("y", "dx", "dw", "db"), got, norm_reference(x.detach(), w.detach(), b.detach(), dy, 1e-3, dtype, wdtype)):
        assert g.dtype == (dtype if name in ("y", "dx") else wdtype)
        within(g.detach(), want, bound, f"{name} of {rows} x {C}")


def test_norm_without_weights_odd_addresses_and_many_dimensions(package):
    gen = generator(5)
    flat = randn(gen, 1 + 6 * 5 * 64, dtype=BF16)
    x = flat[1:].view(6, 5, 64)                                    # two bytes off a 16-byte boundary
    (want, bound), *_ = norm_reference(x.reshape(30, 64), None, None, torch.zeros(30, 64, device="cuda"), 1e-5, BF16, F32)
    within(package.layer_norm(x).reshape(30, 64), want, bound, "unaligned")
    t = randn(gen, 64, 40).T                                       # not contiguous
    (want, bound), *_ = norm_reference(t, None, None, torch.zeros(40, 64, device="cuda"), 1e-5, F32, F32)
    within(package.layer_norm(t), want, bound, "transposed")
    b = randn(gen, 64)
    (want, bound), *_ = norm_reference(t, None, b, torch.zeros(40, 64, device="cuda"), 1e-5, F32, F32)
    within(package.layer_norm(t, None, b), want, bound, "bias alone")


def test_norm_of_a_large_offset_keeps_the_spread(package):
    """Values of 1000 that differ in their last bits: sums of squares less a squared mean would lose all of it."""
    gen = generator(6)
    x = 1000.0 + randn(gen, 8, 512, std=0.25)
    (want, bound), *_ = norm_reference(x, None, None, torch.zeros_like(x), 1e-5, F32, F32)
    within(package.layer_norm(x), want, bound, "offset")
    constant = torch.full((3, 96), 7.0, device="cuda")
    assert torch.equal(package.layer_norm(constant), torch.zeros_like(constant))


def test_norm_gradient_against_differences(package):
    gen = generator(7)
    x, w, b, dy = randn(gen, 3, 9), randn(gen, 9, mean=1.0), randn(gen, 9), randn(gen, 3, 9)
    x.requires_grad_(), w.requires_grad_(), b.requires_grad_()
    grads = torch.autograd.grad(package.layer_norm(x, w, b), (x, w, b), dy)
    def value(x, w, b):
        xd = x.double()
        xc = xd - xd.mean(1, keepdim=True)
        return float(((xc / ((xc ** 2).mean(1, keepdim=True) + 1e-5).sqrt() * w.double() + b.double()) * dy.double()).sum())
    h = 1e-4      # central differences in 64 bits: h^2 f''' / 6 < 1e-7 here, fp32 gradients ~1e-6
    for t, g in zip((x, w, b), grads):
        for k in range(t.numel()):
            e = torch.zeros(t.numel(), device="cuda", dtype=torch.float64)
            e[k] = h
            args = lambda s: [u.detach().double() + (s * e.view_as(u) if u is t else 0) for u in (x, w, b)]  # noqa: E731
            assert float(g.flatten()[k]) == pytest.approx((value(*args(1)) - value(*args(-1))) / (2 * h), rel=1e-4, abs=1e-5)


# --- rotary positions ---------------------------------------------------------------------------

def rotated(x, table, positions, interleaved, inverse=False):
    """The definition in 64 bits and its bound: two products and one sum, rounded."""
    R, N = 2 * table.shape[1], x.shape[1]
    rows = table.double()[torch.arange(N, device="cuda") if positions is None else positions.long()]
    c, s = rows[..., None, :, 0], rows[..., None, :, 1] * (-1 if inverse else 1)
    if rows.dim() == 3:
        c, s = c[None], s[None]
    dt, x = x.dtype, x.double()
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., :R // 2], x[..., R // 2:R])
    out, size = x.clone(), x.abs().clone()
    first, second, fsize, ssize = a * c - b * s, b * c + a * s, (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    if interleaved:
        out[..., 0:R:2], out[..., 1:R:2], size[..., 0:R:2], size[..., 1:R:2] = first, second, fsize, ssize
    else:
        out[..., :R // 2], out[..., R // 2:R], size[..., :R // 2], size[..., R // 2:R] = first, second, fsize, ssize
    return out, 3 * U32 * size + UT[dt] * out.abs() + TINY[dt]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,N,Hq,Hkv,D,R", [(1, 1, 1, 1, 2, 2), (2, 1, 8, 2, 64, 32), (3, 37, 4, 4, 80, 80), (2, 129, 5, 1, 66, 34),
                                            (1, 2100, 8, 8, 128, 128), (2, 50, 3, 2, 7, 4), (1, 9, 2, 2, 96, 48)])
def test_rotary_and_its_gradient(package, B, N, Hq, Hkv, D, R, interleaved, dtype):
    gen = generator(B * 1000 + N + D)
    table = package.rotary_table(4096, R)
    q, k = randn(gen, B, N, Hq, D, dtype=dtype).requires_grad_(), randn(gen, B, N, Hkv, D, dtype=dtype).requires_grad_()
    dq, dk = randn(gen, B, N, Hq, D, dtype=dtype), randn(gen, B, N, Hkv, D, dtype=dtype)
    each = torch.randint(0, 4096, (B, N), generator=gen, device="cuda", dtype=torch.int32)
    for positions in (None, each, each[0].long()):
        out = package.rotary(q, k, table=table, positions=positions, interleaved=interleaved)
        grads = torch.autograd.grad(out, (q, k), (dq, dk))
        for name, got, x, inverse in (("q", out[0], q, False), ("k", out[1], k, False), ("dq", grads[0], dq, True), ("dk", grads[1], dk, True)):
            want, bound = rotated(x.detach(), table, positions, interleaved, inverse)
            within(got.detach(), want, bound, name)
    assert torch.equal(package.rotary(q.detach(), table=table, interleaved=interleaved),
                       package.rotary(q.detach(), k.detach(), table=table, interleaved=interleaved)[0])


def test_rotary_of_slices_of_one_projection(package):
    gen = generator(8)
    table = package.rotary_table(64, 64)
    packed = randn(gen, 2, 33, 6, 64, dtype=BF16)
    q, k = packed[:, :, :4], packed[:, :, 4:5]
    for got, x in zip(package.rotary(q, k, table=table), (q, k)):
        within(got, *rotated(x, table, None, False), "slice")
    odd = randn(gen, 2, 33, 2, 65, dtype=BF16)[..., 1:]            # features begin off a 16-byte boundary
    within(package.rotary(odd, table=table), *rotated(odd, table, None, False), "odd slice")
    turned = randn(gen, 2, 64, 2, 33).transpose(1, 3)              # features are not contiguous
    within(package.rotary(turned, table=table), *rotated(turned, table, None, False), "transposed")


def test_rotary_positions_outside_the_table_give_nan(package):
    table = package.rotary_table(16, 4)
    x = torch.ones(1, 4, 1, 6, device="cuda")
    got = package.rotary(x, table=table, positions=torch.tensor([3, 16, -1, 15], device="cuda"))
    assert torch.isnan(got[0, 1:3, 0, :4]).all() and torch.isfinite(got[0, [0, 3]]).all()
    assert torch.equal(got[..., 4:], x[..., 4:])


# --- attention ----------------------------------------------------------------------------------

def visible(B, N, M, causal, window, ql, kl):
    i = torch.arange(N, device="cuda")[None, :, None]
    j = torch.arange(M, device="cuda")[None, None, :]
    n = torch.full((B,), N, device="cuda") if ql is None else ql.clamp(0, N)
    m = torch.full((B,), M, device="cuda") if kl is None else kl.clamp(0, M)
    n, m = n[:, None, None], m[:, None, None]
    see, at = (i < n) & (j < m), i + (m - n)
    if causal:
        see = see & (j <= at)
    if window:
        see = see & ((at - j) < window) & ((j - at) < window)
    return see


def attention_reference(q, k, v, do, scale, see, dtype, tc):
    """{name: (value, bound)}, and lse. tc: probabilities and their gradients are rounded to the type."""
    q, k, v, do = (t.double().transpose(1, 2) for t in (q, k, v, do))      # (B, H, L, D)
    B, Hq, N, D = q.shape
    Hkv, M = k.shape[1], k.shape[2]
    G = Hq // Hkv
    live_k, live_q = see.any(1)[:, None, :, None], see.any(2)[:, None, :, None]
    k, v = (torch.where(live_k, t, 0.0).repeat_interleave(G, 1) for t in (k, v))
    q, do = torch.where(live_q, q, 0.0), torch.where(live_q, do, 0.0)
    see = see[:, None]
    s = (q @ k.mT * scale).masked_fill(~see, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    lse = (torch.log(total) + top)[..., 0]
    p = torch.where(total > 0, p / total, 0.0)
    ut, tiny = UT[dtype], TINY[dtype]
    up = ut if tc else U32
    size = torch.where(see, q.abs() @ k.abs().mT * scale, 0.0)
    es = (2 * D + 6) * U32 * (size + size.amax(-1, keepdim=True)) + 2.0 ** -21   # of a probability, relative
    # fp16 probabilities below its normal range keep an absolute step of 2^-25 of the row's largest
    low = 2.0 ** -25 if (tc and dtype == F16) else 0.0
    n = 2 * M * U32
    pe = p * (2 * es.amax(-1, keepdim=True) + up + n) + low * see
    o = p @ v
    bo = pe @ v.abs() + n * (p @ v.abs()) + ut * o.abs() + tiny
    dp = do @ v.mT
    delta = (do * o).sum(-1, keepdim=True)
    edp = 2 * D * U32 * (do.abs() @ v.abs().mT)
    # delta from o as it was rounded and what that left: ut^2 of o, and what bounds o's own error
    eo = pe @ v.abs() + n * (p @ v.abs()) + (ut * ut + U32) * o.abs() + tiny * (ut if tc else 1)
    edelta = (do.abs() * eo).sum(-1, keepdim=True) + 2 * D * U32 * (do * o).abs().sum(-1, keepdim=True)
    ds = p * (dp - delta)
    eds = (ds.abs() * (2 * es.amax(-1, keepdim=True) + up) + p * (edp + edelta + 2 * U32 * (dp.abs() + delta.abs()))
           + (low * (dp.abs() + delta.abs()).amax() * see))
    dq = ds @ k * scale
    bdq = (eds @ k.abs() + n * (ds.abs() @ k.abs())) * scale + ut * dq.abs() + tiny
    nr = 2 * N * G * U32
    fold = lambda t: t.unflatten(1, (Hkv, G)).sum(2)  # noqa: E731
    dk, dv = fold(ds.mT @ q) * scale, fold(p.mT @ do)
    bdk = fold(eds.mT @ q.abs() + nr * (ds.abs().mT @ q.abs())) * scale + ut * dk.abs() + tiny
    bdv = fold(pe.mT @ do.abs() + nr * (p.mT @ do.abs())) + ut * dv.abs() + tiny
    back = lambda t: t.transpose(1, 2)  # noqa: E731
    return {"out": (back(o), back(bo)), "dq": (back(dq), back(bdq)), "dk": (back(dk), back(bdk)),
            "dv": (back(dv), back(bdv))}, lse, es.amax(-1)


def check_attention(package, q, k, v, do, dtype, causal=False, window=None, ql=None, kl=None, scale=None):
    (B, N, Hq, D), M = q.shape, k.shape[1]
    leaves = [t.detach().requires_grad_() for t in (q, k, v)]
    args = dict(causal=causal, window=window, q_lengths=ql, k_lengths=kl, scale=scale)
    out, lse = package.attention(*leaves, return_lse=True, **args)
    grads = torch.autograd.grad(out, leaves, do)
    with torch.no_grad():
        assert torch.equal(package.attention(q, k, v, **args), out)
    again = torch.autograd.grad(package.attention(*leaves, **args), leaves, do)
    for a, b in zip(grads, again):
        assert torch.equal(a, b)                                  # the same bits every time
    see = visible(B, N, M, causal, window, ql, kl)
    want, wlse, es = attention_reference(q, k, v, do, scale or D ** -0.5, see, dtype, dtype != F32)
    for name, got in zip(("out", "dq", "dk", "dv"), (out, *grads)):
        assert got.dtype == dtype
        within(got.detach(), *want[name], f"{name} of {tuple(q.shape)} x {tuple(k.shape)}")
    none = ~see.any(2)[:, None, :].expand_as(wlse)
    assert torch.isneginf(lse[none]).all()
    assert (out.transpose(1, 2)[none] == 0).all() and (grads[0].transpose(1, 2)[none] == 0).all()
    off = (lse.double() - wlse)[~none].abs() - (2 * es + 4 * U32 * wlse.abs() + 2 * M * U32)[~none]
    assert off.numel() == 0 or float(off.max()) <= 0


SHAPES = [  # B, N, M, Hq, Hkv, D
    (1, 1, 1, 1, 1, 1), (2, 1, 5, 2, 1, 8), (1, 3, 2, 1, 1, 64), (2, 17, 33, 4, 2, 40), (1, 64, 64, 2, 2, 64),
    (2, 100, 100, 6, 2, 80), (1, 129, 257, 3, 1, 128), (1, 300, 300, 8, 8, 32), (3, 5, 700, 6, 2, 96), (1, 511, 130, 5, 5, 16),
    (1, 130, 513, 7, 1, 72), (1, 700, 700, 2, 1, 128), (2, 96, 48, 2, 2, 24), (1, 385, 385, 3, 3, 63),
]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("causal,window", [(False, None), (True, None), (False, 20), (True, 70)])
def test_attention_and_its_gradients(package, shape, causal, window, dtype):
    B, N, M, Hq, Hkv, D = shape
    gen = generator(N * 7 + M + D)
    q, do = randn(gen, B, N, Hq, D, dtype=dtype, std=1.5), randn(gen, B, N, Hq, D, dtype=dtype, std=0.3)
    k, v = randn(gen, B, M, Hkv, D, dtype=dtype, std=1.5), randn(gen, B, M, Hkv, D, dtype=dtype)
    check_attention(package, q, k, v, do, dtype, causal, window)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("causal,window", [(False, None), (True, None), (True, 33)])
@pytest.mark.parametrize("N,M,D", [(150, 290, 64), (200, 200, 128), (1, 300, 128), (7, 1000, 40), (260, 90, 63)])
def test_attention_of_padded_batches(package, N, M, D, causal, window, dtype):
    """Lengths from none to all, beyond the limits too; what lies past them is NaN and infinite."""
    gen = generator(N + M)
    B, Hq, Hkv = 6, 4, 2
    ql = torch.tensor([N, 0, max(1, N // 3), N, N // 2, N + 5], device="cuda", dtype=torch.int32)
    kl = torch.tensor([M, M // 2, M // 3, 0, 1, M + 9], device="cuda", dtype=torch.int32)
    q, do = randn(gen, B, N, Hq, D, dtype=dtype, std=1.5), randn(gen, B, N, Hq, D, dtype=dtype, std=0.3)
    k, v = randn(gen, B, M, Hkv, D, dtype=dtype, std=1.5), randn(gen, B, M, Hkv, D, dtype=dtype)
    for b in range(B):
        q[b, max(0, int(ql[b])):], do[b, max(0, int(ql[b])):] = math.nan, math.inf
        k[b, max(0, int(kl[b])):], v[b, max(0, int(kl[b])):] = math.nan, -math.inf
    check_attention(package, q, k, v, do, dtype, causal, window, ql, kl)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("D", [40, 64, 128])
@pytest.mark.parametrize("N,G,M", [(1, 1, 3001), (1, 4, 2048), (3, 3, 1300), (2, 8, 1111)])
def test_attention_of_few_rows_over_long_caches(package, N, G, M, D, dtype):
    """New samples over caches of many key tiles, full, odd and empty."""
    gen = generator(M + D)
    q, do = randn(gen, 3, N, 2 * G, D, dtype=dtype, std=1.5), randn(gen, 3, N, 2 * G, D, dtype=dtype, std=0.3)
    k, v = randn(gen, 3, M, 2, D, dtype=dtype, std=1.5), randn(gen, 3, M, 2, D, dtype=dtype)
    kl = torch.tensor([M, 0, M // 2 + 1], device="cuda", dtype=torch.int32)
    for args in (dict(causal=True, kl=kl), dict(), dict(causal=True, window=700)):
        check_attention(package, q, k, v, do, dtype, **args)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("N,M,Hq,Hkv,D", [(1100, 1100, 2, 1, 128), (1300, 2050, 2, 2, 64), (2049, 1153, 3, 1, 128), (600, 1500, 3, 3, 40),
                                          (1024, 1024, 4, 1, 96), (1537, 1537, 6, 2, 64)])
@pytest.mark.parametrize("causal,window,ragged", [(True, None, False), (False, None, True), (True, 600, False), (False, 900, True)])
def test_attention_of_long_sequences(package, N, M, Hq, Hkv, D, causal, window, ragged, dtype):
    """More tiles of rows and keys than a CTA has in flight, in every order of masks."""
    gen = generator(N + M + D)
    q, do = randn(gen, 2, N, Hq, D, dtype=dtype, std=1.5), randn(gen, 2, N, Hq, D, dtype=dtype, std=0.3)
    k, v = randn(gen, 2, M, Hkv, D, dtype=dtype, std=1.5), randn(gen, 2, M, Hkv, D, dtype=dtype)
    lengths = lambda n: torch.tensor([n - 3, n // 3], device="cuda", dtype=torch.int32) if ragged else None  # noqa: E731
    check_attention(package, q, k, v, do, dtype, causal, window, lengths(N), lengths(M))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("N,G,M,D", [(1, 1, 1, 4), (1, 2, 70, 32), (2, 1, 300, 60), (1, 3, 513, 124), (3, 1, 65, 20), (4, 1, 1000, 36),
                                     (2, 2, 31, 100), (5, 1, 200, 28), (2, 8, 90, 52), (17, 1, 90, 52)])
def test_attention_of_one_to_seventeen_rows(package, N, G, M, D, dtype):
    """Heads in packs of four features: of 16 bits, they do not fit the tensor cores."""
    gen = generator(N + G + M + D)
    q, do = randn(gen, 3, N, 2 * G, D, dtype=dtype, std=1.5), randn(gen, 3, N, 2 * G, D, dtype=dtype, std=0.3)
    k, v = randn(gen, 3, M, 2, D, dtype=dtype, std=1.5), randn(gen, 3, M, 2, D, dtype=dtype)
    kl = torch.tensor([M, 0, M // 2 + 1], device="cuda", dtype=torch.int32)
    ql = torch.tensor([N, N, max(N - 1, 0)], device="cuda", dtype=torch.int32)
    for args in (dict(causal=True, kl=kl), dict(), dict(window=9), dict(causal=True, window=40, ql=ql, kl=kl)):
        check_attention(package, q, k, v, do, dtype, **args)


@pytest.mark.parametrize("N,G", [(1, 1), (2, 1), (1, 4), (2, 8), (40, 2)])
@pytest.mark.parametrize("dtype,D", [(F32, 64), (F32, 63), (BF16, 60), (BF16, 64)])
def test_what_no_row_sees_may_be_nan(package, N, G, dtype, D):
    """Keys and values past the lengths or out of every row's window leave no trace, NaN or not."""
    gen = generator(N * G + D)
    q = randn(gen, 2, N, 2 * G, D, dtype=dtype)
    k, v = randn(gen, 2, 700, 2, D, dtype=dtype), randn(gen, 2, 700, 2, D, dtype=dtype)
    kl = torch.tensor([650, 333], device="cuda", dtype=torch.int32)
    want = package.attention(q, k, v, causal=True, window=128, k_lengths=kl)
    for t in (k, v):
        for b, m in enumerate((650, 333)):
            t[b, m:] = float("nan")
            t[b, :(m - N - 127) // 256 * 256] = float("nan")    # whole tiles before the first row's window
    assert torch.equal(package.attention(q, k, v, causal=True, window=128, k_lengths=kl), want)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attention_of_slices_and_of_unaligned_heads(package, dtype):
    gen = generator(11)
    packed = randn(gen, 2, 90, 8, 64, dtype=dtype)                 # one projection's q, k and v
    q, k, v = packed[:, :, :4], packed[:, :, 4:6], packed[:, :, 6:]
    do = randn(gen, 2, 90, 4, 64, dtype=dtype)
    check_attention(package, q, k, v, do, dtype, causal=True)
    heads_first = randn(gen, 2, 4, 90, 64, dtype=dtype).transpose(1, 2)
    check_attention(package, heads_first, k, v, do, dtype)
    wide = randn(gen, 2, 90, 2, 65, dtype=dtype)                   # features begin off a 16-byte boundary
    check_attention(package, q, wide[..., 1:], v, do, dtype)
    cache = randn(gen, 2, 400, 2, 64, dtype=dtype)[:, :90]
    check_attention(package, q, cache, cache, do, dtype, causal=True)
    one = randn(gen, 1, 90, 1, 64, dtype=dtype).expand(2, 90, 2, 64)   # broadcast keys: strides of 0
    check_attention(package, q, one, v, do, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_attention_of_large_scores_and_of_equal_ones(package, dtype):
    gen = generator(12)
    q, k, v, do = (randn(gen, 1, 140, 2, 64, dtype=dtype) for _ in range(4))
    check_attention(package, q, k, v, do, dtype, scale=4.0)                         # a row is nearly one key
    check_attention(package, torch.zeros_like(q), k, v, do, dtype, causal=True)     # every key alike
    rising = (k.float() * 0 + torch.linspace(-1, 1, 140, device="cuda")[None, :, None, None]).to(dtype)
    check_attention(package, q.abs(), rising, v, do, dtype, scale=1.0)              # the maximum moves with every tile


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_attention_gradients_of_small_and_large_upstream_values(package, dtype):
    """A mean over a batch makes upstream gradients small; none of dS may be lost to the type's range."""
    gen = generator(13)
    q, k, v, do = (randn(gen, 1, 200, 2, 64, dtype=dtype) for _ in range(4))
    leaves = [t.requires_grad_() for t in (q, k, v)]
    base = torch.autograd.grad(package.attention(*leaves), leaves, do)
    for factor in (2.0 ** -10, 2.0 ** 6):
        scaled = torch.autograd.grad(package.attention(*leaves), leaves, do * factor)
        for a, b, name in zip(base, scaled, ("dq", "dk", "dv")):
            # powers of two pass through but for fp16's smallest step at either end of the kernel
            assert float((b.double() / factor - a.double()).abs().max()) <= (TINY[dtype] / factor if dtype == F16 else 0.0) + UT[dtype] * float(a.double().abs().max()), name


def test_attention_gradient_against_differences(package):
    gen = generator(14)
    q, k, v, do = randn(gen, 1, 4, 2, 5), randn(gen, 1, 6, 1, 5), randn(gen, 1, 6, 1, 5), randn(gen, 1, 4, 2, 5)
    leaves = [t.requires_grad_() for t in (q, k, v)]
    grads = torch.autograd.grad(package.attention(*leaves, causal=True, window=4), leaves, do)
    see = visible(1, 4, 6, True, 4, None, None)
    def value(q, k, v):
        return float((attention_reference(q, k, v, do, 5 ** -0.5, see, F32, False)[0]["out"][0] * do.double()).sum())
    h = 1e-4
    for t, g in zip(leaves, grads):
        for at in range(t.numel()):
            e = torch.zeros(t.numel(), device="cuda", dtype=torch.float64)
            e[at] = h
            args = lambda s: [u.detach().double() + (s * e.view_as(u) if u is t else 0) for u in leaves]  # noqa: E731
            assert float(g.flatten()[at]) == pytest.approx((value(*args(1)) - value(*args(-1))) / (2 * h), rel=1e-4, abs=1e-5)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_over_a_cache_whose_offsets_pass_32_bits(package, dtype):
    M, H, D = (1 << 31) // 256 + 1000, 2, 128                      # 2^31 elements and more
    cache = torch.zeros(1, M, H, D, device="cuda", dtype=dtype)
    gen = generator(15)
    cache[:, -300:] = randn(gen, 1, 300, H, D, dtype=dtype)
    q = randn(gen, 1, 2, 4, D, dtype=dtype)
    tail = cache[:, -300:]
    got = package.attention(q, cache, cache, causal=True, window=200)
    want = package.attention(q, tail, tail, causal=True, window=200)
    near = 2 * UT[dtype] * float(tail.abs().max())                  # the split of the keys differs
    assert float((got.double() - want.double()).abs().max()) <= near + 1e-5


def test_attention_on_another_stream_and_in_a_graph(package):
    gen = generator(16)
    q, k, v = (randn(gen, 2, 256, 4, 64, dtype=BF16) for _ in range(3))
    want = package.attention(q, k, v, causal=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = package.attention(q, k, v, causal=True)
    side.synchronize()
    assert torch.equal(got, want)
    one, cache = q[:, :1], torch.randn(2, 3000, 4, 64, device="cuda", generator=gen).to(BF16)
    want = package.attention(one, cache, cache)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = package.attention(one, cache, cache)
    kept.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(kept, want)
    assert package.sdtw_encoder_status() == 0


def test_a_wait_that_runs_out_is_reported(package):
    """Nothing is loaded (a test hook; no fault is involved), so every wait of the kernel runs out."""
    gen = generator(17)
    q, k, v = (randn(gen, 1, 200, 2, 64, dtype=BF16) for _ in range(3))
    want = package.attention(q, k, v)
    try:
        package.sdtw_debug_set_wait(0.02, skip_publish=True)
        assert torch.isnan(package.attention(q, k, v)).all()
        assert package.sdtw_encoder_status() == 7                  # SDTW_ERR_TIMEOUT
    finally:
        package.sdtw_debug_set_wait(0.0, skip_publish=False)
    assert package.sdtw_encoder_status() == 0
    assert torch.equal(package.attention(q, k, v), want)


def test_empty_inputs_give_empty_or_zero_results(package):
    q = torch.randn(2, 3, 4, 16, device="cuda", requires_grad=True)
    k = torch.randn(2, 0, 2, 16, device="cuda", requires_grad=True)
    out, lse = package.attention(q, k, k, return_lse=True)
    assert (out == 0).all() and torch.isneginf(lse).all()
    dq, dk = torch.autograd.grad(out, (q, k), torch.ones_like(out))
    assert (dq == 0).all() and dk.shape == k.shape
    assert package.attention(q[:, :0], q[:, :, :2], q[:, :, :2]).shape == (2, 0, 4, 16)
    assert package.layer_norm(torch.empty(0, 8, device="cuda")).shape == (0, 8)
    assert package.rotary(q[:, :0], table=package.rotary_table(4, 8)).shape == (2, 0, 4, 16)


def test_refusals(package):
    x, w = torch.ones(4, 8, device="cuda"), torch.ones(8, device="cuda")
    q, k = torch.ones(2, 3, 4, 16, device="cuda"), torch.ones(2, 5, 2, 16, device="cuda")
    table = package.rotary_table(8, 16)
    for bad in (lambda: package.layer_norm(x.cpu()), lambda: package.layer_norm(x, w[:4]), lambda: package.layer_norm(x, w.cpu()),
                lambda: package.layer_norm(x, eps=-1.0), lambda: package.layer_norm(x, eps=math.nan),
                lambda: package.rotary(q, table=table[:2]), lambda: package.rotary(q[..., :8], table=table),
                lambda: package.rotary(q, k, table=table), lambda: package.rotary(q, table=table.double()),
                lambda: package.rotary(q, table=table, positions=torch.zeros(2, 3, device="cuda")),
                lambda: package.rotary(q, table=table, positions=torch.zeros(3, 2, device="cuda", dtype=torch.int32)),
                lambda: package.rotary_table(8, 7), lambda: package.rotary_table(8, 8, scaling="other"),
                lambda: package.rotary_table(8, 8, scaling="yarn", factor=2.0), lambda: package.rotary_table(8, 8, factor=0.5),
                lambda: package.attention(q, k, k[:, :4]), lambda: package.attention(q, k[:1], k[:1]),
                lambda: package.attention(q[:, :, :3], k, k), lambda: package.attention(q, k, k, window=0),
                lambda: package.attention(q, k, k, scale=0.0), lambda: package.attention(q, k, k, scale=math.inf),
                lambda: package.attention(q, k, k, k_lengths=torch.ones(3, device="cuda", dtype=torch.int32)),
                lambda: package.attention(q, k, k, q_lengths=torch.ones(2, device="cuda")),
                lambda: package.attention(*(torch.ones(1, 2, 1, 129, device="cuda"),) * 3)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: package.layer_norm(x.double()), lambda: package.layer_norm(x, w.half()), lambda: package.attention(q, k.half(), k),
                lambda: package.attention(q.double(), k.double(), k.double()), lambda: package.rotary(q, k.half(), table=table),
                lambda: package.layer_norm(x, w, w.bfloat16())):
        with pytest.raises(TypeError):
            bad()


# The operators together: a few training steps through Soft-DTW, then a stream over the cache against the
# whole causal encoding. The two differ by their roundings alone: some 20 of the type's along a feature's
# way through two layers, each at most half a unit in the last place, against the features' norm.
@pytest.mark.parametrize("dtype,bound", [("fp32", 20 * 2.0 ** -23), ("bf16", 20 * 2.0 ** -8), ("fp16", 20 * 2.0 ** -11)])
def test_example_trains_and_streams(package, capsys, dtype, bound):
    spec = importlib.util.spec_from_file_location("encoder_alignment", os.path.join(ROOT, "examples", "encoder_alignment.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    first, last, off = example.main(["--steps", "3", "--dtype", dtype, "--length", "70"])
    assert math.isfinite(first) and math.isfinite(last)
    assert off < bound
