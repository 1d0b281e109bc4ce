"""Group norm, gated recurrence and gated linear units on the GPU against their definitions in 64 bits.

Tolerances are bounds, element by element, of what the arithmetic of the operators can be off by (first order in the
unit roundoffs), evaluated in 64 bits beside each result:

  u = 2^-24 (fp32), ut = 2^-24 / 2^-8 / 2^-11 (one rounding to fp32 / bf16 / fp16)
  a sum in fp32 whose terms pass at most d additions, truncating or rounding: 2 d u sum |terms|
  activations and their derivatives: (|z| + 8) 2^-22 relative and |z| 2^-22 absolute (erf near -1), and they move by at
  most 1.13 and 1 times an error of z
  a sigmoid: (|z| + 8) 2^-22 relative of exp(-z), which a = 1 / (1 + exp) feels by 1 - a of it, 1 - a by a of it

and a 16-bit result, or a gradient rounded to 16 bits before the product that consumes it, adds ut of itself. fp16 adds
its smallest step (2^-24) to every rounding.
"""
import math

import pytest

from helpers import ensure_built

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
U = 2.0 ** -24
UT = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}
TINY = {F32: 2.0 ** -126, BF16: 2.0 ** -126, F16: 2.0 ** -24}
ACTS = (None, "silu", "gelu", "relu")


@pytest.fixture(scope="module", autouse=True)
def package():
    ensure_built()
    import differentiable_series_alignment_gb300 as p
    p.load()
    return p


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(gen, *shape, dtype=F32, std=1.0, mean=0.0):
    return (torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float64) * std + mean).to(dtype)


def within(got, want, bound, what):
    got, bound = got.detach().double(), bound.expand_as(want)
    assert got.shape == want.shape, what
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - want).abs() / (bound + 1e-300)
    k = int(over.argmax())
    assert float(over.max()) <= 1.0, (f"{what}: off by {float(over.max()):.3g} of its bound at {k}: "
                                     f"{float(got.flatten()[k])!r}, not {float(want.flatten()[k])!r}")


def act(name, z):
    """Value, derivative, and what the arithmetic of either may be off by."""
    s = torch.sigmoid(z)
    if name == "silu":
        v, d = z * s, s * (1 + z * (1 - s))
    elif name == "gelu":
        c = 0.5 * torch.erfc(-z / math.sqrt(2))
        v, d = z * c, c + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    elif name == "relu":
        v, d = z.clamp(min=0), (z > 0).double()
        return v, d, torch.zeros_like(z)
    elif name == "sigmoid":
        v, d = s, s * (1 - s)
    else:
        return z, torch.ones_like(z), torch.zeros_like(z)
    return v, d, (z.abs() + 8) * 2.0 ** -22 * (1 + v.abs())


# --- group norm ---------------------------------------------------------------------------------

def norm_reference(x, G, w, b, dy, name, lengths, eps, wdtype):
    """(y, dx, dw, db) and their bounds."""
    dtype, (B, S, C) = x.dtype, x.shape
    cg = C // G
    ut, tiny = UT[dtype], TINY[dtype]
    split = lambda t: t.double().view(-1, S if t.dim() == 3 else 1, G, cg)  # noqa: E731
    valid = torch.ones(B, S, 1, 1, device="cuda", dtype=torch.float64)
    if lengths is not None:
        valid = (torch.arange(S, device="cuda") < lengths[:, None])[..., None, None].double()
    x, dy = split(torch.where(valid[..., 0] > 0, x, torch.zeros_like(x))), split(torch.where(valid[..., 0] > 0, dy, torch.zeros_like(dy)))
    w = torch.ones(1, 1, G, cg, device="cuda", dtype=torch.float64) if w is None else split(w)
    b = torch.zeros(1, 1, G, cg, device="cuda", dtype=torch.float64) if b is None else split(b)
    n = (valid.sum((1, 2, 3), keepdim=True) * cg).clamp(min=1)
    mean = lambda t: (t * valid).sum((1, 3), keepdim=True) / n  # noqa: E731
    depth = n / 8 + 64
    mu = mean(x)
    xc = (x - mu) * valid
    r = (mean(xc * xc) + eps) ** -0.5
    xh = xc * r
    z = xh * w + b
    d_mu = 2 * depth * U * mean(x.abs())
    d_r = (depth + 8) * U                                    # relative
    d_xh = r * (d_mu + U * (x.abs() + mu.abs())) + xh.abs() * (d_r + 4 * U)
    d_z = w.abs() * d_xh + 2 * U * (z.abs() + b.abs())
    v, slope, own = act(name, z)
    y = v * valid
    bounds = [(1.13 * d_z + own + ut * y.abs() + tiny) * valid]
    dz = dy * slope * valid
    g = dz * w
    d_slope = d_z + 2 * own + ((z.abs() <= d_z).double() if name == "relu" else 0)
    d_dz = dy.abs() * d_slope + 2 * U * dz.abs()
    d_g = d_dz * w.abs() + 2 * U * g.abs()
    m1, m2 = mean(g), mean(g * xh)
    dx = r * (g - m1 - xh * m2) * valid
    d_m1 = mean(d_g) + 2 * depth * U * mean(g.abs())
    d_m2 = mean(d_g * xh.abs() + g.abs() * d_xh) + 2 * depth * U * mean((g * xh).abs())
    bounds.append(((d_r + 4 * U + ut) * dx.abs() + r * (d_g + d_m1 + xh.abs() * d_m2 + m2.abs() * d_xh
                                                       + 4 * U * (g.abs() + m1.abs() + (xh * m2).abs())) + tiny) * valid)
    count = 2 * B * S * U
    dw, db = (dz * xh).sum((0, 1)), dz.sum((0, 1))
    bounds.append((d_dz * xh.abs() + dz.abs() * d_xh + count * (dz * xh).abs()).sum((0, 1)) + UT[wdtype] * dw.abs() + TINY[wdtype])
    bounds.append((d_dz + count * dz.abs()).sum((0, 1)) + UT[wdtype] * db.abs() + TINY[wdtype])
    return [t.reshape(B, S, C) for t in (y, dx)] + [t.flatten() for t in (dw, db)], \
        [t.expand(B, S, G, cg).reshape(B, S, C) for t in bounds[:2]] + [t.flatten() for t in bounds[2:]]


# batch, positions, groups, channels of a group
NORM_SHAPES = [(1, 1, 1, 1), (2, 3, 1, 5), (3, 1, 4, 8), (16, 1, 8, 64), (700, 1, 2, 12), (5, 7, 3, 7), (2, 64, 8, 8), (4, 100, 5, 16),
               (3, 33, 33, 1), (1, 257, 64, 1), (2, 129, 12, 2), (1, 1021, 4, 24), (2, 2000, 2, 40), (1, 17, 1, 1000), (9, 5, 300, 1),
               (1, 3, 2, 2050), (2, 30, 2, 2064), (70, 1, 3, 512), (40, 2, 5, 64), (3, 4, 8, 128)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shape", NORM_SHAPES, ids=str)
def test_group_norm(package, shape, dtype):
    B, S, G, cg = shape
    C, k = G * cg, NORM_SHAPES.index(shape)
    gen = generator(1000 + k)
    wdtype = dtype if k % 2 else F32
    name = ACTS[k % 4]
    x = randn(gen, B, S, C, dtype=dtype, std=1.5, mean=0.7).requires_grad_()
    w = None if k % 5 == 4 else randn(gen, C, dtype=wdtype, std=0.3, mean=1.0).requires_grad_()
    b = None if k % 7 == 6 else randn(gen, C, dtype=wdtype, std=0.3).requires_grad_()
    dy = randn(gen, B, S, C, dtype=dtype)
    y = package.group_norm(x, G, w, b, activation=name)
    leaves = [t for t in (x, w, b) if t is not None]
    grads = torch.autograd.grad(y, leaves, dy)
    want, bound = norm_reference(x.detach(), G, w, b, dy, name, None, 1e-5, wdtype)
    within(y, want[0], bound[0], "y")
    got = dict(zip([i for i, t in enumerate((x, w, b)) if t is not None], grads))
    for i, g in got.items():
        within(g, want[1 + i], bound[1 + i], ("dx", "dw", "db")[i])
    with torch.no_grad():
        assert torch.equal(package.group_norm(x, G, w, b, activation=name), y)          # the same without a backward pass
    again = torch.autograd.grad(package.group_norm(x, G, w, b, activation=name), leaves, dy)
    assert all(torch.equal(p, q) for p, q in zip(grads, again))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(5, 65, 4, 8), (6, 300, 3, 5), (4, 1, 2, 16), (4, 2100, 2, 32)], ids=str)
def test_group_norm_of_a_padded_batch(package, shape, dtype):
    B, S, G, cg = shape
    gen = generator(1100 + S)
    lengths = torch.tensor([S, 0, max(1, S // 3), S + 5, 1, -2][:B], device="cuda")
    x, dy = (randn(gen, B, S, G * cg, dtype=dtype, std=2.0, mean=-1.0) for _ in range(2))
    clean = x.clone(), dy.clone()
    for i, n in enumerate(lengths.clamp(0, S).tolist()):
        x[i, n:] = math.nan
        dy[i, n:] = math.inf
    x.requires_grad_()
    w, b = (randn(gen, G * cg, std=0.3, mean=m).requires_grad_() for m in (1.0, 0.0))
    y = package.group_norm(x, G, w, b, activation="silu", lengths=lengths)
    grads = torch.autograd.grad(y, (x, w, b), dy)
    want, bound = norm_reference(clean[0], G, w, b, clean[1], "silu", lengths, 1e-5, F32)
    for got, wanted, limit, what in zip((y, *grads), want, bound, ("y", "dx", "dw", "db")):
        within(got, wanted, limit, what)


def test_group_norm_dimensions_between_batch_and_channels(package):
    x = randn(generator(5), 2, 3, 5, 16).transpose(1, 2)          # not contiguous either
    got = package.group_norm(x, 4, activation="relu")
    assert got.shape == x.shape and torch.equal(got, package.group_norm(x.reshape(2, 15, 16), 4, activation="relu").view(2, 5, 3, 16))
    rows = randn(generator(6), 40, 16)
    assert torch.equal(package.group_norm(rows, 4), package.group_norm(rows[:, None], 4)[:, 0])


def test_group_norm_off_16_bytes_and_constant_groups(package):
    flat = randn(generator(7), 4 * 50 * 32 + 1, dtype=BF16, mean=1.0)
    x = flat[1:].view(4, 50, 32)
    want, bound = norm_reference(x, 4, None, None, torch.zeros_like(x), "gelu", None, 1e-5, F32)
    within(package.group_norm(x, 4, activation="gelu"), want[0], bound[0], "y")
    same = torch.full((3, 20, 8), 1000.0, device="cuda", requires_grad=True)
    y = package.group_norm(same, 2)
    assert torch.equal(y, torch.zeros_like(y))                     # the mean of equal values is that value
    (dx,) = torch.autograd.grad(y, same, torch.ones_like(y))
    assert torch.isfinite(dx).all()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shape", [(2, 4096, 4, 16), (1, 9000, 1, 256), (3, 2500, 6, 24), (2, 3000, 64, 1), (9000, 1, 4, 64), (3, 700, 3, 1003)], ids=str)
def test_large_group_norms_against_64_bits(package, shape, dtype):
    """Clusters, slabs that they cannot hold, many batch elements a CTA: in quadratic mean against 64 bits. 16-bit results
    are as near as their own rounding; fp32's sums of a group add a few roundings of its values, 16 at the most here."""
    B, S, G, cg = shape
    gen = generator(1200 + S)
    x, dy = randn(gen, B, S, G * cg, dtype=dtype, std=1.5, mean=0.5), randn(gen, B, S, G * cg, dtype=dtype)
    w, b = randn(gen, G * cg, std=0.3, mean=1.0), randn(gen, G * cg, std=0.3)
    leaves = [t.requires_grad_() for t in (x, w, b)]
    y = package.group_norm(x, G, w, b, activation="silu")
    got = (y, *torch.autograd.grad(y, leaves, dy))
    wide = [t.detach().double().requires_grad_() for t in leaves]
    t = wide[0].view(B, S, G, cg)
    var, mean = torch.var_mean(t, dim=(1, 3), unbiased=False, keepdim=True)
    z = ((t - mean) / torch.sqrt(var + 1e-5)).reshape(B, S, G * cg) * wide[1] + wide[2]
    exact = z / (1 + torch.exp(-z))
    for a, want, what in zip(got, (exact, *torch.autograd.grad(exact, wide, dy.double())), ("y", "dx", "dw", "db")):
        error = ((a.detach().double() - want) ** 2).mean().sqrt()
        own = ((want.to(a.dtype).double() - want) ** 2).mean().sqrt()
        assert error <= (16 if a.dtype == F32 else 1.05) * own, (what, float(error / own))
    again = package.group_norm(x, G, w, b, activation="silu")
    assert torch.equal(again, y) and all(torch.equal(p, q) for p, q in zip(torch.autograd.grad(again, leaves, dy), got[1:]))


# --- gated recurrence -----------------------------------------------------------------------------

def recurrence_reference(x, gate, state, dh, dlast, lengths, reverse, tied):
    """(h, last, dx, dgate, dstate) and their bounds, step by step."""
    dtype, (B, N, C) = x.dtype, x.shape
    ut, tiny = UT[dtype], TINY[dtype]
    n = torch.full((B,), N, device="cuda") if lengths is None else lengths.clamp(0, N)
    live = (torch.arange(N, device="cuda") < n[:, None])[..., None]
    zero = torch.zeros((), device="cuda", dtype=torch.float64)
    x, z, dh = (torch.where(live, t.double(), zero) for t in (x, gate, dh))
    e = (z.abs() + 8) * 2.0 ** -22
    a, o = torch.sigmoid(z), torch.sigmoid(-z)
    d_a, d_o = o * e + 8 * U, a * e + 8 * U                    # relative, with the roundings of products
    keep = torch.where(live, a, zero + 1)
    take = torch.where(live, o * x if tied else x, zero)
    d_take = take.abs() * (d_o if tied else 8 * U)
    order = list(range(N - 1, -1, -1) if reverse else range(N))
    h = torch.zeros(B, C, device="cuda", dtype=torch.float64) if state is None else state.double()
    m, d = h.abs(), torch.zeros_like(h)                        # majorant and error
    hs, before, d_before, d_hs = (torch.zeros_like(x) for _ in range(4))
    for t in order:
        before[:, t], d_before[:, t] = h, d
        d = keep[:, t] * d + torch.where(live[:, t], keep[:, t] * d_a[:, t] * m + d_take[:, t] + 8 * U * (keep[:, t] * m + take[:, t].abs()), zero)
        h, m = keep[:, t] * h + take[:, t], keep[:, t] * m + take[:, t].abs()
        hs[:, t], d_hs[:, t] = h, d
    last, d_last = h, d + U * h.abs()
    g = torch.zeros_like(h) if dlast is None else dlast.double()
    m, d = g.abs(), torch.zeros_like(g)
    es, d_es = torch.zeros_like(x), torch.zeros_like(x)
    for t in reversed(order):
        g, m = g + dh[:, t], m + dh[:, t].abs()
        d = d + torch.where(live[:, t], 8 * U * m, zero)
        es[:, t], d_es[:, t] = g, d
        d = keep[:, t] * d + torch.where(live[:, t], keep[:, t] * d_a[:, t] * m, zero)
        g, m = keep[:, t] * g, keep[:, t] * m
    dx = es * o if tied else es
    diff = before - x if tied else before
    dg = es * diff * a * o
    d_dx = d_es * (o if tied else 1) + dx.abs() * (d_o + 4 * U)
    d_dg = (d_es * diff.abs() + es.abs() * (d_before + 2 * U * (before.abs() + x.abs()))) * a * o + dg.abs() * (d_a + d_o + 8 * U)
    mask = live.double()
    return ([hs * mask, last, dx * mask, dg * mask, g],
            [(d_hs + ut * hs.abs() + tiny) * mask, d_last + TINY[F32], (d_dx + ut * dx.abs() + tiny) * mask,
             (d_dg + ut * dg.abs() + tiny) * mask, d + U * g.abs() + TINY[F32]])


RECURRENCE_SHAPES = [(1, 1, 1), (3, 1, 40), (2, 2, 7), (1, 8, 64), (2, 9, 33), (1, 17, 128), (3, 63, 24), (2, 64, 65), (2, 65, 64), (1, 127, 8),
                     (5, 128, 72), (2, 129, 16), (1, 500, 130), (2, 1021, 40), (1, 2600, 264), (40, 70, 32), (3, 257, 250),
                     (2, 4500, 72), (40, 1100, 64), (1, 4200, 8), (10, 1300, 200)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shape", RECURRENCE_SHAPES, ids=str)
def test_gated_recurrence(package, shape, dtype):
    B, N, C = shape
    k = RECURRENCE_SHAPES.index(shape)
    gen = generator(2000 + k)
    reverse, tied, ragged, given = k % 2 == 1, k % 3 != 2, k % 4 >= 2, k % 5 != 0
    x, gate = randn(gen, B, N, C, dtype=dtype), randn(gen, B, N, C, dtype=dtype, mean=2.0, std=2.0)
    state = randn(gen, B, C).requires_grad_() if given else None
    dh, dlast = randn(gen, B, N, C, dtype=dtype), randn(gen, B, C)
    lengths = torch.tensor([(N - 3 * b) // (1 + b % 2) if b != 1 else 0 for b in range(B)], device="cuda") if ragged else None
    want, bound = recurrence_reference(x, gate, state, dh, dlast, lengths, reverse, tied)
    if ragged:
        beyond = torch.arange(N, device="cuda") >= lengths[:, None]
        x[beyond], gate[beyond], dh[beyond] = math.nan, math.inf, math.nan
    x.requires_grad_()
    gate.requires_grad_()
    leaves = (x, gate, state) if given else (x, gate)
    run = lambda: package.gated_recurrence(x, gate, state, lengths=lengths, reverse=reverse, tied=tied, return_state=True)  # noqa: E731
    h, last = run()
    grads = torch.autograd.grad((h, last), leaves, (dh, dlast))
    for got, wanted, limit, what in zip((h, last, *grads), want, bound, ("h", "last", "dx", "dgate", "dstate")):
        within(got, wanted, limit, what)
    with torch.no_grad():
        assert all(torch.equal(p, q) for p, q in zip(run(), (h, last)))
    assert all(torch.equal(p, q) for p, q in zip(torch.autograd.grad(run(), leaves, (dh, dlast)), grads))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_recurrence_in_pieces(package, dtype):
    """A series in pieces, and sample by sample, goes on from the state of what came before."""
    gen = generator(11)
    B, N, C = 3, 150, 48
    x, gate = randn(gen, B, N, C, dtype=dtype), randn(gen, B, N, C, dtype=dtype, mean=1.0)
    want, bound = recurrence_reference(x, gate, None, torch.zeros_like(x), None, None, False, True)
    for cuts in ([0, 1, 9, 70, 71, 150], range(0, 151)):
        cuts, state, out = list(cuts), None, []
        for lo, hi in zip(cuts, cuts[1:]):
            h, state = package.gated_recurrence(x[:, lo:hi], gate[:, lo:hi], state, return_state=True)
            out.append(h)
        within(torch.cat(out, 1), want[0], bound[0], "h")
        within(state, want[1], bound[1], "state")


def test_recurrence_of_slices_and_broadcasts(package):
    gen = generator(12)
    both = randn(gen, 2, 90, 3 * 40, dtype=BF16)
    x, gate, _ = both.split(40, dim=2)
    got = package.gated_recurrence(x, gate)
    assert torch.equal(got, package.gated_recurrence(x.contiguous(), gate.contiguous()))
    odd = randn(gen, 2, 90, 81, dtype=BF16)[..., 1:].split(40, dim=2)            # off 16 bytes
    want, bound = recurrence_reference(odd[0], odd[1], None, torch.zeros_like(odd[0]), None, None, False, True)
    within(package.gated_recurrence(*odd), want[0], bound[0], "h")
    one = randn(gen, 1, 1, 40, dtype=BF16).requires_grad_()
    wide = one.expand(2, 90, 40)
    assert torch.equal(package.gated_recurrence(x, wide), package.gated_recurrence(x, wide.contiguous()))
    (g,) = torch.autograd.grad(package.gated_recurrence(x, wide), one, torch.ones_like(x))
    leaf = wide.detach().clone().requires_grad_()
    (full,) = torch.autograd.grad(package.gated_recurrence(x, leaf), leaf, torch.ones_like(x))
    assert torch.equal(g, full.sum((0, 1), keepdim=True))
    turned = randn(gen, 2, 40, 90).transpose(1, 2)                                # channels not contiguous
    assert torch.equal(package.gated_recurrence(turned, turned), package.gated_recurrence(turned.contiguous(), turned.contiguous()))


def test_recurrence_gates_that_saturate(package):
    x = randn(generator(13), 1, 200, 16).requires_grad_()
    for z, want in ((200.0, torch.zeros_like(x)), (math.inf, torch.zeros_like(x)), (-200.0, x), (-math.inf, x)):
        gate = torch.full_like(x, z).detach().requires_grad_()
        h = package.gated_recurrence(x, gate)
        assert torch.equal(h, want), z
        dx, dgate = torch.autograd.grad(h, (x, gate), torch.ones_like(h))
        assert torch.equal(dx, torch.full_like(dx, 0.0 if z > 0 else 1.0)) and torch.equal(dgate, torch.zeros_like(dgate)), z


def test_recurrence_gradients_of_one_output(package):
    gen = generator(14)
    x, gate = randn(gen, 2, 70, 16).requires_grad_(), randn(gen, 2, 70, 16).requires_grad_()
    state = randn(gen, 2, 16).requires_grad_()
    dh, dl = randn(gen, 2, 70, 16), randn(gen, 2, 16)
    run = lambda: package.gated_recurrence(x, gate, state, return_state=True)  # noqa: E731
    for which in (0, 1):
        got = torch.autograd.grad(run()[which], (x, gate, state), (dh, dl)[which])
        want, bound = recurrence_reference(x.detach(), gate, state, dh if which == 0 else torch.zeros_like(dh), dl if which == 1 else None, None, False, True)
        for a, b, c in zip(got, want[2:], bound[2:]):
            within(a, b, c, f"gradients of output {which}")
    (only,) = torch.autograd.grad(run()[0], state, dh)
    assert torch.equal(only, torch.autograd.grad(run()[0], (x, gate, state), dh)[2])


# --- gated linear units ---------------------------------------------------------------------------

def gated_reference(x, wg, wu, bg, bu, dh, name):
    """(h, dx, dwg, dwu, dbg, dbu) and their bounds."""
    dtype = x.dtype
    ut, tiny = UT[dtype], TINY[dtype]
    R, K = x.shape
    F = wg.shape[0]
    x, wg, wu, dh = (t.double() for t in (x, wg, wu, dh))
    bg, bu = (torch.zeros(F, device="cuda", dtype=torch.float64) if t is None else t.double() for t in (bg, bu))
    g, u = x @ wg.T + bg, x @ wu.T + bu
    d_g, d_u = (2 * (K + 4) * U * (x.abs() @ w.abs().T + b.abs()) for w, b in ((wg, bg), (wu, bu)))
    v, slope, own = act(name, g)
    h = v * u
    d_v = 1.13 * d_g + own
    d_slope = d_g + 2 * own + ((g.abs() <= d_g).double() if name == "relu" else 0)
    bounds = [d_v * u.abs() + v.abs() * d_u + (2 * U + ut) * h.abs() + tiny]
    dg, du = dh * u * slope, dh * v
    once = 0.0 if dtype == F32 else ut                          # rounded before the products that consume them
    step = 0.0 if dtype == F32 else tiny
    d_dg = dh.abs() * (u.abs() * d_slope + slope.abs() * d_u) + (4 * U + once) * dg.abs() + step
    d_du = dh.abs() * d_v + (4 * U + once) * du.abs() + step
    dx = dg @ wg + du @ wu
    bounds.append(d_dg @ wg.abs() + d_du @ wu.abs() + 2 * (2 * F + 4) * U * (dg.abs() @ wg.abs() + du.abs() @ wu.abs()) + ut * dx.abs() + tiny)
    want = [h, dx]
    for d, err in ((dg, d_dg), (du, d_du)):
        want.append(d.T @ x)
        bounds.append(err.T @ x.abs() + 2 * (R + 4) * U * (d.abs().T @ x.abs()) + ut * want[-1].abs() + tiny)
    for d, err in ((dg, d_dg), (du, d_du)):
        want.append(d.sum(0))
        bounds.append(err.sum(0) + 2 * (R + 4) * U * d.abs().sum(0) + ut * want[-1].abs() + tiny)
    return want, bounds


# rows, K, F
GATED_SHAPES = [(1, 1, 1), (1, 64, 64), (2, 5, 3), (3, 128, 200), (8, 256, 96), (9, 72, 130), (16, 1000, 40), (17, 33, 65), (33, 64, 128),
                (64, 130, 48), (100, 96, 264), (129, 64, 72), (128, 200, 128), (250, 17, 129), (257, 264, 136), (300, 8, 8), (513, 72, 300),
                (1000, 64, 256), (8, 8, 8), (24, 264, 72), (32, 1024, 48), (31, 36, 50)]
GATED_ACTS = ("silu", "gelu", "relu", "sigmoid")


def check_gated(package, x, wg, wu, bg, bu, dh, name):
    leaves = [t.detach().requires_grad_() if t is not None else None for t in (x, wg, wu, bg, bu)]
    have = [t for t in leaves if t is not None]
    h = package.gated_linear(*leaves, activation=name)
    grads = torch.autograd.grad(h, have, dh)
    want, bound = gated_reference(x, wg, wu, bg, bu, dh, name)
    within(h, want[0], bound[0], "h")
    got = iter(grads)
    for t, a, b, what in zip(leaves, want[1:], bound[1:], ("dx", "dgate_weight", "dup_weight", "dgate_bias", "dup_bias")):
        if t is not None:
            within(next(got), a, b, what)
    with torch.no_grad():
        assert torch.equal(package.gated_linear(*leaves, activation=name), h)
    again = torch.autograd.grad(package.gated_linear(*leaves, activation=name), have, dh)
    assert all(torch.equal(p, q) for p, q in zip(grads, again))
    return h, grads


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shape", GATED_SHAPES, ids=str)
def test_gated_linear(package, shape, dtype):
    R, K, F = shape
    k = GATED_SHAPES.index(shape)
    gen = generator(3000 + k)
    x, wg, wu = randn(gen, R, K, dtype=dtype), randn(gen, F, K, dtype=dtype, std=K ** -0.5), randn(gen, F, K, dtype=dtype, std=K ** -0.5)
    bg = randn(gen, F, dtype=dtype, std=0.5) if k % 3 else None
    bu = randn(gen, F, dtype=dtype, std=0.5) if k % 4 else None
    check_gated(package, x, wg, wu, bg, bu, randn(gen, R, F, dtype=dtype), GATED_ACTS[k % 4])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gated_linear_of_slices(package, dtype):
    """One matrix of both weights, rows with a stride, addresses off 16 bytes."""
    gen = generator(21)
    for off in (0, 1):
        both = randn(gen, 200, 64 + off, dtype=dtype, std=0.1)[:, off:]
        x = randn(gen, 70, 100 + off, dtype=dtype)[:, off:off + 64]
        check_gated(package, x, both[:100], both[100:], None, None, randn(gen, 70, 100, dtype=dtype), "silu")
    turned = randn(gen, 64, 100, dtype=dtype, std=0.1).T                          # features not contiguous
    check_gated(package, x, turned, turned.contiguous(), None, None, randn(gen, 70, 100, dtype=dtype), "gelu")
    check_gated(package, randn(gen, 1, 64, dtype=dtype).expand(70, 64), turned, turned, None, None, randn(gen, 70, 100, dtype=dtype), "relu")


def test_gated_linear_dimensions_and_some_gradients(package):
    gen = generator(22)
    x = randn(gen, 2, 3, 5, 24, dtype=BF16)
    wg, wu = (randn(gen, 40, 24, dtype=BF16, std=0.2) for _ in range(2))
    h = package.gated_linear(x, wg, wu)
    assert h.shape == (2, 3, 5, 40) and torch.equal(h.view(30, 40), package.gated_linear(x.view(30, 24), wg, wu))
    assert package.gated_linear(x[0, 0, 0], wg, wu).shape == (40,)
    dh = randn(gen, 30, 40, dtype=BF16)
    full = check_gated(package, x.view(30, 24), wg, wu, None, None, dh, "silu")[1]
    for i in range(3):
        leaves = [t.detach().requires_grad_(i == k) for k, t in enumerate((x.view(30, 24), wg, wu))]
        assert torch.equal(torch.autograd.grad(package.gated_linear(*leaves), leaves[i], dh)[0], full[i])


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_results_are_as_near_as_their_rounding(package, dtype):
    """How far 16-bit results are from 64 bits, in quadratic mean, against their own rounding. Gradients that are rounded
    before the products that consume them add as much as the result's rounding in squares: a factor of sqrt 2, and 1.6
    at the most here."""
    gen = generator(23)
    R, K, F = 600, 256, 384
    x, wg, wu = randn(gen, R, K, dtype=dtype), *(randn(gen, F, K, dtype=dtype, std=K ** -0.5) for _ in range(2))
    for scale in (1.0, 2.0 ** -12):                              # small gradients, which fp16 must not lose
        dh = randn(gen, R, F, dtype=dtype, std=scale)
        want, _ = gated_reference(x, wg, wu, None, None, dh, "silu")
        h, grads = check_gated(package, x, wg, wu, None, None, dh, "silu")
        for got, exact, what in zip((h, *grads), want, ("h", "dx", "dwg", "dwu")):
            error = ((got.double() - exact) ** 2).mean().sqrt()
            own = ((exact.to(dtype).double() - exact) ** 2).mean().sqrt()
            assert error <= (1.02 if what == "h" else 1.6) * own, (what, scale, float(error / own))


# --- together, and around -------------------------------------------------------------------------

class Block:
    """norm, recurrence and gated units as an encoder of long series has them."""

    def __init__(self, gen, width, hidden, dtype):
        std = width ** -0.5
        self.mix, self.out = randn(gen, 2 * width, width, dtype=dtype, std=std), randn(gen, width, width, dtype=dtype, std=std)
        self.wg, self.wu = (randn(gen, hidden, width, dtype=dtype, std=std) for _ in range(2))
        self.down = randn(gen, width, hidden, dtype=dtype, std=hidden ** -0.5)
        self.scale, self.shift = randn(gen, width, std=0.1, mean=1.0), randn(gen, width, std=0.1)
        for t in self.weights():
            t.requires_grad_()

    def weights(self):
        return [self.mix, self.out, self.wg, self.wu, self.down, self.scale, self.shift]

    def __call__(self, package, x, state=None, lengths=None):
        rows = lambda t: package.group_norm(t.reshape(-1, t.shape[-1]), 4, self.scale, self.shift).view_as(t)  # noqa: E731
        v, gate = torch.nn.functional.linear(rows(x), self.mix).chunk(2, dim=-1)
        h, state = package.gated_recurrence(v, gate, state, lengths=lengths, return_state=True)
        x = x + torch.nn.functional.linear(h, self.out)
        return x + torch.nn.functional.linear(package.gated_linear(rows(x), self.wg, self.wu), self.down), state


def test_block_streams_as_it_encodes(package):
    """A whole series, and the same sample by sample from the state: the same features up to fp32's rounding. Each of the
    operators is within 1e-4 of its definition at these sizes (sums of at most 128 terms of order one, 2 * 128 u each, and a
    recurrence whose gates forget), and the block multiplies an input's error by less than 100."""
    gen = generator(31)
    block = Block(gen, 64, 128, F32)
    x = randn(gen, 3, 90, 64)
    with torch.no_grad():
        whole, last = block(package, x)
        state, out = None, []
        for t in range(x.shape[1]):
            y, state = block(package, x[:, t:t + 1], state)
            out.append(y)
    assert (torch.cat(out, 1) - whole).abs().max() < 1e-2 * whole.abs().max()
    assert (state - last).abs().max() < 1e-2 * last.abs().max()


def test_block_gradients_against_differences(package):
    """The derivative along a direction against a central difference with a step of 2^-8: the third derivatives of a loss of
    order one make (2^-8)^2 of it, some 1e-4 of the derivative's scale; fp32's rounding of the loss 1e-6 / 2^-7 = 1e-4."""
    gen = generator(32)
    block = Block(gen, 32, 64, F32)
    x, up = randn(gen, 2, 70, 32), randn(gen, 2, 70, 32)
    lengths = torch.tensor([70, 41], device="cuda")
    leaves = [x.requires_grad_()] + block.weights()

    def loss():
        y, last = block(package, x, lengths=lengths)
        return (y[0] * up[0]).double().mean() + (y[1, :41] * up[1, :41]).double().mean() + last.double().mean()

    grads = torch.autograd.grad(loss(), leaves)
    for leaf, grad in zip(leaves, grads):
        v = randn(gen, *leaf.shape)
        slope = float((grad.double() * v).sum())
        with torch.no_grad():
            leaf += 2.0 ** -8 * v
            high = float(loss())
            leaf -= 2.0 ** -7 * v
            low = float(loss())
            leaf += 2.0 ** -8 * v
        scale = float(grad.double().norm() * v.double().norm())
        assert abs((high - low) / 2.0 ** -7 - slope) <= 2e-2 * scale, leaf.shape


def calls(package, gen, dtype=BF16):
    """One call of each operator, forward and backward, as a function of nothing."""
    leaves = dict(x=randn(gen, 4, 200, 64, dtype=dtype), gate=randn(gen, 4, 200, 64, dtype=dtype, mean=1.0),
                  wg=randn(gen, 96, 64, dtype=dtype, std=0.1), wu=randn(gen, 96, 64, dtype=dtype, std=0.1),
                  w=randn(gen, 64), b=randn(gen, 64), bg=randn(gen, 96, dtype=dtype))
    for t in leaves.values():
        t.requires_grad_()
    x, gate, wg, wu, w, b, bg = leaves.values()
    dy, dh = randn(gen, 4, 200, 64, dtype=dtype), randn(gen, 4, 200, 96, dtype=dtype)
    lengths = torch.tensor([200, 0, 77, 130], device="cuda", dtype=torch.int32)

    def norm():
        y = package.group_norm(x, 8, w, b, activation="silu", lengths=lengths)
        return [y, *torch.autograd.grad(y, (x, w, b), dy)]

    def recurrence():
        y = package.gated_recurrence(x, gate, lengths=lengths, reverse=True)
        return [y, *torch.autograd.grad(y, (x, gate), dy)]

    def gated():
        y = package.gated_linear(x, wg, wu, bg)
        return [y, *torch.autograd.grad(y, (x, wg, wu, bg), dh)]

    return [norm, recurrence, gated]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("which", [0, 1, 2], ids=["norm", "recurrence", "gated"])
def test_captured_calls_replay(package, which, dtype):
    """Two graphs of the same call share no workspace, and replay in any order and at once."""
    call = calls(package, generator(41), dtype)[which]
    want = [t.detach().clone() for t in call()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    outs = []
    for g in graphs:
        with torch.cuda.graph(g):
            outs.append([t.detach() for t in call()])
    for out in outs:
        for t in out:
            t.fill_(math.nan)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for out in outs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_other_streams_at_once(package):
    jobs = calls(package, generator(42))
    want = [[t.detach().clone() for t in f()] for f in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(6)]
    got = []
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            got.append([t.detach() for t in jobs[i % 3]()])
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 3]))


def test_empty_calls(package):
    x = torch.empty(0, 5, 16, device="cuda", requires_grad=True)
    w = torch.ones(16, device="cuda", requires_grad=True)
    y = package.group_norm(x, 4, w)
    assert y.shape == x.shape and torch.equal(torch.autograd.grad(y, w, torch.empty_like(x))[0], torch.zeros_like(w))
    x = torch.empty(3, 0, 16, device="cuda", requires_grad=True)
    state = randn(generator(1), 3, 16).requires_grad_()
    h, last = package.gated_recurrence(x, x, state, return_state=True)
    assert h.shape == x.shape and torch.equal(last, state)
    assert torch.equal(torch.autograd.grad(last, state, 2 * torch.ones_like(last))[0], torch.full_like(state, 2.0))
    assert package.group_norm(x, 4).shape == x.shape
    wide = randn(generator(2), 24, 16).requires_grad_()
    h = package.gated_linear(x, wide, wide)
    assert h.shape == (3, 0, 24) and torch.equal(torch.autograd.grad(h, wide, torch.empty_like(h))[0], torch.zeros_like(wide))


def test_refusals(package):
    x, w = torch.ones(2, 3, 8, device="cuda"), torch.ones(8, device="cuda")
    m = torch.ones(4, 8, device="cuda")
    for call, error in [
        (lambda: package.group_norm(x.cpu(), 2), ValueError), (lambda: package.group_norm(x.double(), 2), TypeError),
        (lambda: package.group_norm(x, 3), ValueError), (lambda: package.group_norm(x, 0), ValueError),
        (lambda: package.group_norm(x, 2, w[:4]), ValueError), (lambda: package.group_norm(x, 2, w.bfloat16()), TypeError),
        (lambda: package.group_norm(x, 2, w, activation="tanh"), ValueError), (lambda: package.group_norm(x, 2, eps=-1.0), ValueError),
        (lambda: package.group_norm(x, 2, activation="sigmoid"), ValueError), (lambda: package.group_norm(x[0, 0], 2), ValueError),
        (lambda: package.group_norm(x, 2, lengths=torch.ones(3, dtype=torch.int32, device="cuda")), ValueError),
        (lambda: package.group_norm(x[0], 2, lengths=torch.ones(3, dtype=torch.int32, device="cuda")), ValueError),
        (lambda: package.group_norm(x, 2, lengths=torch.ones(2, device="cuda")), ValueError),
        (lambda: package.gated_recurrence(x, x[:, :2]), ValueError), (lambda: package.gated_recurrence(x, x.half()), TypeError),
        (lambda: package.gated_recurrence(x[0], x[0]), ValueError), (lambda: package.gated_recurrence(x, x, w), ValueError),
        (lambda: package.gated_recurrence(x, x, torch.ones(2, 8, device="cuda").half()), TypeError),
        (lambda: package.gated_recurrence(x, x, lengths=torch.ones(2, device="cuda")), ValueError),
        (lambda: package.gated_recurrence(x, x.cpu()), ValueError),
        (lambda: package.gated_linear(x, m, m[:3]), ValueError), (lambda: package.gated_linear(x, m[:, :4], m[:, :4]), ValueError),
        (lambda: package.gated_linear(x, m, m.half()), TypeError), (lambda: package.gated_linear(x, m, m, w), ValueError),
        (lambda: package.gated_linear(x, m, m, w[:4].half()), TypeError), (lambda: package.gated_linear(x, m, m, activation=None), ValueError),
        (lambda: package.gated_linear(x, m, m, activation="tanh"), ValueError), (lambda: package.gated_linear(x.cpu(), m, m), ValueError),
        (lambda: package.gated_linear(x, m.cpu(), m), ValueError), (lambda: package.gated_linear(x.int(), m, m), TypeError),
    ]:
        with pytest.raises(error):
            call()
    for call in (lambda t: package.group_norm(t, 2), lambda t: package.gated_recurrence(t, t), lambda t: package.gated_linear(t, m, m)):
        leaf = x.clone().requires_grad_()
        (g,) = torch.autograd.grad(call(leaf).sum(), leaf, create_graph=False)
        assert g.shape == leaf.shape
        with pytest.raises(RuntimeError, match="once"):
            torch.autograd.grad(call(leaf).sum(), leaf, create_graph=True)
        import torch.autograd.forward_ad as fwd
        with fwd.dual_level(), pytest.raises(NotImplementedError):
            call(fwd.make_dual(x, x))


def test_waits_that_run_out(package):
    """A kernel that gives up a wait leaves NaN, reports it, and the next call is right again."""
    gen = generator(51)
    x, gate = randn(gen, 1, 2000, 64, dtype=BF16), randn(gen, 1, 2000, 64, dtype=BF16, mean=1.0)
    rows, w = randn(gen, 300, 64, dtype=BF16), randn(gen, 128, 64, dtype=BF16)
    dh = randn(gen, 300, 128, dtype=BF16)
    jobs = [lambda: package.gated_recurrence(x, gate), lambda: package.gated_linear(rows, w, w)]

    def backward():
        leaf = rows.detach().requires_grad_()
        return torch.autograd.grad(package.gated_linear(leaf, w, w), leaf, dh)[0]

    want = [f() for f in jobs] + [backward()]
    assert package.sdtw_encoder_status() == 0
    try:
        for f, right in zip(jobs, want):
            package.sdtw_debug_set_wait(0.05, 1)
            got = f()
            assert package.sdtw_encoder_status() == 7 and torch.isnan(got).any()
            assert package.sdtw_encoder_status() == 0
            assert torch.equal(f(), right)
        leaf = rows.detach().requires_grad_()
        h = package.gated_linear(leaf, w, w)
        package.sdtw_debug_set_wait(0.05, 1)
        (got,) = torch.autograd.grad(h, leaf, dh)
        assert package.sdtw_encoder_status() == 7 and torch.isnan(got).all()
    finally:
        package.sdtw_debug_set_wait(0.0, 0)
    assert torch.equal(backward(), want[2])


def test_first_call_of_a_thread(package):
    """A thread that has made no other CUDA call yet has no context of its own; tensor maps need one."""
    import subprocess
    import sys
    code = """if 1:
        import threading, torch
        from differentiable_series_alignment_gb300 import attention, gated_linear
        q = torch.randn(1, 200, 2, 64, device="cuda", dtype=torch.bfloat16)
        x, w = q.reshape(-1, 64), torch.randn(256, 64, device="cuda", dtype=torch.bfloat16)
        want = attention(q, q, q), gated_linear(x, w, w)
        del want
        got = []
        for f in (lambda: attention(q, q, q), lambda: gated_linear(x, w, w)):
            t = threading.Thread(target=lambda: got.append(f()))
            t.start()
            t.join()
        assert torch.equal(got[0], attention(q, q, q)) and torch.equal(got[1], gated_linear(x, w, w))
        leaf = x.detach().requires_grad_()
        torch.autograd.grad(gated_linear(leaf, w, w), leaf, torch.ones(400, 256, device="cuda", dtype=torch.bfloat16))
        torch.cuda.synchronize()
    """
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_large_products_against_64_bits(package, dtype):
    """Tiles of two CTAs, shares of a sum, ragged last tiles: in quadratic mean against 64 bits, where a tile that is
    missing, doubled or misplaced shows. fp32's sums of up to 8192 terms have errors of 64 roundings of a term at the least."""
    gen = generator(24)
    R, K, F = (2100, 300, 3001) if dtype == F32 else (5000, 520, 4100)
    x, wg, wu = randn(gen, R, K, dtype=dtype), *(randn(gen, F, K, dtype=dtype, std=K ** -0.5) for _ in range(2))
    bg, dh = randn(gen, F, dtype=dtype), randn(gen, R, F, dtype=dtype, std=1e-3)
    leaves = [t.requires_grad_() for t in (x, wg, wu, bg)]
    h = package.gated_linear(x, wg, wu, bg, activation="gelu")
    grads = torch.autograd.grad(h, leaves, dh)
    wide = [t.detach().double().requires_grad_() for t in leaves]
    g = wide[0] @ wide[1].T + wide[3]
    exact = g * 0.5 * torch.erfc(-g / math.sqrt(2)) * (wide[0] @ wide[2].T)
    want = torch.autograd.grad(exact, wide, dh.double())
    for got, right, what in zip((h, *grads), (exact, *want), ("h", "dx", "dwg", "dwu", "dbg")):
        error = ((got.detach().double() - right) ** 2).mean().sqrt()
        own = ((right.to(dtype).double() - right) ** 2).mean().sqrt()
        assert error <= (64 if dtype == F32 else 1.02 if what in ("h", "dbg") else 1.6) * own, (what, float(error / own))
    assert all(torch.equal(a, b) for a, b in zip(torch.autograd.grad(package.gated_linear(x, wg, wu, bg, activation="gelu"), leaves, dh), grads))


def test_problems_keep_their_tensors():
    """A problem holds pointers alone as far as the library is concerned; the tensors have to live as long as it does."""
    import gc
    import weakref

    from differentiable_series_alignment_gb300 import _lib as lib

    def made():
        x, gate, state = (torch.zeros(s, device="cuda") for s in ((2, 3, 4), (2, 3, 4), (2, 4)))
        rows, wg, wu, bias = (torch.zeros(s, device="cuda") for s in ((5, 4), (6, 4), (6, 4), (6,)))
        return ((lib.recurrence_problem(x, gate, state), [weakref.ref(t) for t in (x, gate, state)]),
                (lib.gated_problem(rows, wg, wu, bias), [weakref.ref(t) for t in (rows, wg, wu, bias)]))

    problems = made()
    gc.collect()
    for problem, tensors in problems:
        assert all(t() is not None for t in tensors)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_overlapping_rows(package, dtype):
    """Windows of one series as rows: a stride shorter than a row."""
    gen = generator(51)
    series = randn(gen, 8 * 300 + 64, dtype=dtype)
    windows = series.unfold(0, 64, 8)                                             # (301, 64), a row every 8
    wg, wu = (randn(gen, 96, 64, dtype=dtype, std=0.1) for _ in range(2))
    check_gated(package, windows, wg, wu, None, None, randn(gen, 301, 96, dtype=dtype), "silu")
    few = series[:8 * 7 + 64].unfold(0, 64, 8)
    assert torch.equal(package.gated_linear(few, wg, wu), package.gated_linear(few.contiguous(), wg, wu))
    x, gate = windows[None], series.flip(0).unfold(0, 64, 8)[None]
    dh = randn(gen, 1, 301, 64, dtype=dtype)
    outs = []
    for a, b in ((x, gate), (x.contiguous(), gate.contiguous())):
        a, b = a.detach().requires_grad_(), b.detach().requires_grad_()
        h = package.gated_recurrence(a, b)
        outs.append((h, *torch.autograd.grad(h, (a, b), dh)))
    assert all(torch.equal(p, q) for p, q in zip(*outs))


def test_the_same_tensor_twice(package):
    gen = generator(52)
    x, w = randn(gen, 70, 40), randn(gen, 48, 40, std=0.2)
    dh = randn(gen, 70, 48)
    want, bound = gated_reference(x, w, w, None, None, dh, "silu")
    w.requires_grad_()
    h = package.gated_linear(x, w, w)
    within(h, want[0], bound[0], "h")
    within(torch.autograd.grad(h, w, dh)[0], want[2] + want[3], bound[2] + bound[3] + U * (want[2] + want[3]).abs(), "dw")
    x = randn(gen, 2, 90, 24)
    dh = randn(gen, 2, 90, 24)
    want, bound = recurrence_reference(x, x, None, dh, None, None, False, True)
    x.requires_grad_()
    got = torch.autograd.grad(package.gated_recurrence(x, x), x, dh)[0]
    within(got, want[2] + want[3], bound[2] + bound[3] + U * (want[2] + want[3]).abs(), "dx + dgate")


def test_second_derivatives_are_refused(package):
    x = randn(generator(53), 3, 5, 16).requires_grad_()
    w = randn(generator(53), 8, 16).requires_grad_()
    for y in (package.group_norm(x, 4), package.gated_recurrence(x, x), package.gated_linear(x, w, w)):
        with pytest.raises(RuntimeError, match="differentiable once"):
            torch.autograd.grad(y.sum(), x, create_graph=True)


# one accumulator of 256, of 128 and of 64 columns is what the least time asks for
@pytest.mark.parametrize("shape", [(2048, 64, 4096), (1024, 64, 1024), (128, 72, 256)], ids=str)
def test_widths_of_accumulators(package, shape):
    R, K, F = shape
    gen = generator(54)
    x, wg, wu = randn(gen, R, K, dtype=BF16), randn(gen, F, K, dtype=BF16, std=K ** -0.5), randn(gen, F, K, dtype=BF16, std=K ** -0.5)
    check_gated(package, x, wg, wu, randn(gen, F, dtype=BF16, std=0.5), None, randn(gen, R, F, dtype=BF16), "gelu")


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("shape", [(3, 2200, 264), (6, 1500, 200), (1, 2049, 64), (1, 1025, 128)], ids=str)
def test_recurrences_of_some_clusters(package, shape, dtype):
    """Between the few clusters that take sixteen CTAs and the many: eight CTAs, of sixteen warps or of eight."""
    gen = generator(55)
    B, N, C = shape
    x, gate = (randn(gen, B, N, C, dtype=dtype, mean=m, std=s).requires_grad_() for m, s in ((0.0, 1.0), (2.0, 2.0)))
    state, dh, dlast = randn(gen, B, C).requires_grad_(), randn(gen, B, N, C, dtype=dtype), randn(gen, B, C)
    want, bound = recurrence_reference(x, gate, state, dh, dlast, None, False, True)
    h, last = package.gated_recurrence(x, gate, state, return_state=True)
    grads = torch.autograd.grad((h, last), (x, gate, state), (dh, dlast))
    for got, wanted, limit, what in zip((h, last, *grads), want, bound, ("h", "last", "dx", "dgate", "dstate")):
        within(got, wanted, limit, what)


# --- what the shared memory of a cluster's exchange takes

@pytest.mark.parametrize("shape,dtype", [((1, 4096, 2008, 1), BF16), ((2, 2100, 1004, 1), F32), ((1, 300, 1016, 1), F16), ((3, 700, 772, 2), BF16)],
                         ids=str)
def test_group_norm_of_many_groups_in_a_slab(package, shape, dtype):
    """Channels of whose divisors none makes a narrow slab: a slab is all of them, with up to 2008 groups, and what a cluster's
    CTAs exchange of these has to fit their shared memory."""
    B, S, G, cg = shape
    gen = generator(1300 + S)
    x = randn(gen, B, S, G * cg, dtype=dtype, std=1.5, mean=0.5).requires_grad_()
    w, b = (randn(gen, G * cg, std=0.3, mean=m).requires_grad_() for m in (1.0, 0.0))
    dy = randn(gen, B, S, G * cg, dtype=dtype)
    y = package.group_norm(x, G, w, b, activation="silu")
    grads = torch.autograd.grad(y, (x, w, b), dy)
    want, bound = norm_reference(x.detach(), G, w, b, dy, "silu", None, 1e-5, F32)
    for got, wanted, limit, what in zip((y, *grads), want, bound, ("y", "dx", "dw", "db")):
        within(got, wanted, limit, what)


# --- channels by themselves

@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shape", [(3, 1, 16), (2, 7, 24), (3, 150, 64), (1, 2600, 72), (2, 90, 33), (2, 300, 42)], ids=str)
@pytest.mark.parametrize("tied", [True, False])
def test_a_gate_that_is_no_number_stays_in_its_channel(package, shape, dtype, tied):
    """NaN and infinities in one channel's gate: the others are what they are without, bit for bit. Single samples, few, whole
    tiles by TMA, and channels that lanes load one by one."""
    B, N, C = shape
    gen = generator(2100 + N)
    x, gate, dh = (randn(gen, B, N, C, dtype=dtype, mean=m) for m in (0.0, 1.0, 0.0))
    state, dlast = randn(gen, B, C), randn(gen, B, C)

    def run(gate):
        leaves = [t.detach().clone().requires_grad_() for t in (x, gate, state)]
        h, last = package.gated_recurrence(*leaves, tied=tied, return_state=True)
        return [h.detach(), last.detach(), *torch.autograd.grad((h, last), leaves, (dh, dlast))]

    clean = run(gate)
    for c, value in ((4, math.nan), (5, math.nan), (4, math.inf), (5, -math.inf), (C - 1, math.nan)):
        for t in {0, N // 2}:
            spoilt = gate.clone()
            spoilt[0, t, c] = value
            got = run(spoilt)
            mine = torch.zeros(B, C, dtype=torch.bool, device="cuda")
            mine[0, c] = True
            for a, b, what in zip(got, clean, ("h", "last", "dx", "dgate", "dstate")):
                other = ~mine if a.dim() == 2 else (~mine)[:, None].expand_as(a)
                assert torch.equal(a[other], b[other]), (what, c, value, t)
            if math.isnan(value):
                assert torch.isnan(got[0][0, t:, c]).all() and torch.isnan(got[1][0, c]), (c, t)
                assert torch.equal(got[0][0, :t, c], clean[0][0, :t, c])
                assert torch.isnan(got[4][0, c]) and torch.isnan(got[3][0, t, c])
            else:
                assert not torch.isnan(got[0]).any() and not torch.isnan(got[2]).any()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("N", [1, 5, 200])
@pytest.mark.parametrize("C", [16, 15])
@pytest.mark.parametrize("tied", [True, False])
def test_gates_at_the_ends_of_their_range(package, dtype, N, C, tied):
    """Neighbouring channels at opposite extremes. A gate that is wide open keeps the state, one that is closed drops it, however
    large it is: both factors are as near as their own rounding wherever fp32 has normal numbers (exp(-87) and up)."""
    values = [math.inf, -math.inf, 200.0, -200.0, -math.inf, 30.0, -50.0, 60.0, -64.0, -200.0, 0.0, -86.0, -85.0, -41.0, -42.0, math.inf][:C]
    z = torch.tensor(values, device="cuda").to(dtype)
    gen = generator(2200 + N)
    gate = z.expand(2, N, C).contiguous().requires_grad_()
    x = randn(gen, 2, N, C, dtype=dtype).requires_grad_()
    state = torch.full((2, C), 1e25, device="cuda")
    state[0] = randn(gen, C)
    state[1, 11:13] = 1e37
    state.requires_grad_()
    dh, dlast = randn(gen, 2, N, C, dtype=dtype), randn(gen, 2, C)
    h, last = package.gated_recurrence(x, gate, state, tied=tied, return_state=True)
    dx, dgate, dstate = torch.autograd.grad((h, last), (x, gate, state), (dh, dlast))
    wide = z.double()
    a, o = torch.sigmoid(wide), torch.sigmoid(-wide)
    e = torch.where(torch.isinf(wide), torch.zeros_like(wide), (wide.abs() + 8) * 2.0 ** -22)
    f, m, d = state.detach().double(), state.detach().double().abs(), torch.zeros(2, C, dtype=torch.float64, device="cuda")
    want, limit = (torch.empty(2, N, C, dtype=torch.float64, device="cuda") for _ in range(2))
    floor = 2.0 ** -126
    for t in range(N):
        u = (o if tied else 1.0) * x.detach().double()[:, t]
        d = a * d + a * m * (o * e + 16 * U) + u.abs() * (a * e + 16 * U) + floor * (1 + m)
        f, m = a * f + u, a * m + u.abs()
        want[:, t], limit[:, t] = f, d + UT[dtype] * f.abs() + TINY[dtype]
    top = torch.finfo(dtype).max
    fits = want.abs() < 0.99 * top                     # fp16 has no 1e25
    got = torch.where(fits, h.double(), torch.zeros_like(want))
    within(got, torch.where(fits, want, torch.zeros_like(want)), limit, "h")
    assert torch.isinf(h[want.abs() > 1.01 * top]).all()
    within(last, f, d + U * f.abs() + floor, "last")
    g, md, dd = dlast.double(), dlast.double().abs(), torch.zeros_like(d)
    for t in reversed(range(N)):
        g, md = g + dh.double()[:, t], md + dh.double()[:, t].abs()
        dd = dd + 8 * U * md
        right = g * (o if tied else 1.0)
        within(dx[:, t], right, dd * (o if tied else 1.0) + right.abs() * (a * e + 16 * U + UT[dtype]) + TINY[dtype] + floor * md, f"dx {t}")
        dd = a * dd + a * md * (o * e + 8 * U) + floor * md
        g, md = a * g, a * md
    within(dstate, g, dd + U * g.abs() + floor, "dstate")
    open_ = torch.isinf(wide)
    assert torch.equal(dgate[..., open_], torch.zeros_like(dgate[..., open_]))
    closed = wide < -150
    assert torch.equal(h[..., closed], x[..., closed])


# --- fp16 gradients over a wide range

def test_large_gradients_of_some_rows_leave_the_others_exact(package):
    """fp16: dg and du are scaled by one power of two. A row of dh that is 2^18 times the others must not push theirs below fp16's
    normal numbers: each row's dx is as near as in test_results_are_as_near_as_their_rounding."""
    gen = generator(25)
    R, K, F = 600, 256, 384
    x, wg, wu = randn(gen, R, K, dtype=F16), *(randn(gen, F, K, dtype=F16, std=K ** -0.5) for _ in range(2))
    for large, at in ((2000.0, (7, 11)), (30000.0, (7, slice(0, 2))), (0.0, (0, 0))):
        dh = randn(gen, R, F, dtype=F16, std=1e-2)
        dh[at] = large
        want, _ = gated_reference(x, wg, wu, None, None, dh, "silu")
        leaf = x.detach().requires_grad_()
        (dx,) = torch.autograd.grad(package.gated_linear(leaf, wg, wu), leaf, dh)
        others = torch.arange(R, device="cuda") != at[0]
        error, own = (((t.double() - want[1])[others] ** 2).mean().sqrt() for t in (dx, want[1].to(F16)))
        assert error <= 1.6 * own, (large, float(error / own))
        if large < 4000:                                # what is off by less than a step of fp16 unscaled
            check_gated(package, x, wg, wu, None, None, dh, "silu")


@pytest.mark.parametrize("name", ["silu", "gelu", "relu", "sigmoid"])
def test_fp16_gradients_do_not_overflow_on_their_way(package, name):
    """dg and du beyond 65504 whose products with small weights are not: dx is finite, and right."""
    gen = generator(26)
    R, K, F = 100, 64, 96
    x = randn(gen, R, K, dtype=F16, std=8.0)
    wg, wu = randn(gen, F, K, dtype=F16, std=2.0 ** -9), randn(gen, F, K, dtype=F16, std=K ** -0.5)
    bg, bu = randn(gen, F, dtype=F16), randn(gen, F, dtype=F16)
    wu[:5] *= 8
    dh = randn(gen, R, F, dtype=F16, std=3e-2)
    dh[:, :5] = 3000.0                                  # u of these: up to 200
    want, bound = gated_reference(x, wg, wu, bg, bu, dh, name)
    assert float((dh.double()[:, :5] * (x.double() @ wu.double().T + bu.double())[:, :5]).abs().max()) > 4 * 65504
    leaf = x.detach().requires_grad_()
    (dx,) = torch.autograd.grad(package.gated_linear(leaf, wg, wu, bg, bu, activation=name), leaf, dh)
    keep = want[1].abs() < 65000
    assert float(keep.double().mean()) > 0.3
    within(torch.where(keep, dx.double(), 0.0), torch.where(keep, want[1], 0.0), bound[1], "dx")


@pytest.mark.parametrize("value", [math.inf, math.nan])
def test_fp16_rows_that_are_no_numbers_leave_the_others(package, value):
    """A row of x or of a weight that is not finite has no norm to scale dg and du by; the other rows' dx are right all the same."""
    gen = generator(27)
    R, K, F = 150, 64, 96
    x, wg, wu = randn(gen, R, K, dtype=F16), *(randn(gen, F, K, dtype=F16, std=K ** -0.5) for _ in range(2))
    dh = randn(gen, R, F, dtype=F16, std=1e-2)
    want, bound = gated_reference(x, wg, wu, None, None, dh, "silu")
    x[3, 5] = value
    leaf = x.detach().requires_grad_()
    (dx,) = torch.autograd.grad(package.gated_linear(leaf, wg, wu), leaf, dh)
    others = torch.arange(R, device="cuda") != 3
    within(dx[others], want[1][others], bound[1][others], "dx")
    assert not torch.isfinite(dx[3]).all()


# --- few rows, launched behind what comes before them

def test_few_rows_behind_other_work(package):
    """The kernels of few rows begin before what is in front of them on the stream has ended: behind a copy, behind a kernel that
    rewrites the weights or the rows in place, on several streams at once, and in graphs."""
    gen = generator(61)
    for dtype, K in ((BF16, 1024), (F16, 250), (F32, 512)):
        x = [randn(gen, 16, K, dtype=dtype) for _ in range(4)]
        w = [randn(gen, 512, K, dtype=dtype, std=K ** -0.5) for _ in range(4)]
        want = [[package.gated_linear(a, b, b).clone() for b in w] for a in x]
        torch.cuda.synchronize()
        a, b = x[0].clone(), w[0].clone()
        for turn in range(40):
            i, j = turn % 4, turn // 4 % 4
            a.copy_(x[i])
            if turn % 2:
                b.copy_(w[j])
            else:
                b.zero_()
                b.add_(w[j])
            assert torch.equal(package.gated_linear(a, b, b), want[i][j]), (dtype, turn)
        streams, got = [torch.cuda.Stream() for _ in range(4)], [[] for _ in range(4)]
        torch.cuda.synchronize()
        for turn in range(5):
            for i, s in enumerate(streams):
                with torch.cuda.stream(s):
                    own = w[i] * 1.0
                    own.add_(0)
                    got[i].append(package.gated_linear(x[(i + turn) % 4], own, own))
        torch.cuda.synchronize()
        assert all(torch.equal(got[i][t], want[(i + t) % 4][i]) for i in range(4) for t in range(5))
        # a graph: a copy in front of a call, the call, another on its result
        a, b, graph = x[0].clone(), w[0].clone(), torch.cuda.CUDAGraph()
        square = randn(gen, 512, 512, dtype=dtype, std=0.05)
        source = x[0].clone()
        with torch.cuda.graph(graph):
            a.copy_(source)
            h = package.gated_linear(a, b, b)
            out = package.gated_linear(h, square, square)
        for i in (2, 1, 3):
            source.copy_(x[i])
            b.copy_(w[i])
            graph.replay()
            assert torch.equal(h, want[i][i]) and torch.equal(out, package.gated_linear(want[i][i], square, square))


# 1: a cluster's first CTA sends nothing (there have to be several); 2: one warp gives up its loads
@pytest.mark.parametrize("shape,which", [((1, 2000, 64), 1), ((2, 5000, 64), 1), ((1, 2000, 64), 2), ((2, 5000, 64), 2), ((400, 70, 64), 2)], ids=str)
def test_recurrence_waits_that_run_out(package, shape, which):
    """Whoever gives up a wait, the warp that folds the others' runs or one that does not: all results of the cluster are NaN, forward
    and backward, the status says so, and the next call is right again."""
    B, N, C = shape
    gen = generator(71)
    lengths = torch.full((B,), N - 1, device="cuda", dtype=torch.int32)
    x, gate = (randn(gen, *shape, dtype=BF16, mean=m).requires_grad_() for m in (0.0, 1.0))
    state, dh, dlast = randn(gen, B, C).requires_grad_(), randn(gen, *shape, dtype=BF16), randn(gen, B, C)
    run = lambda: package.gated_recurrence(x, gate, state, lengths=lengths, return_state=True)  # noqa: E731
    back = lambda out: torch.autograd.grad(out, (x, gate, state), (dh, dlast))  # noqa: E731
    want = run()
    grads = back(want)
    assert package.sdtw_encoder_status() == 0
    try:
        for forward in (True, False):
            out = None if forward else run()
            torch.cuda.synchronize()
            package.sdtw_debug_set_wait(0.02, which)
            got = run() if forward else back(out)
            assert package.sdtw_encoder_status() == 7 and package.sdtw_encoder_status() == 0
            package.sdtw_debug_set_wait(0.0, 0)
            for t in got:
                t = t.detach()
                if t.dim() == 3:
                    assert torch.equal(t[:, N - 1:], torch.zeros_like(t[:, N - 1:]))
                    t = t[:, :N - 1]
                assert torch.isnan(t).all()
    finally:
        package.sdtw_debug_set_wait(0.0, 0)
    again = run()
    assert all(torch.equal(a, b) for a, b in zip((*again, *back(again)), (*want, *grads)))


def test_group_norm_of_as_many_positions_as_32_bits_count(package):
    """One channel over 2^31 - 1 positions, all 0 but for some at both ends and in the middle: the mean is 0 to a part in 10^7 of the
    deviation, and what is not 0 is where it was."""
    S = 2 ** 31 - 1
    x = torch.zeros(1, S, 1, device="cuda", dtype=BF16)
    at = torch.tensor([0, 1, S // 2, S - 17, S - 16, S - 2, S - 1], device="cuda")
    x[0, at, 0] = torch.tensor([1.0, -2.0, 3.0, 4.0, -5.0, 6.0, -7.0], device="cuda", dtype=BF16)
    y = package.group_norm(x, 1, eps=1.0)
    assert torch.equal(y[0, at, 0], x[0, at, 0])              # a variance of 7e-8 beside eps = 1
    rest = y.view(-1)
    assert all(float(c.abs().sum(dtype=torch.float64)) <= 28.1 for c in rest.split(1 << 29))
    assert int((rest.abs() > 1e-6).sum()) == 7
    del x, y, rest
    torch.cuda.empty_cache()


@pytest.mark.parametrize("value", [math.inf, 3.395e38, 3.4e38])
def test_fp32_values_without_three_parts(package, value):
    """A forward pass of at most 32 rows of fp32 takes a weight as it is. More rows, and every backward pass, take it in three bf16 parts,
    which infinities and what rounds to one in bf16, from (2 - 2^-8) 2^127 = 3.3961e38 on, have not: NaN where such a value takes
    part, and all else right."""
    gen = generator(28)
    R, K, F = 8, 64, 40
    x, wg, wu, dh = randn(gen, R, K), *(randn(gen, F, K, std=K ** -0.5) for _ in range(2)), randn(gen, R, F)
    x[:, 3] = 2.0 ** -20
    want, bound = gated_reference(x, wg, wu, None, None, dh, "silu")
    wu[5, 3] = value
    x, wg, wu = (t.requires_grad_() for t in (x, wg, wu))
    h = package.gated_linear(x, wg, wu)
    others = torch.arange(F, device="cuda") != 5
    within(h[:, others], want[0][:, others], bound[0][:, others], "h")
    assert not torch.isnan(h).any() and torch.isinf(h[:, 5]).all() == math.isinf(value)
    dx, dwg, dwu = torch.autograd.grad(h, (x, wg, wu), dh)
    none = value >= (2 - 2.0 ** -8) * 2.0 ** 127
    assert torch.isnan(dx).all() if none else not torch.isnan(dx).any()
    assert torch.isnan(dwg[5]).all() if none else torch.isfinite(dwg[5]).all()
    within(dwg[others], want[2][others], bound[2][others], "dgate_weight")
    within(dwu, want[3], bound[3], "dup_weight")                # needs g alone
    many = package.gated_linear(x.repeat(5, 1), wg, wu)
    assert torch.isnan(many[:, 5]).all() == none and not torch.isnan(many[:, others]).any()


def test_captured_fp16_gradients_follow_their_inputs(package):
    """What fp16's gradients are scaled by is found anew in every replay."""
    gen = generator(62)
    R, K, F = 300, 72, 136
    x, wg, wu = randn(gen, R, K, dtype=F16), *(randn(gen, F, K, dtype=F16, std=K ** -0.5) for _ in range(2))
    dh = randn(gen, R, F, dtype=F16)
    run = lambda: torch.autograd.grad(package.gated_linear(*leaves), leaves, dh)  # noqa: E731
    leaves = [t.requires_grad_() for t in (x, wg, wu)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for scale in (2.0 ** -14, 1.0, 2.0 ** 4, 2.0 ** -8):
        dh.copy_(randn(gen, R, F, dtype=F16, std=scale))
        with torch.no_grad():
            x.copy_(randn(gen, R, K, dtype=F16, std=0.5))
        graph.replay()
        want, _ = gated_reference(x.detach(), wg.detach(), wu.detach(), None, None, dh, "silu")
        for g, exact, what in zip(got, want[1:], ("dx", "dwg", "dwu")):
            error, own = (((t.double() - exact) ** 2).mean().sqrt() for t in (g, exact.to(F16)))
            assert error <= 1.6 * own, (what, scale, float(error / own))
