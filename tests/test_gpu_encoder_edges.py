"""The encoder operators at the edges of their arguments: addresses, index types, sizes, and rows that take no part."""
import math

import pytest

from helpers import ensure_built

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def package():
    ensure_built()
    import differentiable_series_alignment_gb300 as p
    p.load()
    return p


def randn(gen, *shape, dtype=F32, std=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float64) * std).to(dtype)


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# --- rotary positions ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("offset", [1, 2, 3])
def test_a_rotary_table_may_begin_anywhere(package, offset, interleaved, dtype):
    """A contiguous view that begins at any element of a flat buffer: 4, 8 and 12 bytes off a 16-byte boundary."""
    gen = generator(1)
    table = package.rotary_table(40, 16)
    flat = torch.empty(offset + table.numel(), device="cuda")
    view = flat[offset:].view(table.shape).copy_(table)
    q = randn(gen, 2, 33, 3, 24, dtype=dtype).requires_grad_()
    up = randn(gen, 2, 33, 3, 24, dtype=dtype)
    got, want = (package.rotary(q, table=t, interleaved=interleaved) for t in (view, table))
    assert torch.equal(got, want)
    assert torch.equal(*(torch.autograd.grad(y, q, up)[0] for y in (got, want)))


@pytest.mark.parametrize("wide", [torch.int64, torch.uint32])
def test_positions_past_32_bits_are_outside_the_table(package, wide):
    table = package.rotary_table(16, 4)
    x = randn(generator(2), 1, 5, 2, 6)
    far = [2 ** 32 + 3, 2 ** 31, -2 ** 32 + 1, -2 ** 63] if wide == torch.int64 else [2 ** 31, 2 ** 32 - 1, 2 ** 31 + 3, 16]
    positions = torch.tensor([3] + far, dtype=wide, device="cuda")
    got = package.rotary(x, table=table, positions=positions)
    assert torch.isnan(got[:, 1:, :, :4]).all()
    assert torch.equal(got[:, :1], package.rotary(x[:, :1], table=table, positions=torch.tensor([3], device="cuda", dtype=torch.int32)))
    assert torch.equal(got[..., 4:], x[..., 4:])


# --- attention ----------------------------------------------------------------------------------

@pytest.mark.parametrize("place", ["cuda", "cpu"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_lengths_past_32_bits_are_all_there_is(package, dtype, place):
    gen = generator(3)
    B, N, M = 6, 9, 70
    q, k, v = randn(gen, B, N, 2, 32, dtype=dtype), randn(gen, B, M, 2, 32, dtype=dtype), randn(gen, B, M, 2, 32, dtype=dtype)
    far = torch.tensor([2 ** 63 - 1, 2 ** 31, 2 ** 32 + 5, -2 ** 40, -2 ** 63, 8], device=place)
    near = lambda n: torch.tensor([n, n, n, 0, 0, 8], dtype=torch.int32, device="cuda")  # noqa: E731
    got = package.attention(q, k, v, causal=True, q_lengths=far, k_lengths=far, return_lse=True)
    want = package.attention(q, k, v, causal=True, q_lengths=near(N), k_lengths=near(M), return_lse=True)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


# --- sizes --------------------------------------------------------------------------------------

def test_dimensions_past_32_bits_are_refused(package):
    """Views whose strides are 0 have any size for a few bytes: none of it may be cut to 32 bits."""
    table = package.rotary_table(8, 4)
    one = torch.zeros(1, 1, 1, 8, device="cuda")
    for shape in ((2 ** 32 + 2, 1, 1, 8), (1, 2 ** 32 + 2, 1, 8), (1, 1, 2 ** 32 + 2, 8), (1, 2 ** 31, 1, 8)):
        long = one.expand(shape)
        with pytest.raises(ValueError):
            package.rotary(long, table=table, positions=torch.zeros((), dtype=torch.int32, device="cuda").expand(shape[:2]))
        with pytest.raises(ValueError):
            package.attention(long, one.expand(shape[0], 1, 1, 8), one.expand(shape[0], 1, 1, 8))
    with pytest.raises(ValueError):
        package.rotary(one, one.expand(1, 1, 2 ** 32 + 2, 8), table=table)
    for shape in ((1, 2 ** 32 + 5, 1, 8), (1, 1, 2 ** 32 + 1, 8)):
        long = one.expand(shape)
        with pytest.raises(ValueError):
            package.attention(one.expand(1, 1, shape[2], 8), long, long)


def test_a_table_may_have_more_positions_than_32_bits_count(package):
    """17 GB, of which a call reads a few lines."""
    table = torch.zeros(2 ** 31 + 8, 1, 2, device="cuda")
    table[7, 0, 0] = 1.0
    x = randn(generator(4), 1, 2, 1, 2)
    got = package.rotary(x, table=table, positions=torch.tensor([7, -1], device="cuda"))
    assert torch.equal(got[:, 0], x[:, 0]) and torch.isnan(got[:, 1]).all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rotary_of_no_heads_beside_some(package, dtype, interleaved):
    """Slices of a projection that leave q or k without a head: the other one is turned as it is alone."""
    gen = generator(5)
    table = package.rotary_table(16, 8)
    some, none = randn(gen, 2, 5, 3, 16, dtype=dtype), randn(gen, 2, 5, 0, 16, dtype=dtype)
    up = randn(gen, 2, 5, 3, 16, dtype=dtype)
    alone = some.clone().requires_grad_()
    want = package.rotary(alone, table=table, interleaved=interleaved)
    gradient, = torch.autograd.grad(want, alone, up)
    for first in (True, False):
        torch.full((2, 5, 3, 16), math.nan, device="cuda", dtype=dtype)      # what the allocator gives next holds NaN
        leaf = some.clone().requires_grad_()
        out = package.rotary(*((leaf, none) if first else (none, leaf)), table=table, interleaved=interleaved)
        got, empty = out if first else out[::-1]
        assert torch.equal(got, want) and empty.shape == none.shape
        assert torch.equal(torch.autograd.grad(got, leaf, up)[0], gradient)
    assert package.rotary(none, table=table).shape == none.shape
    assert [t.shape for t in package.rotary(none, none, table=table)] == [none.shape] * 2


# --- derivatives --------------------------------------------------------------------------------

def test_forward_mode_tangents_are_refused(package):
    """There is no forward-mode derivative; a result without a tangent would stand for a derivative of zero."""
    fwd = torch.autograd.forward_ad
    gen = generator(6)
    x, w, q, k = randn(gen, 4, 8), randn(gen, 8), randn(gen, 1, 5, 2, 8), randn(gen, 1, 7, 2, 8)
    table = package.rotary_table(8, 8)
    calls = [(package.layer_norm, (x, w, w)), (lambda a, b: package.rotary(a, b, table=table), (q, q.clone())),
             (package.attention, (q, k, k.clone()))]
    for call, args in calls:
        for grad in (False, True):
            leaves = [t.clone().requires_grad_(grad) for t in args]
            call(*leaves)
            for at in range(len(args)):
                with fwd.dual_level():
                    dual = [fwd.make_dual(t, torch.ones_like(t)) if n == at else t for n, t in enumerate(leaves)]
                    with pytest.raises(RuntimeError):          # NotImplementedError is one
                        call(*dual)
                    with torch.no_grad(), pytest.raises(RuntimeError):
                        call(*dual)
    with fwd.dual_level():
        dual = fwd.make_dual(x, torch.ones_like(x))
        with fwd._set_fwd_grad_enabled(False):                 # as in a function that brings its own rule
            got = package.layer_norm(dual, w, w)
        assert torch.equal(got, package.layer_norm(x, w, w))


# --- rows that see no key -----------------------------------------------------------------------

@pytest.mark.parametrize("dtype,D", [(F32, 64), (F32, 63), (F32, 128), (BF16, 64), (BF16, 128), (BF16, 36), (F16, 40), (F16, 128)])
@pytest.mark.parametrize("N,M,Hq,Hkv", [(200, 90, 2, 2), (130, 5, 4, 2), (70, 69, 3, 1), (300, 40, 8, 2), (9, 3, 2, 1)])
@pytest.mark.parametrize("padded", [False, True])
def test_rows_that_see_no_key_leave_no_trace(package, N, M, Hq, Hkv, padded, dtype, D):
    """More rows than keys under a causal mask: the first rows stand before every key. Their output is 0, so what follows
    may well give them a gradient of NaN (a division by their norm), and their queries may hold anything."""
    gen = generator(N + M + D)
    B = 3
    ql = torch.tensor([N, N - 2, N], dtype=torch.int32, device="cuda") if padded else None
    kl = torch.tensor([M, M - 1, 0], dtype=torch.int32, device="cuda") if padded else None
    n, m = (t.tolist() if padded else [e] * B for t, e in ((ql, N), (kl, M)))
    q, do = randn(gen, B, N, Hq, D, dtype=dtype, std=1.5), randn(gen, B, N, Hq, D, dtype=dtype, std=0.3)
    k, v = randn(gen, B, M, Hkv, D, dtype=dtype, std=1.5), randn(gen, B, M, Hkv, D, dtype=dtype)
    blind = [range(n[b] if m[b] == 0 else max(0, n[b] - m[b])) for b in range(B)]
    for window in (None, 30):
        results = []
        for anything in (0.0, math.nan, math.inf, 6e4):
            for b in range(B):
                q[b, blind[b]], do[b, blind[b]] = anything, anything
            leaves = [t.clone().requires_grad_() for t in (q, k, v)]
            out = package.attention(*leaves, causal=True, window=window, q_lengths=ql, k_lengths=kl)
            results.append((out.detach(), *torch.autograd.grad(out, leaves, do)))
        for b in range(B):
            assert (results[0][0][b, blind[b]] == 0).all() and (results[0][1][b, blind[b]] == 0).all()
        for other in results[1:]:
            for a, b in zip(results[0], other):
                assert torch.equal(a, b)


@pytest.mark.parametrize("dtype,D", [(F32, 64), (BF16, 64), (BF16, 128), (F16, 36)])
def test_rows_that_see_no_key_are_0_beside_rows_of_nan(package, dtype, D):
    """Keys that other rows see may be NaN: the rows that see none are 0 all the same, and so is their gradient."""
    gen = generator(D)
    q, k, v = (randn(gen, 1, n, 2, D, dtype=dtype) for n in (40, 10, 10))
    do = randn(gen, 1, 40, 2, D, dtype=dtype)
    k[:, 4], v[:, 4] = math.nan, math.inf
    leaves = [t.requires_grad_() for t in (q, k, v)]
    out = package.attention(*leaves, causal=True)
    dq, = torch.autograd.grad(out, leaves[:1], do)
    assert (out[:, :30] == 0).all() and (dq[:, :30] == 0).all()
    assert torch.isnan(out[:, 34:]).all() and torch.isnan(dq[:, 34:]).all()


# --- waits that run out -------------------------------------------------------------------------

@pytest.mark.parametrize("how", [1, 2])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("N,M,D", [(1, 256, 128), (3, 250, 64), (200, 500, 64), (200, 500, 128)])
def test_a_wait_that_runs_out_leaves_nan_in_all_that_hangs_on_it(package, N, M, D, dtype, how):
    """The loads are withheld, all of them or those of one chain of waits (a test hook; no fault is involved): whatever
    the others of the CTA have computed by then, no row keeps a number that the missing part should have entered."""
    gen = generator(M)
    leaves = [randn(gen, 1, n, 2, D, dtype=dtype).requires_grad_() for n in (N, M, M)]
    do = randn(gen, 1, N, 2, D, dtype=dtype)
    out = package.attention(*leaves)
    want = (out.detach(), *torch.autograd.grad(out, leaves, do, retain_graph=True))
    debug, late = package.load().sdtw_debug_set_wait, 7            # SDTW_ERR_TIMEOUT
    assert package.sdtw_encoder_status() == 0
    try:
        debug(0.02, how)
        assert torch.isnan(package.attention(*leaves).detach()).all()
        assert package.sdtw_encoder_status() == late
        debug(0.02, how)
        grads = torch.autograd.grad(out, leaves, do, retain_graph=True)
        assert package.sdtw_encoder_status() == late
        for g in grads:
            assert torch.isnan(g).all()
    finally:
        debug(0.0, 0)
    again = package.attention(*leaves)
    for a, b in zip((again.detach(), *torch.autograd.grad(again, leaves, do)), want):
        assert torch.equal(a, b)
    assert package.sdtw_encoder_status() == 0


# --- refusals -----------------------------------------------------------------------------------

def test_values_outside_fp32_are_refused_like_other_wrong_values(package):
    x, q = torch.ones(2, 8, device="cuda"), torch.ones(1, 2, 1, 8, device="cuda")
    for eps in (1e39, 1e300):
        with pytest.raises(ValueError):
            package.layer_norm(x, eps=eps)
    for scale in (1e-60, 1e39, 1e300):
        with pytest.raises(ValueError):
            package.attention(q, q, q, scale=scale)
    assert torch.isfinite(package.attention(q, q, q, scale=1e-30)).all()


def test_what_the_library_refuses_is_the_package_s_own_error(package):
    """Sizes that only the C entry knows the limits of: the same error as from every other entry, with its status."""
    x = torch.zeros(1, (1 << 24) + 1, device="cuda")
    q = torch.zeros(1, 1, 1, 1, device="cuda")
    rows = q.expand(1, (1 << 27) + 1, 1, 1)
    for call in (lambda: package.layer_norm(x), lambda: package.attention(q, rows, rows), lambda: package.layer_norm(x.requires_grad_())):
        with pytest.raises(package.SdtwError) as e:
            call()
        assert e.value.code == 8 and "SDTW_ERR_TOO_LARGE" in str(e.value)
