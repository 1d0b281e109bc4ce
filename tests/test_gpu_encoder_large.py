"""The encoder operators at sizes whose kernels no small call takes, and with gradients of some inputs only.

References and their bounds, which grow with the sums' lengths, are those of test_gpu_encoder.py."""
import itertools

import pytest

from test_gpu_encoder import (BF16, F16, F32, check_attention, generator, norm_reference, package, randn, rotated,  # noqa: F401
                              within)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# --- attention ----------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("B,N,M,Hq,Hkv,D", [(3, 1100, 1100, 12, 3, 128), (2, 1300, 1537, 16, 16, 80), (5, 700, 333, 24, 8, 96),
                                            (4, 130, 1900, 40, 40, 72)])
@pytest.mark.parametrize("causal,window,ragged", [(True, None, False), (False, None, True), (True, 600, True), (False, 150, False)])
def test_attention_of_two_row_tiles_a_cta(package, B, N, M, Hq, Hkv, D, causal, window, ragged, dtype):  # noqa: F811
    """Wide heads and enough tiles for every SM: two tiles of rows share the keys, and see parts of them."""
    rows = 128 // (Hq // Hkv) * (Hq // Hkv)
    assert D > 64 and N * (Hq // Hkv) > rows and -(-N * (Hq // Hkv) // rows) * B * Hkv >= 2 * sms()
    gen = generator(N + M + D)
    q, do = randn(gen, B, N, Hq, D, dtype=dtype, std=1.5), randn(gen, B, N, Hq, D, dtype=dtype, std=0.3)
    k, v = randn(gen, B, M, Hkv, D, dtype=dtype, std=1.5), randn(gen, B, M, Hkv, D, dtype=dtype)

    def lengths(n):
        return torch.tensor([n - 3, n // 3, n, 0, n // 2 + 1][:B], device="cuda", dtype=torch.int32) if ragged else None
    if ragged:
        for b, (n, m) in enumerate(zip(lengths(N).tolist(), lengths(M).tolist())):
            q[b, n:], do[b, n:], k[b, m:], v[b, m:] = (float("nan"),) * 4
    check_attention(package, q, k, v, do, dtype, causal, window, lengths(N), lengths(M))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("N,M,G", [(3, 200, 128), (2, 130, 200), (5, 77, 100)])
def test_attention_of_many_heads_on_one_key_head(package, N, M, G, dtype):  # noqa: F811
    """A position's heads fill a tile of rows, or more than one."""
    gen = generator(G)
    q, do = randn(gen, 2, N, G, 64, dtype=dtype, std=1.5), randn(gen, 2, N, G, 64, dtype=dtype, std=0.3)
    k, v = randn(gen, 2, M, 1, 64, dtype=dtype, std=1.5), randn(gen, 2, M, 1, 64, dtype=dtype)
    for args in (dict(), dict(causal=True, window=20)):
        check_attention(package, q, k, v, do, dtype, **args)


@pytest.mark.parametrize("dtype,D,N,M", [(F32, 64, 100, 130), (BF16, 64, 100, 300), (BF16, 128, 300, 200), (F16, 40, 100, 130), (F16, 63, 33, 70),
                                         (BF16, 64, 1, 500)])
def test_attention_gradients_of_some_inputs(package, dtype, D, N, M):  # noqa: F811
    gen = generator(D)
    q, do = randn(gen, 2, N, 4, D, dtype=dtype), randn(gen, 2, N, 4, D, dtype=dtype)
    k, v = randn(gen, 2, M, 2, D, dtype=dtype), randn(gen, 2, M, 2, D, dtype=dtype)
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    every = torch.autograd.grad(package.attention(*leaves, causal=True), leaves, do)
    for want in itertools.product((False, True), repeat=3):
        if any(want):
            some = [t.clone().requires_grad_(w) for t, w in zip((q, k, v), want)]
            out = package.attention(*some, causal=True)
            got = torch.autograd.grad(out, [t for t, w in zip(some, want) if w], do)
            assert all(torch.equal(a, b) for a, b in zip(got, [g for g, w in zip(every, want) if w])), want


# --- layer norm ---------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,wdtype,rows,C", [
    (F32, F32, 30001, 256), (F32, F32, 20011, 300), (F32, F32, 160003, 16), (F32, F32, 90001, 28), (F32, F32, 5003, 1024),
    (F32, F32, 2503, 2000), (F32, F32, 2503, 4096), (F32, F32, 9800, 101), (BF16, F32, 30001, 512), (BF16, F32, 20011, 1000),
    (BF16, BF16, 160003, 32), (BF16, F32, 90001, 120), (BF16, F32, 5003, 2048), (BF16, F32, 3001, 4096), (BF16, F32, 2503, 8192),
    (BF16, F32, 9800, 1003), (F16, F16, 20011, 264), (F16, F32, 20011, 1024), (F16, F16, 9728, 520), (F16, F16, 9727, 520)])
def test_norm_of_many_rows(package, dtype, wdtype, rows, C):  # noqa: F811
    """More rows than all CTAs take in the rounds that they have on their way, so that every place in shared memory is used again."""
    gen = generator(rows + C)
    x = randn(gen, rows, C, dtype=dtype, std=1.7, mean=0.6).requires_grad_()
    w, b = randn(gen, C, dtype=wdtype, std=0.3, mean=1.0).requires_grad_(), randn(gen, C, dtype=wdtype, std=0.3).requires_grad_()
    dy = randn(gen, rows, C, dtype=dtype, std=0.1)
    y = package.layer_norm(x, w, b, 1e-3)
    got = (y, *torch.autograd.grad(y, (x, w, b), dy))
    reference = norm_reference(x.detach(), w.detach(), b.detach(), dy, 1e-3, dtype, wdtype)
    for name, g, (want, bound) in zip(("y", "dx", "dw", "db"), got, reference):
        within(g.detach(), want, bound, f"{name} of {rows} x {C}")


@pytest.mark.parametrize("dtype,rows,C", [(F32, 300, 64), (BF16, 700, 1024), (BF16, 40, 8200), (F16, 33, 101)])
def test_norm_gradients_of_some_inputs(package, dtype, rows, C):  # noqa: F811
    gen = generator(rows + C)
    x, dy = randn(gen, rows, C, dtype=dtype, mean=0.5), randn(gen, rows, C, dtype=dtype)
    w, b = randn(gen, C, mean=1.0), randn(gen, C)
    leaves = [t.clone().requires_grad_() for t in (x, w, b)]
    every = torch.autograd.grad(package.layer_norm(*leaves), leaves, dy)
    for want in itertools.product((False, True), repeat=3):
        if any(want):
            some = [t.clone().requires_grad_(q) for t, q in zip((x, w, b), want)]
            got = torch.autograd.grad(package.layer_norm(*some), [t for t, q in zip(some, want) if q], dy)
            assert all(torch.equal(a, c) for a, c in zip(got, [g for g, q in zip(every, want) if q])), want
    # without weights, and with a bias alone: a weight of ones, a bias of zeros
    for given in ((False, False), (False, True), (True, False)):
        leaf, ones, zeros = x.clone().requires_grad_(), torch.ones_like(w), torch.zeros_like(b)
        parts = [t.clone().requires_grad_() if g else None for t, g in zip((w, b), given)]
        y = package.layer_norm(leaf, *parts)
        got = torch.autograd.grad(y, [leaf] + [t for t in parts if t is not None], dy)
        full = [leaf, *(t if t is not None else o.requires_grad_() for t, o in zip(parts, (ones, zeros)))]
        z = package.layer_norm(*full)
        same = torch.autograd.grad(z, full, dy)
        assert torch.equal(y, z)
        assert all(torch.equal(a, c) for a, c in zip(got, [same[0]] + [s for s, g in zip(same[1:], given) if g])), given


# --- rotary positions ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,N,Hq,Hkv,D,R", [(2, 4096, 9, 3, 128, 128), (3, 2731, 11, 2, 96, 32), (5, 6007, 6, 1, 64, 64)])
def test_rotary_of_two_heads_a_thread(package, B, N, Hq, Hkv, D, R, interleaved, dtype):  # noqa: F811
    units = ((R if interleaved else R // 2) + D - R) // (4 if dtype == F32 else 8)
    assert -(-B * N * units // 256) * ((Hq + Hkv + 1) // 2) >= 9 * 152
    gen = generator(N)
    table = package.rotary_table(8192, R)
    q, k = randn(gen, B, N, Hq, D, dtype=dtype).requires_grad_(), randn(gen, B, N, Hkv, D, dtype=dtype).requires_grad_()
    dq, dk = randn(gen, B, N, Hq, D, dtype=dtype), randn(gen, B, N, Hkv, D, dtype=dtype)
    for positions in (None, torch.randint(0, 8192, (B, N), generator=gen, device="cuda", dtype=torch.int32)):
        out = package.rotary(q, k, table=table, positions=positions, interleaved=interleaved)
        grads = torch.autograd.grad(out, (q, k), (dq, dk))
        for name, got, x, inverse in (("q", out[0], q, False), ("k", out[1], k, False), ("dq", grads[0], dq, True), ("dk", grads[1], dk, True)):
            within(got.detach(), *rotated(x.detach(), table, positions, interleaved, inverse), name)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rotary_gradients_of_some_inputs(package, dtype):  # noqa: F811
    gen = generator(9)
    table = package.rotary_table(64, 32)
    q, k, dq, dk = (randn(gen, 2, 50, h, 48, dtype=dtype) for h in (4, 2, 4, 2))
    leaves = [t.clone().requires_grad_() for t in (q, k)]
    both = torch.autograd.grad(package.rotary(*leaves, table=table), leaves, (dq, dk))
    only = q.clone().requires_grad_()
    assert torch.equal(torch.autograd.grad(package.rotary(only, k, table=table)[0], only, dq)[0], both[0])
    assert torch.equal(torch.autograd.grad(package.rotary(only, table=table), only, dq)[0], both[0])
    only = k.clone().requires_grad_()
    assert torch.equal(torch.autograd.grad(package.rotary(q, only, table=table)[1], only, dk)[0], both[1])
    # an output that nothing follows from
    assert torch.equal(torch.autograd.grad(package.rotary(*leaves, table=table)[0], leaves, dq)[1], torch.zeros_like(k))
