"""How far attention's 16-bit results are from 64 bits, against what rounding them once to the type costs.

In the 2-norm over a whole result, independent roundings add in squares. out and dv have their own rounding and that of the
probabilities, each one rounding to the type of terms of the result: sqrt(2). dq and dk have their own, that of the gradients of
the scores, and what rounded probabilities leave in delta, which is a part of one more: at most sqrt(3). 6 % are left for roundings
that are not quite alike. Results of few values differ by more than that among themselves, so that small problems come in
many heads."""
import pytest

from test_gpu_encoder import BF16, F16, attention_reference, generator, package, randn, visible  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("B,N,M,Hq,Hkv,D", [(32, 3, 3, 8, 8, 48), (32, 6, 6, 8, 4, 104), (64, 2, 2, 8, 8, 40), (16, 5, 40, 12, 4, 64), (8, 10, 528, 6, 6, 56),
                                            (2, 276, 276, 8, 8, 40), (4, 512, 512, 8, 8, 64), (2, 700, 700, 8, 4, 128), (1, 1100, 1300, 8, 8, 80)])
@pytest.mark.parametrize("causal", [False, True])
def test_results_are_as_near_as_their_own_rounding(package, B, N, M, Hq, Hkv, D, causal, dtype):  # noqa: F811
    gen = generator(N + M + D)
    q, do = randn(gen, B, N, Hq, D, dtype=dtype, std=1.5), randn(gen, B, N, Hq, D, dtype=dtype, std=0.01)
    k, v = randn(gen, B, M, Hkv, D, dtype=dtype, std=1.5), randn(gen, B, M, Hkv, D, dtype=dtype)
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    out = package.attention(*leaves, causal=causal)
    got = dict(zip(("out", "dq", "dk", "dv"), (out.detach(), *torch.autograd.grad(out, leaves, do))))
    want, _, _ = attention_reference(q, k, v, do, D ** -0.5, visible(B, N, M, causal, None, None, None), dtype, True)
    for name, g in got.items():
        exact = want[name][0]
        off, own = float((g.double() - exact).norm()), float((exact.to(dtype).double() - exact).norm())
        assert off <= 1.06 * (2 if name in ("out", "dv") else 3) ** 0.5 * own, f"{name}: {off / own:.3f} times its own rounding"
