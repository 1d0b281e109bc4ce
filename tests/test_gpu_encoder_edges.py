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
