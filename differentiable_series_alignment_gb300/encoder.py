"""Operators of a sequence encoder whose outputs Soft-DTW aligns, differentiable (once):

    layer_norm(x, weight, bias, eps=1e-5)
    rotary_table(length, dim, ...), rotary(q, k, table=..., positions=None, interleaved=False)
    attention(q, k, v, causal=False, window=None, q_lengths=None, k_lengths=None, scale=None)

Tensors are fp32, bf16 or fp16 on a CUDA device; every step of the operators runs
in libsdtw.so's kernels, on the current stream of the tensors' device. Wrong shapes and
values raise ValueError, wrong types TypeError, tangents of forward-mode differentiation NotImplementedError,
and what the library itself refuses (sizes beyond its limits) SdtwError, as every other entry.
"""
from __future__ import annotations

import math

import torch

from . import _lib


def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
               eps: float = 1e-5) -> torch.Tensor:
    """(x - mean) / sqrt(var + eps) * weight + bias over the last dimension of x (..., C),
    differentiable in x, weight and bias. weight and bias (C,) are of x's type or fp32, both
    alike; the statistics and the sums of the weights' gradients are formed in fp32."""
    return _lib.binding().layer_norm(x, weight, bias, eps)


def rotary_table(length: int, dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                 original_length: int | None = None, beta_fast: float = 32.0, beta_slow: float = 1.0,
                 device=None) -> torch.Tensor:
    """Cosines and sines (length, dim / 2, 2) of the angles position * base^(-2i / dim), for
    `rotary`; made once, in 64 bits, and rounded to fp32.

    scaling stretches a model trained on original_length positions to factor times as many:
    "linear" divides every position by factor; "ntk" raises the base by factor^(dim / (dim - 2)),
    which leaves the fastest pair as it was and divides the slowest by factor; "yarn" divides only the
    pairs that turn less than beta_slow times over original_length, leaves those that turn more than
    beta_fast times, goes from one to the other linearly in the pair's index, and multiplies cosines and
    sines by 0.1 ln(factor) + 1 (Peng et al., 2023)."""
    if length < 1 or dim < 2 or dim % 2:
        raise ValueError("length must be >= 1 and dim even and >= 2")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError("scaling must be None, 'linear', 'ntk' or 'yarn'")
    if not (1 < base < math.inf and 1 <= factor < math.inf):
        raise ValueError("base must be > 1 and factor >= 1, both finite")
    pair = torch.arange(dim // 2, dtype=torch.float64, device="cuda" if device is None else device)
    magnitude = 1.0
    if scaling == "ntk":
        if dim < 4:
            raise ValueError("scaling='ntk' needs dim >= 4")
        base = base * factor ** (dim / (dim - 2))
    freq = base ** (-2.0 * pair / dim)
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "yarn":
        if original_length is None or original_length < 1:
            raise ValueError("scaling='yarn' needs original_length")
        if not 0 < beta_slow < beta_fast < math.inf:
            raise ValueError("scaling='yarn' needs 0 < beta_slow < beta_fast")
        # the pair that turns `turns` times over the original length
        at = lambda turns: dim * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        # either end of the ramp may lie beyond the pairs that there are
        first, last = math.floor(at(beta_fast)), math.ceil(at(beta_slow))
        slow = ((pair - first) / max(last - first, 1)).clamp(0, 1)
        freq = freq * (1 - slow) + freq / factor * slow
        magnitude = 0.1 * math.log(factor) + 1.0
    angle = torch.arange(length, dtype=torch.float64, device=pair.device)[:, None] * freq
    return (torch.stack([angle.cos(), angle.sin()], dim=-1) * magnitude).to(torch.float32)


def rotary(q: torch.Tensor, k: torch.Tensor | None = None, *, table: torch.Tensor,
           positions: torch.Tensor | None = None, interleaved: bool = False):
    """q (B, N, Hq, D) and, where given, k (B, N, Hkv, D) with the first 2 * table.shape[1]
    features of every head turned by their position's angles, differentiable in q and k. Returns the
    turned q, or (q, k). Pairs are neighbouring features (interleaved) or (i, i + R/2). positions (B, N) or
    (N,) integers of any width index the table; None stands for 0 .. N-1. A position outside the table gives NaN."""
    out = _lib.binding().rotary(q, k, table, positions, interleaved)
    return out[0] if k is None else tuple(out)


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, causal: bool = False, window: int | None = None,
              q_lengths: torch.Tensor | None = None, k_lengths: torch.Tensor | None = None,
              scale: float | None = None, return_lse: bool = False):
    """softmax(scale q k^T) v over the visible keys, (B, N, Hq, D), differentiable in q, k and v.

    q is (B, N, Hq, D), k and v are (B, M, Hkv, D) with Hq a multiple of Hkv: query head h reads key
    head h // (Hq // Hkv). D is at most 128; scale defaults to 1 / sqrt(D). Any strides do where features
    are contiguous (slices of one projection, a cache longer than what is filled of it).

    q_lengths and k_lengths (B,), bounded by N and M, make a padded batch: element b has n_b rows and m_b keys, and
    what lies beyond them is not used. Row n stands at key n + (m_b - n_b), so the newest row stands at the newest
    key: causal hides the keys after a row's own, window=w the keys w or more away from it. Rows without a
    visible key, and rows from n_b on, are 0 and pass no gradient.

    Scores, sums and accumulators are fp32. In bf16 and fp16 the tensor cores take the probabilities and, in the
    backward pass, the gradients of the scores rounded to the type: results are some 1.2 (out), 1.4 (dk, dv) and 1.5
    (dq) times as far from exact as their own rounding. float32 rounds results alone.

    N = 1 over a cache of M keys is the step of a growing series; the key axis is then split over the SMs.
    return_lse gives (out, lse): the logarithm (B, Hq, N) of each row's sum of exp(score), fp32, not
    differentiable, -inf for rows that see nothing."""
    out = _lib.binding().attention(q, k, v, causal, window, q_lengths, k_lengths, scale, return_lse)
    return tuple(out) if return_lse else out[0]
