"""Operators of a sequence encoder whose outputs Soft-DTW aligns, differentiable:

    layer_norm(x, weight, bias, eps=1e-5)
    rotary_table(length, dim, ...), rotary(q, k, table=..., positions=None, interleaved=False)
    attention(q, k, v, causal=False, window=None, q_lengths=None, k_lengths=None, scale=None)

Tensors are fp32, bf16 or fp16 on a CUDA device; every step of the operators runs
in libsdtw.so's kernels, on the current stream of the tensors' device.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib


def _check_cuda(t: torch.Tensor, name: str, dtype=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is None:
        if t.dtype not in _lib.DTYPES:
            raise TypeError(f"{name} must be float32, bfloat16 or float16")
    elif t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, like the tensor it goes with")


def _grad_wanted(*tensors) -> bool:
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


# The wrappers of _lib check every tensor of a call again. Here the tensors are checked or made
# on the way, and a call from autograd's own thread pays two or three times for every line of
# Python, so the entry points are called with plain addresses.

def _call(name: str, device: torch.device, *args):
    """One entry point of the library on the device's current stream."""
    fn = getattr(_lib.quick(), name)
    if torch.cuda.current_device() == device.index:
        code = fn(*args, torch._C._cuda_getCurrentRawStream(device.index))
    else:
        with torch.cuda.device(device):
            code = fn(*args, torch._C._cuda_getCurrentRawStream(device.index))
    if code:
        raise _lib.SdtwError(code, name)


def _at(t):
    return None if t is None else t.data_ptr()


def _new(t: torch.Tensor) -> torch.Tensor:
    """An uninitialised contiguous tensor of t's shape, type and device."""
    return torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _workspace(n: int, device):
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


# --- layer norm ------------------------------------------------------------------------

def _norm_forward(x, weight, bias, eps, keep):
    y = torch.empty_like(x)
    rows, C = x.numel() // x.shape[-1], x.shape[-1]
    stats = torch.empty((2, rows), dtype=torch.float32, device=x.device) if keep else None
    if rows:
        w = weight if weight is not None else bias
        at = None if stats is None else stats.data_ptr()
        _call("sdtw_layernorm_forward", x.device, x.data_ptr(), _at(weight), _at(bias), rows, C, eps,
              _lib.DTYPES[x.dtype], 0 if w is None else _lib.DTYPES[w.dtype], y.data_ptr(), at,
              None if at is None else at + 4 * rows)
    return y, stats


class _LayerNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, stats = _norm_forward(x, weight, bias, eps, True)
        ctx.save_for_backward(x, weight, bias, stats)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, bias, stats = ctx.saved_tensors
        need_x, need_w, need_b, _ = ctx.needs_input_grad
        rows, C = x.numel() // x.shape[-1], x.shape[-1]
        dx, dw, db = _new(x) if need_x else None, _new(weight) if need_w else None, _new(bias) if need_b else None
        if rows == 0:
            return dx, None if dw is None else dw.zero_(), None if db is None else db.zero_(), None
        n = _lib.quick().sdtw_layernorm_workspace_bytes(rows, C) if need_w or need_b else 0
        ws = _workspace(n, x.device)
        w = weight if weight is not None else bias
        at = stats.data_ptr()
        dy = dy.contiguous()
        _call("sdtw_layernorm_backward", x.device, dy.data_ptr(), x.data_ptr(), _at(weight), at, at + 4 * rows, rows, C,
              _lib.DTYPES[x.dtype], 0 if w is None else _lib.DTYPES[w.dtype], _at(dx), _at(dw), _at(db), _at(ws), n)
        return dx, dw, db, None


def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
               eps: float = 1e-5) -> torch.Tensor:
    """(x - mean) / sqrt(var + eps) * weight + bias over the last dimension of x (..., C),
    differentiable in x, weight and bias. weight and bias (C,) are of x's type or fp32, both
    alike; the statistics and the sums of the weights' gradients are formed in fp32."""
    _check_cuda(x, "x")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must have a last dimension of at least 1")
    if not (eps >= 0 and math.isfinite(eps)):
        raise ValueError("eps must be finite and >= 0")
    for name, t in (("weight", weight), ("bias", bias)):
        if t is None:
            continue
        _check_cuda(t, name)
        if t.shape != x.shape[-1:]:
            raise ValueError(f"{name} must be ({x.shape[-1]},)")
        if t.dtype not in (x.dtype, torch.float32):
            raise TypeError(f"{name} must be float32 or of x's type")
        if t.device != x.device:
            raise ValueError(f"{name} must be on x's device")
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise TypeError("weight and bias must be of one type")
    x = x.contiguous()
    weight = None if weight is None else weight.contiguous()
    bias = None if bias is None else bias.contiguous()
    if _grad_wanted(x, weight, bias):
        return _LayerNormFn.apply(x, weight, bias, float(eps))
    return _norm_forward(x, weight, bias, float(eps), False)[0]


# --- rotary positions ------------------------------------------------------------------

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
    if not (base > 1 and factor >= 1):
        raise ValueError("base must be > 1 and factor >= 1")
    pair = torch.arange(dim // 2, dtype=torch.float64, device=device or "cuda")
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
        # the pair that turns `turns` times over the original length
        at = lambda turns: dim * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        first, last = max(0, math.floor(at(beta_fast))), min(dim // 2 - 1, math.ceil(at(beta_slow)))
        slow = ((pair - first) / max(last - first, 1e-3)).clamp(0, 1)
        freq = freq * (1 - slow) + freq / factor * slow
        magnitude = 0.1 * math.log(factor) + 1.0
    angle = torch.arange(length, dtype=torch.float64, device=pair.device)[:, None] * freq
    return (torch.stack([angle.cos(), angle.sin()], dim=-1) * magnitude).to(torch.float32)


def _features_contiguous(t: torch.Tensor) -> torch.Tensor:
    return t if t.stride(3) == 1 or t.shape[3] == 1 else t.contiguous()


def _strides(t):
    return (ctypes.c_longlong * 3)(*t.stride()[:3])


def _rotate(q, k, table, positions, interleaved, inverse):
    q = _features_contiguous(q)
    qo, ko = _new(q), None
    if k is not None:
        k = _features_contiguous(k)
        ko = _new(k)
    if q.numel():
        B, N, Hq, D = q.shape
        _call("sdtw_rotary", q.device, q.data_ptr(), _strides(q), _at(k), None if k is None else _strides(k), B, N, Hq,
              0 if k is None else k.shape[2], D, 2 * table.shape[1], table.data_ptr(), table.shape[0], _at(positions),
              N if positions is not None and positions.dim() == 2 else 0, interleaved, inverse, _lib.DTYPES[q.dtype],
              qo.data_ptr(), _at(ko))
    return qo, ko


class _RotaryFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, table, positions, interleaved):
        ctx.save_for_backward(table, positions)
        ctx.interleaved = interleaved
        qo, ko = _rotate(q, k, table, positions, interleaved, False)
        return qo if k is None else (qo, ko)

    @staticmethod
    def backward(ctx, dq, dk=None):
        table, positions = ctx.saved_tensors
        gq, gk = _rotate(dq, dk, table, positions, ctx.interleaved, True)
        return gq, gk, None, None, None


def rotary(q: torch.Tensor, k: torch.Tensor | None = None, *, table: torch.Tensor,
           positions: torch.Tensor | None = None, interleaved: bool = False):
    """q (B, N, Hq, D) and, where given, k (B, N, Hkv, D) with the first 2 * table.shape[1]
    features of every head turned by their position's angles, differentiable in q and k. Returns the
    turned q, or (q, k). Pairs are neighbouring features (interleaved) or (i, i + R/2). positions (B, N) or
    (N,) integers index the table; None stands for 0 .. N-1. A position outside the table gives NaN."""
    _check_cuda(q, "q")
    if q.dim() != 4:
        raise ValueError("q must be (B, N, H, D)")
    if k is not None:
        _check_cuda(k, "k", q.dtype)
        if k.dim() != 4 or k.shape[:2] != q.shape[:2] or k.shape[3] != q.shape[3] or k.device != q.device:
            raise ValueError("k must be (B, N, H, D) with q's batch, positions and features, on q's device")
    if (not isinstance(table, torch.Tensor) or table.dim() != 3 or table.shape[2] != 2
            or table.dtype != torch.float32 or table.device != q.device):
        raise ValueError("table must be a (length, R / 2, 2) float32 tensor on q's device, as rotary_table gives")
    if not 2 <= 2 * table.shape[1] <= q.shape[3]:
        raise ValueError("the table turns more features than a head has, or none")
    B, N = q.shape[:2]
    if positions is None:
        if N > table.shape[0]:
            raise ValueError("the table has fewer positions than q")
    else:
        if positions.is_floating_point() or positions.shape not in ((B, N), (N,)):
            raise ValueError("positions must be (B, N) or (N,) integers")
        positions = positions.to(device=q.device, dtype=torch.int32).contiguous()
    table = table.detach().contiguous()
    if _grad_wanted(q, k):
        return _RotaryFn.apply(q, k, table, positions, bool(interleaved))
    qo, ko = _rotate(q, k, table, positions, bool(interleaved), False)
    return qo if k is None else (qo, ko)


# --- attention -------------------------------------------------------------------------

def _problem(q, k, v, scale, left, right, q_lengths, k_lengths):
    (B, N, Hq, D), (M, Hkv) = q.shape, k.shape[1:3]
    return _lib.Attention(q.data_ptr(), k.data_ptr(), v.data_ptr(), q.stride()[:3], k.stride()[:3], v.stride()[:3],
                          _at(q_lengths), _at(k_lengths), B, N, M, Hq, Hkv, D, _lib.DTYPES[q.dtype], left, right, scale)


def _attend(q, k, v, scale, left, right, q_lengths, k_lengths, keep, want_lse):
    """(out, what its rounding left, lse): the last two for the backward pass, where kept."""
    B, N, Hq, D = q.shape
    out = torch.empty((B, N, Hq, D), dtype=q.dtype, device=q.device)
    rest = torch.empty_like(out) if keep and q.dtype != torch.float32 else None
    lse = torch.empty((B, Hq, N), dtype=torch.float32, device=q.device) if keep or want_lse else None
    if out.numel() == 0 or k.numel() == 0:
        out.zero_()
        return out, rest, None if lse is None else lse.fill_(-math.inf)
    problem = ctypes.byref(_problem(q, k, v, scale, left, right, q_lengths, k_lengths))
    n = _lib.quick().sdtw_attention_workspace_bytes(problem, 0)
    ws = _workspace(n, q.device)
    _call("sdtw_attention_forward", q.device, problem, out.data_ptr(), _at(rest), _at(lse), _at(ws), n)
    return out, rest, lse


class _AttentionFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, scale, left, right, q_lengths, k_lengths):
        out, rest, lse = _attend(q, k, v, scale, left, right, q_lengths, k_lengths, True, True)
        ctx.save_for_backward(q, k, v, out, rest, lse, q_lengths, k_lengths)
        ctx.rest = scale, left, right
        ctx.mark_non_differentiable(lse)
        return out, lse

    @staticmethod
    def backward(ctx, dout, _):
        q, k, v, out, rest, lse, q_lengths, k_lengths = ctx.saved_tensors
        scale, left, right = ctx.rest
        need_q, need_k, need_v = ctx.needs_input_grad[:3]
        dq = _new(q) if need_q else None
        dk, dv = (_new(k), _new(v)) if need_k or need_v else (None, None)
        if q.numel() == 0 or k.numel() == 0:
            return *(None if t is None else t.zero_() for t in (dq, dk, dv)), None, None, None, None, None
        problem = ctypes.byref(_problem(q, k, v, scale, left, right, q_lengths, k_lengths))
        n = _lib.quick().sdtw_attention_workspace_bytes(problem, 1)
        ws = _workspace(n, q.device)
        dout = dout.contiguous()
        _call("sdtw_attention_backward", q.device, problem, out.data_ptr(), _at(rest), lse.data_ptr(), dout.data_ptr(),
              _at(dq), _at(dk), _at(dv), _at(ws), n)
        return dq, dk if need_k else None, dv if need_v else None, None, None, None, None, None


def _lengths(t, B, device, name):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.is_floating_point() or t.shape != (B,):
        raise ValueError(f"{name} must be a (B,) integer tensor")
    return t.to(device=device, dtype=torch.int32).contiguous()


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, causal: bool = False, window: int | None = None,
              q_lengths: torch.Tensor | None = None, k_lengths: torch.Tensor | None = None,
              scale: float | None = None, return_lse: bool = False):
    """softmax(scale q k^T) v over the visible keys, (B, N, Hq, D), differentiable in q, k and v.

    q is (B, N, Hq, D), k and v are (B, M, Hkv, D) with Hq a multiple of Hkv: query head h reads key
    head h // (Hq // Hkv). D is at most 128; scale defaults to 1 / sqrt(D). Any strides do where features
    are contiguous (slices of one projection, a cache longer than what is filled of it).

    q_lengths and k_lengths (B,) make a padded batch: element b has n_b rows and m_b keys, and what lies
    beyond them is not used. Row n stands at key n + (m_b - n_b), so the newest row stands at the newest
    key: causal hides the keys after a row's own, window=w the keys w or more away from it. Rows without a
    visible key, and rows from n_b on, are 0 and pass no gradient.

    N = 1 over a cache of M keys is the step of a growing series; the key axis is then split over the SMs.
    return_lse gives (out, lse): the logarithm (B, Hq, N) of each row's sum of exp(score), fp32, not
    differentiable, -inf for rows that see nothing."""
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check_cuda(t, name, None if t is q else q.dtype)
        if t.dim() != 4 or t.device != q.device:
            raise ValueError(f"{name} must be (B, L, H, D), on q's device")
    B, N, Hq, D = q.shape
    if k.shape != v.shape or k.shape[0] != B or k.shape[3] != D:
        raise ValueError("k and v must both be (B, M, Hkv, D) with q's batch and features")
    if D < 1 or D > 128:
        raise ValueError("the head size must be 1 to 128")
    Hkv = k.shape[2]
    if Hkv < 1 or Hq < 1 or Hq % Hkv:
        raise ValueError("the query heads must be a multiple of the key heads")
    if window is not None and window < 1:
        raise ValueError("window must be >= 1")
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    if not (scale > 0 and math.isfinite(scale)):
        raise ValueError("scale must be finite and > 0")
    left = -1 if window is None else min(int(window) - 1, 2**31 - 2)
    right = 0 if causal else left
    q_lengths = _lengths(q_lengths, B, q.device, "q_lengths")
    k_lengths = _lengths(k_lengths, B, q.device, "k_lengths")
    q, k, v = _features_contiguous(q), _features_contiguous(k), _features_contiguous(v)
    if _grad_wanted(q, k, v):
        out, lse = _AttentionFn.apply(q, k, v, scale, left, right, q_lengths, k_lengths)
    else:
        out, _, lse = _attend(q, k, v, scale, left, right, q_lengths, k_lengths, False, return_lse)
    return (out, lse) if return_lse else out
