"""Rotary positions, and the norm of every query and key head with the rotation
in the same pass: the binding of sla_rope and sla_qk_norm_rope.

    table = sla.rope_table(128, layout="interleaved", sections=(22, 21, 21))  # time, height, width
    q, k = sla.qk_norm_rope(q, k, wq, wk, table, positions)   # positions [3, N]
    x = sla.rope(x, table, positions)

Tensors are head rows [B, H, N, d] in any memory order with contiguous rows (a
projection's [B, N, H, d] output goes in as x.transpose(1, 2)), or packed tokens
[T, H, d]; bfloat16, float16 or float32. Outputs are contiguous in the same
logical shape. Both calls are differentiable: in the inputs and the weights.
"""
from __future__ import annotations

import math
from typing import Optional, Sequence

import torch

from . import Heads, RopeSpec, _check, load

LAYOUTS = {"interleaved": 0, "half": 1}
SCALINGS = ("none", "linear", "ntk", "yarn")


class RopeTable:
    """What a rotation keeps between calls (see rope_table): the pairs' frequencies on the device."""

    def __init__(self, turns, axis, gain: float, rot_dim: int, layout: str, n_axes: int, freqs: tuple):
        self.turns, self.axis = turns, axis  # int64 (the bits of uint64) [rot_dim / 2]; uint8 or None
        self.gain, self.rot_dim, self.layout, self.n_axes = gain, rot_dim, layout, n_axes
        self.freqs = freqs  # radians per position, float64
        self.device = turns.device
        self._fixed = (turns.data_ptr(), None if axis is None else axis.data_ptr())
        self._tail = (float(gain), int(rot_dim), LAYOUTS[layout], int(n_axes))


def rope_frequencies(rot_dim: int, *, theta: float = 10000.0, sections: Optional[Sequence[int]] = None,
                     scaling: str = "none", factor: float = 1.0, original: int = 0, beta_fast: float = 32.0,
                     beta_slow: float = 1.0):
    """(radians per position of every pair, the pair's axis, gain), float64.

    An axis with n pairs has the frequencies theta^(-i/n), i = 0 .. n - 1; `sections`
    gives the pairs of each axis (default: one axis with all of them). Scalings for
    contexts `factor` times as long:
      "linear"  f / factor (positions interpolated);
      "ntk"     theta -> theta factor^(n / (n - 1)): the slowest pair is stretched by
                factor, the fastest keeps its frequency;
      "yarn"    pairs that turn more than beta_fast times over `original` positions keep
                their frequency, those below beta_slow turns are divided by factor, with a
                linear ramp between, and cos and sin are scaled by 0.1 ln(factor) + 1.
    """
    if rot_dim < 0 or rot_dim % 2:
        raise ValueError("rot_dim must be even and not negative")
    sections = [rot_dim // 2] if sections is None else [int(n) for n in sections]
    if any(n < 0 for n in sections) or 2 * sum(sections) != rot_dim or not 1 <= len(sections) <= 255:
        raise ValueError("sections must sum to rot_dim / 2")
    if scaling not in SCALINGS:
        raise ValueError(f"scaling must be one of {SCALINGS}")
    if not (theta > 0.0 and math.isfinite(theta)):
        raise ValueError("theta must be positive")
    if scaling != "none" and not (factor > 0.0 and math.isfinite(factor)):
        raise ValueError("factor must be positive")
    if scaling == "yarn" and (original < 1 or not beta_fast > beta_slow > 0.0 or theta <= 1.0):
        raise ValueError("yarn needs original >= 1, beta_fast > beta_slow > 0 and theta > 1")
    freqs, axes, gain = [], [], 1.0
    for a, n in enumerate(sections):
        base = theta * factor ** (n / (n - 1.0)) if scaling == "ntk" and n > 1 else theta
        f = [base ** (-i / n) for i in range(n)]
        if scaling == "linear":
            f = [x / factor for x in f]
        elif scaling == "yarn":
            def pair_of(turns):  # the (real-valued) pair that makes `turns` turns over the original length
                return n * math.log(original / (turns * 2.0 * math.pi)) / math.log(theta)

            lo, hi = max(0, math.floor(pair_of(beta_fast))), min(2 * n - 1, math.ceil(pair_of(beta_slow)))
            ramp = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(n)]
            f = [x * (1.0 - r) + x / factor * r for x, r in zip(f, ramp)]
            gain = 0.1 * math.log(factor) + 1.0
        freqs += f
        axes += [a] * n
    return freqs, axes, gain


def rope_table(rot_dim: int, *, layout: str = "interleaved", freqs: Optional[Sequence[float]] = None,
               gain: Optional[float] = None, device="cuda", **kw) -> RopeTable:
    """The table of a rotation of the first rot_dim values of each head row, built once.

    layout "interleaved": pair i is (x[2i], x[2i+1]); "half": (x[i], x[i + rot_dim/2]).
    The other arguments are rope_frequencies'; `freqs` (radians per position, rot_dim / 2
    numbers, in place of theta and the scaling) and `gain` set them directly."""
    if layout not in LAYOUTS:
        raise ValueError(f"layout must be one of {tuple(LAYOUTS)}")
    if freqs is not None:
        unknown = set(kw) - {"sections"}
        if unknown:
            raise ValueError(f"freqs replaces {sorted(unknown)}")
    made, axes, g = rope_frequencies(rot_dim, **kw)
    if freqs is not None:
        made = [float(x) for x in freqs]
        if len(made) != rot_dim // 2 or not all(math.isfinite(x) for x in made):
            raise ValueError("freqs must be rot_dim / 2 finite numbers")
    gain = g if gain is None else float(gain)
    if not math.isfinite(gain):
        raise ValueError("gain must be finite")
    turns = []
    for x in made:
        # 2^64 f / 2 pi: a float64 times a power of two, then reduced in whole numbers
        t = int(math.ldexp(math.fmod(x / (2.0 * math.pi), 1.0), 64)) % (1 << 64)
        turns.append(t - (1 << 64) if t >= 1 << 63 else t)
    n_axes = 1 + max(axes, default=0)
    n_axes = max(n_axes, len(kw["sections"]) if kw.get("sections") is not None else 1)
    axis = torch.tensor(axes, dtype=torch.uint8).to(device) if n_axes > 1 else None
    return RopeTable(torch.tensor(turns, dtype=torch.int64).to(device), axis, gain, rot_dim, layout, n_axes,
                     tuple(made))


_CODES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # the current stream's handle, without an object


def current_stream() -> int:
    """The current device's current stream as an integer handle."""
    if _raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(torch.cuda.current_device())


def _check_rows(x, like=None, what="x"):
    if x.dim() not in (3, 4):
        raise ValueError(f"{what}: [B, H, N, d] or [T, H, d], not {tuple(x.shape)}")
    if not x.is_cuda:
        raise ValueError(f"{what}: a CUDA tensor")
    if x.dtype not in _CODES:
        raise ValueError(f"{what}: bfloat16, float16 or float32, not {x.dtype}")
    if like is not None and (x.dim() != like.dim() or x.dtype != like.dtype or x.device != like.device
                             or x.shape[-1] != like.shape[-1]):
        raise ValueError(f"{what}: dtype, device, head size or rank differ")


def _rows(x):
    """x with contiguous rows."""
    return x if x.stride(-1) == 1 or x.shape[-1] == 1 else x.contiguous()


def _heads(x):
    if x.dim() == 4:
        sb, sh, sn, _ = x.stride()
        return Heads(x.data_ptr(), x.shape[1], sb, sh, sn)
    sn, sh, _ = x.stride()
    return Heads(x.data_ptr(), x.shape[1], 0, sh, sn)


def _tokens(x):
    return (x.shape[0], x.shape[2]) if x.dim() == 4 else (1, x.shape[0])


def _spec(table: Optional[RopeTable], positions, B: int, N: int, device):
    """The sla_rope_spec of a call, positions checked against B and N."""
    if table is None:
        if positions is not None:
            raise ValueError("positions without a table")
        return None
    if table.device != device:
        raise ValueError("the table is on another device")
    turns, axis = table._fixed
    gain, rot_dim, layout, n_axes = table._tail
    if positions is None:
        return RopeSpec(turns, axis, None, 0, 0, 0, gain, 32, rot_dim, layout, n_axes)
    bits = 32 if positions.dtype is torch.int32 else 64
    if (bits == 64 and positions.dtype is not torch.int64) or positions.device != device:
        raise ValueError("positions: int32 or int64 on the tensors' device")
    shape, stride, s_axis, s_b = positions.shape, positions.stride(), 0, 0
    if n_axes > 1:
        if len(shape) < 2 or shape[0] != n_axes:
            raise ValueError(f"positions: [{n_axes}, (B,) N] for {n_axes} axes")
        s_axis, shape, stride = stride[0], shape[1:], stride[1:]
    if len(shape) == 2 and shape[0] in (1, B):
        s_b = stride[0] if shape[0] > 1 else 0
    elif len(shape) != 1:
        shape = (-1,)
    if shape[-1] < N:
        raise ValueError(f"positions: one for each of {B} x {N} tokens, not {tuple(positions.shape)}")
    return RopeSpec(turns, axis, positions.data_ptr(), s_axis, s_b, stride[-1], gain, bits, rot_dim, layout, n_axes)


def _on(x, stream):
    """A context that makes x's device current and `stream` its current stream, or None."""
    if stream is not None:
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=x.device)
        return torch.cuda.stream(stream)
    if x.is_cuda and x.get_device() != torch.cuda.current_device():
        return torch.cuda.device(x.device)
    return None


def _out_for(x, out, rows: Optional[int], N: int, what="out"):
    if out is None:
        if rows is None:
            return torch.empty_like(x, memory_format=torch.contiguous_format)
        if x.dim() != 4:
            raise ValueError("rows is for [B, H, N, d] tensors")
        B, H, _, d = x.shape
        if int(rows) < N:
            raise ValueError("rows must be at least N")
        return x.new_empty((B, H, int(rows), d))
    _check_rows(out, x, what)
    if out.shape[1] != x.shape[1] or (out.dim() == 4 and out.shape[0] != x.shape[0]) or _tokens(out)[1] < N:
        raise ValueError(f"{what}: shape {tuple(out.shape)} does not take the result")
    if out.stride(-1) != 1 and out.shape[-1] != 1:
        raise ValueError(f"{what}: rows must be contiguous")
    return out


def _count(x, N):
    n = _tokens(x)[1]
    if N is None:
        return n
    if not 0 <= int(N) <= n:
        raise ValueError(f"N must be 0 .. {n}")
    return int(N)


def _run_rope(x, table, positions, N, out, inverse):
    B = x.shape[0] if x.dim() == 4 else 1
    spec = _spec(table, positions, B, N, x.device)
    if N and x.numel():
        _check(load().sla_rope(_heads(x), _heads(out), B, N, x.shape[-1], _CODES[x.dtype], spec, int(inverse),
                               current_stream()), "sla_rope")
    return out


def _zero_tail(t, N):
    """Rows behind N of a [B, H, rows, d] or [rows, H, d] gradient are zero."""
    if _tokens(t)[1] > N:
        (t[:, :, N:] if t.dim() == 4 else t[N:]).zero_()
    return t


class _Rope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, table, positions, N, rows, inverse):
        ctx.save_for_backward(positions)
        ctx.meta = (table, N, inverse, x.shape)
        x = _rows(x)
        return _run_rope(x, table, positions, N, _out_for(x, None, rows, N), inverse)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        table, N, inverse, shape = ctx.meta
        (positions,) = ctx.saved_tensors
        dx = torch.empty(shape, dtype=dy.dtype, device=dy.device)
        _run_rope(_rows(dy), table, positions, N, dx, not inverse)
        return _zero_tail(dx, N), None, None, None, None, None


class _QKNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, wq, wk, table, positions, eps, N, rows):
        ctx.meta = (table, eps, N)
        ctx.save_for_backward(q, k, wq, wk, positions)
        q, k = _rows(q), _rows(k)
        return _run_norm(q, k, wq, wk, table, positions, eps, N, _out_for(q, None, rows, N),
                         _out_for(k, None, rows, N))

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dyq, dyk):
        q, k, wq, wk, positions = ctx.saved_tensors
        table, eps, N = ctx.meta
        need_w = ctx.needs_input_grad[2] or ctx.needs_input_grad[3]
        return (*_run_norm_backward(q, k, wq, wk, dyq, dyk, table, positions, eps, N, need_w, None),
                None, None, None, None, None)


def rope(x, table: RopeTable, positions=None, *, N: Optional[int] = None, rows: Optional[int] = None, out=None,
         inverse: bool = False, stream=None):
    """x with every head row rotated by its token's position (sla_rope).

    positions: int32 / int64, [N] or [B, N], with a leading axis for a table of several
    axes; None counts 0 .. N - 1 on every axis. Only the first N tokens (default: all) of
    a [B, H, n, d] tensor are taken; `rows` (>= N) is the length of the result, whose rows
    behind N are not written. out: a tensor to write to (x itself is allowed).
    inverse rotates back by the same angles."""
    on = _on(x, stream)
    if on is not None:
        with on:
            return rope(x, table, positions, N=N, rows=rows, out=out, inverse=inverse)
    _check_rows(x)
    N = _count(x, N)
    if torch.is_grad_enabled() and x.requires_grad:
        if out is not None:
            raise ValueError("out cannot be given for a tensor that requires grad")
        return _Rope.apply(x, table, positions, N, rows, inverse)
    x = _rows(x)
    return _run_rope(x, table, positions, N, _out_for(x, out, rows, N), inverse)


def _check_pair(q, k, wq, wk):
    _check_rows(q, what="q")
    _check_rows(k, q, "k")
    if _tokens(q) != _tokens(k):
        raise ValueError("q and k hold different tokens")
    for w, what in ((wq, "wq"), (wk, "wk")):
        if w.dim() != 1 or w.shape[0] != q.shape[-1] or w.device != q.device:
            raise ValueError(f"{what}: [d] on the tensors' device")
    if wq.dtype != wk.dtype or wq.dtype not in (q.dtype, torch.float32):
        raise ValueError("wq and wk: the tensors' dtype, or float32")


def _weight(w):
    return w if w.stride(0) == 1 or w.shape[0] == 1 else w.contiguous()


def _run_norm(q, k, wq, wk, table, positions, eps, N, yq, yk):
    B = _tokens(q)[0]
    spec = _spec(table, positions, B, N, q.device)
    if B and N:
        wq, wk = _weight(wq), _weight(wk)
        _check(load().sla_qk_norm_rope(_heads(q), _heads(k), wq.data_ptr(), wk.data_ptr(),
                                       int(wq.dtype == torch.float32), eps, _heads(yq), _heads(yk), B, N,
                                       q.shape[-1], _CODES[q.dtype], spec, current_stream()),
               "sla_qk_norm_rope")
    return yq, yk


def qk_norm_rope(q, k, wq, wk, table: Optional[RopeTable] = None, positions=None, *, eps: float = 1e-6,
                 N: Optional[int] = None, rows: Optional[int] = None, out=None, stream=None):
    """(rope(q / rms(q) * wq), rope(k / rms(k) * wk)) in one pass (sla_qk_norm_rope).

    The root mean square is taken over each head row, rms(x)^2 = mean(x^2) + eps;
    wq, wk: [d], of the tensors' dtype or float32. table None: the norm alone.
    q and k may have different numbers of heads. The other arguments are rope()'s;
    out: a pair of tensors."""
    on = _on(q, stream)
    if on is not None:
        with on:
            return qk_norm_rope(q, k, wq, wk, table, positions, eps=eps, N=N, rows=rows, out=out)
    _check_pair(q, k, wq, wk)
    N = _count(q, N)
    if torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or wq.requires_grad or wk.requires_grad):
        if out is not None:
            raise ValueError("out cannot be given for tensors that require grad")
        return _QKNormRope.apply(q, k, wq, wk, table, positions, float(eps), N, rows)
    q, k = _rows(q), _rows(k)
    yq, yk = (None, None) if out is None else out
    return _run_norm(q, k, wq, wk, table, positions, eps, N, _out_for(q, yq, rows, N),
                     _out_for(k, yk, rows, N, "out"))


def _run_norm_backward(q, k, wq, wk, dyq, dyk, table, positions, eps, N, need_w, workspace):
    B, d = _tokens(q)[0], q.shape[-1]
    dq, dk = (torch.empty_like(x, memory_format=torch.contiguous_format) for x in (q, k))
    dwq, dwk = (torch.empty_like(wq), torch.empty_like(wk)) if need_w else (None, None)
    spec = _spec(table, positions, B, N, q.device)
    if B and N:
        lib = load()
        if workspace is None:
            workspace = q.new_empty(lib.sla_qk_norm_rope_backward_workspace_size(B, N, q.shape[1], k.shape[1], d),
                                    dtype=torch.uint8)
        q, k, dyq, dyk, wq, wk = _rows(q), _rows(k), _rows(dyq), _rows(dyk), _weight(wq), _weight(wk)
        _check(lib.sla_qk_norm_rope_backward(
            _heads(q), _heads(k), wq.data_ptr(), wk.data_ptr(), int(wq.dtype == torch.float32), eps, _heads(dyq),
            _heads(dyk), _heads(dq), _heads(dk), dwq.data_ptr() if need_w else None,
            dwk.data_ptr() if need_w else None, B, N, d, _CODES[q.dtype], spec, workspace.data_ptr(),
            workspace.numel(), current_stream()), "sla_qk_norm_rope_backward")
    elif need_w:
        dwq.zero_()
        dwk.zero_()
    return _zero_tail(dq, N), _zero_tail(dk, N), dwq, dwk


def qk_norm_rope_backward(q, k, wq, wk, dyq, dyk, table: Optional[RopeTable] = None, positions=None, *,
                          eps: float = 1e-6, N: Optional[int] = None, want_weight_grad: bool = True,
                          workspace=None, stream=None):
    """Gradients (dq, dk, dwq, dwk) of qk_norm_rope for the upstream dyq, dyk
    (sla_qk_norm_rope_backward); dwq, dwk of the weights' dtype, or None. Rows behind N
    of dq and dk are zero, those of dyq and dyk are not read."""
    on = _on(q, stream)
    if on is not None:
        with on:
            return qk_norm_rope_backward(q, k, wq, wk, dyq, dyk, table, positions, eps=eps, N=N,
                                         want_weight_grad=want_weight_grad, workspace=workspace)
    _check_pair(q, k, wq, wk)
    N = _count(q, N)
    for g, x, what in ((dyq, q, "dyq"), (dyk, k, "dyk")):
        _check_rows(g, x, what)
        if g.shape[1] != x.shape[1] or _tokens(g)[0] != _tokens(x)[0] or _tokens(g)[1] < N:
            raise ValueError(f"{what}: shape {tuple(g.shape)}")
    return _run_norm_backward(q, k, wq, wk, dyq, dyk, table, positions, float(eps), N, want_weight_grad, workspace)
