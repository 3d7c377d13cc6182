"""Rotary positions, and the norm of every query and key head with the rotation
in the same pass: the binding of sla_rope and sla_qk_norm_rope.

    table = sla.rope_table(128, layout="interleaved", sections=(22, 21, 21))  # time, height, width
    q, k = sla.qk_norm_rope(q, k, wq, wk, table, positions)   # positions [3, N]
    x = sla.rope(x, table, positions)

Tensors are head rows [B, H, N, d] in any memory order with contiguous rows (a
projection's [B, N, H, d] output goes in as x.transpose(1, 2)), or packed tokens
[T, H, d]; bfloat16, float16 or float32. Outputs are contiguous in the same
logical shape. Both calls are differentiable in the inputs and the weights, in reverse
mode (forward-mode dual tensors are refused).
"""
from __future__ import annotations

import math
from typing import Optional, Sequence

import torch

from . import binding

_sla = binding()

LAYOUTS = {"interleaved": 0, "half": 1}
SCALINGS = ("none", "linear", "ntk", "yarn")


class RopeTable:
    """What a rotation keeps between calls (see rope_table): the pairs' frequencies on the device."""

    def __init__(self, turns, axis, gain: float, rot_dim: int, layout: str, n_axes: int, freqs: tuple):
        self.turns, self.axis = turns, axis  # int64 (the bits of uint64) [rot_dim / 2]; uint8 or None
        self.gain, self.rot_dim, self.layout, self.n_axes = gain, rot_dim, layout, n_axes
        self.freqs = freqs  # radians per position, float64
        self.device = turns.device
        self._c = _sla.RopeTable(turns, axis, gain, rot_dim, LAYOUTS[layout], n_axes)


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
                linear ramp between, and cos and sin are scaled by 0.1 ln(factor) + 1 (by 1
                for a factor of at most 1).
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
            gain = 0.1 * math.log(factor) + 1.0 if factor > 1.0 else 1.0
        freqs += f
        axes += [a] * n
    return freqs, axes, gain


_PI = 314159265358979323846264338327950288419716939937510582097494459  # 10^62 pi


def _turns(f: float) -> int:
    """round(2^64 f / 2 pi) mod 2^64, as the int64 of the same bits: in whole numbers, for a float64
    quotient would be off by hundreds of units (and position p turns p times as far)."""
    num, den = f.as_integer_ratio()
    num, den = (num << 64) * 10 ** 62, 2 * _PI * den
    t = (2 * num + den) // (2 * den) % (1 << 64)
    return t - (1 << 64) if t >= 1 << 63 else t


def rope_table(rot_dim: int, *, layout: str = "interleaved", freqs: Optional[Sequence[float]] = None,
               gain: Optional[float] = None, device="cuda", **kw) -> RopeTable:
    """The table of a rotation of the first rot_dim values of each head row, built once (and kept
    as long as a captured graph that reads it).

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
    turns = [_turns(x) for x in made]
    n_axes = 1 + max(axes, default=0)
    n_axes = max(n_axes, len(kw["sections"]) if kw.get("sections") is not None else 1)
    axis = torch.tensor(axes, dtype=torch.uint8).to(device) if n_axes > 1 else None
    return RopeTable(torch.tensor(turns, dtype=torch.int64).to(device), axis, gain, rot_dim, layout, n_axes,
                     tuple(made))


def on_stream(stream, device, *used):
    """A context in which `stream` (a torch stream or an integer handle) is the current one. The
    memory of the tensors `used` is not handed out again before that stream is done with it."""
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    if stream.device != device:
        raise ValueError(f"stream: of {stream.device}, the tensors are on {device}")
    for t in used:
        if isinstance(t, (tuple, list)):
            on_stream(stream, device, *t)
        elif isinstance(t, torch.Tensor) and t.is_cuda:
            t.record_stream(stream)
    return torch.cuda.stream(stream)


def rope(x, table: RopeTable, positions=None, *, N: Optional[int] = None, rows: Optional[int] = None, out=None,
         inverse: bool = False, stream=None):
    """x with every head row rotated by its token's position (sla_rope).

    positions: int32 / int64, [N] or [B, N], with a leading axis for a table of several
    axes; None counts 0 .. N - 1 on every axis. Only the first N tokens (default: all) of
    a [B, H, n, d] tensor are taken; `rows` (>= N) is the length of the result, whose rows
    behind N are not written. out: a tensor to write to (x itself is allowed).
    inverse rotates back by the same angles."""
    if stream is not None:
        with on_stream(stream, x.device, x, positions, out):
            return _sla.rope(x, table._c, positions, N, rows, out, inverse)
    return _sla.rope(x, table._c, positions, N, rows, out, inverse)


def qk_norm_rope(q, k, wq, wk, table: Optional[RopeTable] = None, positions=None, *, eps: float = 1e-6,
                 N: Optional[int] = None, rows: Optional[int] = None, out=None, stream=None):
    """(rope(q / rms(q) * wq), rope(k / rms(k) * wk)) in one pass (sla_qk_norm_rope).

    The root mean square is taken over each head row, rms(x)^2 = mean(x^2) + eps;
    wq, wk: [d], of the tensors' dtype or float32. table None: the norm alone.
    q and k may have different numbers of heads. The other arguments are rope()'s;
    out: a pair of tensors."""
    t = None if table is None else table._c
    if stream is not None:
        with on_stream(stream, q.device, q, k, wq, wk, positions, out):
            return _sla.qk_norm_rope(q, k, wq, wk, t, positions, eps, N, rows, out)
    return _sla.qk_norm_rope(q, k, wq, wk, t, positions, eps, N, rows, out)


def qk_norm_rope_backward(q, k, wq, wk, dyq, dyk, table: Optional[RopeTable] = None, positions=None, *,
                          eps: float = 1e-6, N: Optional[int] = None, want_weight_grad: bool = True,
                          workspace=None, stream=None):
    """Gradients (dq, dk, dwq, dwk) of qk_norm_rope for the upstream dyq, dyk
    (sla_qk_norm_rope_backward); dwq, dwk of the weights' dtype, or None. Rows behind N
    of dq and dk are zero, those of dyq and dyk are not read."""
    t = None if table is None else table._c
    args = (q, k, wq, wk, dyq, dyk, t, positions, eps, N, want_weight_grad, workspace)
    if stream is not None:
        with on_stream(stream, q.device, *args):
            return _sla.qk_norm_rope_backward(*args)
    return _sla.qk_norm_rope_backward(*args)
