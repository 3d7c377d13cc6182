"""Exact attention over packed prompts: the binding of sla_prompt_*.

    plan = sla.prompt_plan([512, 77, 1], Hq=32, Hkv=8, d=128)     # lengths, on the host
    o = sla.prompt_attention(q, k, v, plan)                        # q [590, 32, 128], k, v [590, 8, 128]

    # a piece of a prompt, or single tokens, behind what a cache holds
    plan = sla.prompt_plan([1, 1], [4097, 300], Hq=32, Hkv=8, d=128)

Tensors are packed tokens [T, H, d], bfloat16, the sequences behind one another;
their rows may be strided (the heads of q, k and v side by side in a projection's
output). Query heads share key heads in groups. Causal unless causal=False: a
sequence's last query sits at its last key.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from . import SLA_ERR_INVALID_ARG, SLA_ERR_UNSUPPORTED, PromptParams, SLAError, load
from .rotary import _sla, on_stream


class PromptPlan:
    """The work lists of a batch of sequences (see prompt_plan): host bytes and their device copy."""

    def __init__(self, host, device_bytes, lens_q, lens_k, Hq, Hkv, d, causal, grad):
        self.host, self.device_bytes = host, device_bytes
        self.lens_q, self.lens_k = tuple(lens_q), tuple(lens_k)
        self.Hq, self.Hkv, self.d, self.causal, self.grad = Hq, Hkv, d, causal, grad
        self.Tq, self.Tk = sum(self.lens_q), sum(self.lens_k)
        self.device = device_bytes.device
        self._c = _sla.PromptPlan(host.raw, device_bytes, self.Tq, self.Tk, Hq, Hkv, d, grad)
        self.workspace_size = self._c.forward_workspace  # bytes of prompt_forward's scratch, 0: none
        self.backward_workspace_size = self._c.backward_workspace

    def positions(self):
        """int32 [Tq] on the device: each query token's position in its sequence (for rope())."""
        return torch.cat([torch.arange(lk - lq, lk, dtype=torch.int32) for lq, lk in zip(self.lens_q, self.lens_k)]
                         ).to(self.device)


def _lengths(lens, what):
    lens = [int(x) for x in lens]
    if not lens or min(lens) < 0 or max(lens) > 0x7fffffff:
        raise ValueError(f"{what}: one length >= 0 for each sequence")
    return lens


def prompt_plan(lens_q: Sequence[int], lens_k: Optional[Sequence[int]] = None, *, Hq: int, Hkv: int, d: int,
                causal: bool = True, softmax_scale: float = 0.0, grad: Optional[bool] = None, device="cuda") -> PromptPlan:
    """Plans the attention of sequences of lens_q query tokens over lens_k keys (default:
    the same lengths). Made once for a batch of lengths, and good for any number of calls (a
    model's layers; a decoding step, whose caches have grown, needs one of its own). Keep it as
    long as a captured graph that reads it.
    softmax_scale 0 selects 1 / sqrt(d). grad: whether the plan serves the backward pass too
    (default: for whole prompts, where lens_k is not given)."""
    lens_q = _lengths(lens_q, "lens_q")
    grad = lens_k is None if grad is None else bool(grad)
    lens_k = lens_q if lens_k is None else _lengths(lens_k, "lens_k")
    if len(lens_k) != len(lens_q):
        raise ValueError("lens_q and lens_k name different numbers of sequences")
    n = len(lens_q)
    Hq, Hkv, d = int(Hq), int(Hkv), int(d)
    # 32-bit fields of the struct, which cut what does not fit them
    if any(not -0x80000000 <= x <= 0x7fffffff for x in (Hq, Hkv, d, n)):
        raise SLAError(SLA_ERR_UNSUPPORTED, "sla_prompt_plan")
    if softmax_scale != 0.0 and abs(softmax_scale) < 1e-30:
        raise SLAError(SLA_ERR_INVALID_ARG, "sla_prompt_plan")
    aq, ak = (ctypes.c_int32 * n)(*lens_q), (ctypes.c_int32 * n)(*lens_k)
    p = PromptParams(n, ctypes.addressof(aq), ctypes.addressof(ak), Hq, Hkv, d, int(bool(causal)),
                     int(grad), float(softmax_scale))
    lib = load()
    st = lib.sla_prompt_validate(p)
    if st:
        raise SLAError(st, "sla_prompt_plan")
    words = (ctypes.c_longlong * (lib.sla_prompt_plan_size(p) // 8))()  # 8-byte aligned
    st = lib.sla_prompt_plan(p, words, ctypes.sizeof(words))
    if st:
        raise SLAError(st, "sla_prompt_plan")
    host = (ctypes.c_char * lib.sla_prompt_plan_used(words)).from_buffer(words)
    return PromptPlan(host, torch.frombuffer(host, dtype=torch.uint8).to(device, copy=True), lens_q, lens_k, Hq, Hkv, d,
                      bool(causal), grad)


def prompt_forward(q, k, v, plan: PromptPlan, *, out=None, want_lse: bool = True, want_rest: bool = False,
                   workspace=None, stream=None):
    """(O, lse), or (O, lse, rest) with want_rest: sla_prompt_forward. O [rows of q, Hq, d]; lse
    [Tq, Hq] float32 or None; rest [Tq, Hq, d], what O's rounding left off, which makes the
    backward's gradients a little more exact. Rows of O behind the plan's last token are not written."""
    args = (q, k, v, plan._c, out, want_lse, want_rest, workspace)
    if stream is not None:
        with on_stream(stream, q.device, *args):
            made = _sla.prompt_forward(*args)
    else:
        made = _sla.prompt_forward(*args)
    return made if want_rest else made[:2]


def prompt_backward(q, k, v, o, lse, do, plan: PromptPlan, *, rest=None, out=None, workspace=None, stream=None):
    """(dq, dk, dv): sla_prompt_backward for the upstream do of a prompt_forward's o, lse and
    (optionally) rest. out: a triple of tensors to write to. Gradient rows behind the plan's
    last token are zero, or with `out` as they were."""
    args = (q, k, v, o, lse, rest, do, plan._c, out, workspace)
    if stream is not None:
        with on_stream(stream, q.device, *args):
            return _sla.prompt_backward(*args)
    return _sla.prompt_backward(*args)


def prompt_attention(q, k, v, plan: PromptPlan, *, stream=None):
    """O = softmax(scale Q K^T + mask) V for the plan's packed sequences, [rows of q, Hq, d]; rows
    behind the plan's last token are not written.
    Differentiable in q, k and v (with a plan made for it), in reverse mode."""
    if stream is not None:
        with on_stream(stream, q.device, q, k, v):
            return _sla.prompt_attention(q, k, v, plan._c)
    return _sla.prompt_attention(q, k, v, plan._c)
