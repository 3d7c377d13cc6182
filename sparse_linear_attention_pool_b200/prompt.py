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

from . import PromptParams, Rows, SLAError, _check, load
from .rotary import _on, current_stream


class PromptPlan:
    """The work lists of a batch of sequences (see prompt_plan): host bytes and their device copy."""

    def __init__(self, host, device_bytes, lens_q, lens_k, Hq, Hkv, d, causal, grad):
        self.host, self.device_bytes = host, device_bytes
        self.lens_q, self.lens_k = tuple(lens_q), tuple(lens_k)
        self.Hq, self.Hkv, self.d, self.causal, self.grad = Hq, Hkv, d, causal, grad
        self.Tq, self.Tk = sum(self.lens_q), sum(self.lens_k)
        self.device = device_bytes.device
        self._sizes = (self.Tq, self.Tk, Hq, Hkv, d)
        self._at = (ctypes.addressof(host), ctypes.sizeof(host), device_bytes.data_ptr())
        self._workspace = load().sla_prompt_workspace_size(host)
        self._backward_workspace = load().sla_prompt_backward_workspace_size(host)

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
    the same lengths). Made once for a batch of lengths, and good for any number of calls.
    softmax_scale 0 selects 1 / sqrt(d). grad: whether the plan serves the backward pass too
    (default: for whole prompts, where lens_k is not given)."""
    lens_q = _lengths(lens_q, "lens_q")
    grad = lens_k is None if grad is None else bool(grad)
    lens_k = lens_q if lens_k is None else _lengths(lens_k, "lens_k")
    if len(lens_k) != len(lens_q):
        raise ValueError("lens_q and lens_k name different numbers of sequences")
    n = len(lens_q)
    aq, ak = (ctypes.c_int32 * n)(*lens_q), (ctypes.c_int32 * n)(*lens_k)
    p = PromptParams(n, ctypes.addressof(aq), ctypes.addressof(ak), int(Hq), int(Hkv), int(d), int(bool(causal)),
                     int(grad), float(softmax_scale))
    lib = load()
    st = lib.sla_prompt_validate(p)
    if st:
        raise SLAError(st, "sla_prompt_plan")
    size = lib.sla_prompt_plan_size(p)
    host = ctypes.create_string_buffer(size + 8)
    at = (ctypes.addressof(host) + 7) // 8 * 8 - ctypes.addressof(host)
    host = (ctypes.c_char * size).from_buffer(host, at)  # 8-byte aligned
    st = lib.sla_prompt_plan(p, host, size)
    if st:
        raise SLAError(st, "sla_prompt_plan")
    return PromptPlan(host, torch.frombuffer(bytearray(host.raw), dtype=torch.uint8).to(device), lens_q, lens_k,
                      int(Hq), int(Hkv), int(d), bool(causal), grad)


def _rows(x, T: int, H: int, d: int, plan, what: str):
    """(x, its sla_rows): rows of whole 16-byte pieces at 16-byte steps, copied where x's are not."""
    if x.dtype is not torch.bfloat16 or not x.is_cuda:
        raise ValueError(f"{what}: a bfloat16 CUDA tensor")
    shape = x.shape
    if len(shape) != 3 or shape[0] < T or shape[1] != H or shape[2] != d:
        raise ValueError(f"{what}: [>= {T}, {H}, {d}] for this plan, not {tuple(shape)}")
    if x.device != plan.device:
        raise ValueError(f"{what}: on another device than the plan")
    row, head, one = x.stride()
    if one != 1 or (T > 1 and (row <= 0 or row % 8)) or (H > 1 and (head <= 0 or head % 8)) or x.data_ptr() % 16:
        x = x.contiguous()
        row, head, _ = x.stride()
    return x, Rows(x.data_ptr(), row, head)


def _out(x, out, T, H, d, what):
    """(out, its sla_rows): a new tensor like x, or the given one."""
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    elif out.dtype != x.dtype or out.device != x.device or out.dim() != 3 or out.shape[0] < T or \
            out.shape[1] != H or out.shape[2] != d or out.stride(2) != 1:
        raise ValueError(f"{what}: a [>= {T}, {H}, {d}] {x.dtype} tensor with contiguous rows")
    row, head, _ = out.stride()
    return out, Rows(out.data_ptr(), row, head)


def _forward(q, k, v, plan, out, want_lse, workspace):
    Tq, Tk, Hq, Hkv, d = plan._sizes
    q, q_rows = _rows(q, Tq, Hq, d, plan, "q")
    k, k_rows = _rows(k, Tk, Hkv, d, plan, "k")
    v, v_rows = _rows(v, Tk, Hkv, d, plan, "v")
    out, o_rows = _out(q, out, Tq, Hq, d, "out")
    lse = q.new_empty((Tq, Hq), dtype=torch.float32) if want_lse else None
    if workspace is None and plan._workspace:
        workspace = q.new_empty(plan._workspace, dtype=torch.uint8)
    host, size, dev = plan._at
    _check(load().sla_prompt_forward(
        q_rows, k_rows, v_rows, o_rows, None if lse is None else lse.data_ptr(), host, size, dev,
        None if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.numel(),
        current_stream()), "sla_prompt_forward")
    return out, lse


def prompt_forward(q, k, v, plan: PromptPlan, *, out=None, want_lse: bool = True, workspace=None, stream=None):
    """(O, lse): sla_prompt_forward. O [rows of q, Hq, d]; lse [Tq, Hq] float32 or None.
    Rows of O behind the plan's last token are not written."""
    on = _on(q, stream)
    if on is not None:
        with on:
            return _forward(q, k, v, plan, out, want_lse, workspace)
    return _forward(q, k, v, plan, out, want_lse, workspace)


def _backward(q, k, v, o, lse, do, plan, out, workspace):
    Tq, Tk, Hq, Hkv, d = plan._sizes
    q, q_rows = _rows(q, Tq, Hq, d, plan, "q")
    k, k_rows = _rows(k, Tk, Hkv, d, plan, "k")
    v, v_rows = _rows(v, Tk, Hkv, d, plan, "v")
    o, o_rows = _rows(o, Tq, Hq, d, plan, "o")
    do, do_rows = _rows(do, Tq, Hq, d, plan, "do")
    if lse.dtype is not torch.float32 or tuple(lse.shape) != (Tq, Hq) or not lse.is_contiguous() or \
            lse.device != plan.device:
        raise ValueError(f"lse: prompt_forward's [{Tq}, {Hq}] float32")
    dq, dk, dv = (None, None, None) if out is None else out
    dq, dq_rows = _out(q, dq, Tq, Hq, d, "dq")
    dk, dk_rows = _out(k, dk, Tk, Hkv, d, "dk")
    dv, dv_rows = _out(v, dv, Tk, Hkv, d, "dv")
    if workspace is None:
        workspace = q.new_empty(plan._backward_workspace, dtype=torch.uint8)
    host, size, dev = plan._at
    _check(load().sla_prompt_backward(
        q_rows, k_rows, v_rows, o_rows, lse.data_ptr(), do_rows, dq_rows, dk_rows, dv_rows, host, size, dev,
        workspace.data_ptr(), workspace.numel(), current_stream()), "sla_prompt_backward")
    if out is None:
        for t, n in ((dq, Tq), (dk, Tk), (dv, Tk)):
            if t.shape[0] > n:
                t[n:].zero_()
    return dq, dk, dv


def _needs_backward(plan):
    if not plan.grad:
        raise ValueError("the plan was made without the backward pass (grad=True)")


def prompt_backward(q, k, v, o, lse, do, plan: PromptPlan, *, out=None, workspace=None, stream=None):
    """(dq, dk, dv): sla_prompt_backward for the upstream do of a prompt_forward's o and lse.
    out: a triple of tensors to write to. Gradient rows behind the plan's last token are
    zero, or with `out` as they were."""
    _needs_backward(plan)
    on = _on(q, stream)
    if on is not None:
        with on:
            return _backward(q, k, v, o, lse, do, plan, out, workspace)
    return _backward(q, k, v, o, lse, do, plan, out, workspace)


class _PromptAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, plan):
        o, lse = _forward(q, k, v, plan, None, True, None)
        ctx.plan = plan
        ctx.save_for_backward(q, k, v, o, lse)
        return o

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, do):
        return (*_backward(*ctx.saved_tensors, do, ctx.plan, None, None), None)


def prompt_attention(q, k, v, plan: PromptPlan, *, stream=None):
    """O = softmax(scale Q K^T + mask) V for the plan's packed sequences, [rows of q, Hq, d].
    Differentiable in q, k and v (with a plan made for it)."""
    on = _on(q, stream)
    if on is not None:
        with on:
            return prompt_attention(q, k, v, plan)
    if torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad):
        _needs_backward(plan)
        return _PromptAttention.apply(q, k, v, plan)
    return _forward(q, k, v, plan, None, False, None)[0]
