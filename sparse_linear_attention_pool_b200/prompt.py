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


class PromptPlan:
    """The work lists of a batch of sequences (see prompt_plan): host bytes and their device copy."""

    def __init__(self, host, device_bytes, lens_q, lens_k, Hq, Hkv, d, causal, grad):
        self.host, self.device_bytes = host, device_bytes
        self.lens_q, self.lens_k = tuple(lens_q), tuple(lens_k)
        self.Hq, self.Hkv, self.d, self.causal, self.grad = Hq, Hkv, d, causal, grad
        self.Tq, self.Tk = sum(self.lens_q), sum(self.lens_k)
        self.device = device_bytes.device
        self._at = (ctypes.addressof(host), ctypes.sizeof(host), device_bytes.data_ptr())
        from . import load

        self._workspace = load().sla_prompt_workspace_size(host)
        self._backward_workspace = load().sla_prompt_backward_workspace_size(host)

    def positions(self):
        """int32 [Tq] on the device: each query token's position in its sequence (for rope())."""
        import torch

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
    import torch

    from . import PromptParams, SLAError, load

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


def _rows(x, T: int, H: int, d: int, what: str):
    """x as the kernels take it: rows of whole 16-byte pieces at 16-byte steps (copied where it is not)."""
    import torch

    if x.dtype != torch.bfloat16 or not x.is_cuda:
        raise ValueError(f"{what}: a bfloat16 CUDA tensor")
    if x.dim() != 3 or x.shape[1] != H or x.shape[2] != d or x.shape[0] < T:
        raise ValueError(f"{what}: [>= {T}, {H}, {d}] for this plan, not {tuple(x.shape)}")
    row, head, one = x.stride()
    if one != 1 or (T > 1 and (row <= 0 or row % 8)) or (H > 1 and (head <= 0 or head % 8)) or x.data_ptr() % 16:
        x = x.contiguous()
    return x


def _struct(x):
    from . import Rows

    return Rows(x.data_ptr(), x.stride(0), x.stride(1))


def _same_device(plan, *tensors):
    for t in tensors:
        if t.device != plan.device:
            raise ValueError("the plan and the tensors are on different devices")


def _out(x, out, T, H, d, what):
    import torch

    if out is None:
        return torch.empty((x.shape[0], H, d), dtype=x.dtype, device=x.device)
    if out.dtype != x.dtype or out.device != x.device or out.dim() != 3 or out.shape[0] < T or \
            out.shape[1] != H or out.shape[2] != d or out.stride(2) != 1:
        raise ValueError(f"{what}: a [>= {T}, {H}, {d}] {x.dtype} tensor with contiguous rows")
    return out


def prompt_forward(q, k, v, plan: PromptPlan, *, out=None, want_lse: bool = True, workspace=None, stream=None):
    """(O, lse): sla_prompt_forward. O [rows of q, Hq, d]; lse [Tq, Hq] float32 or None.
    Rows of O behind the plan's last token are not written."""
    import torch

    from . import _check, load
    from .rope import _on

    on = _on(q, stream)
    if on is not None:
        with on:
            return prompt_forward(q, k, v, plan, out=out, want_lse=want_lse, workspace=workspace)
    q, k, v = (_rows(q, plan.Tq, plan.Hq, plan.d, "q"), _rows(k, plan.Tk, plan.Hkv, plan.d, "k"),
               _rows(v, plan.Tk, plan.Hkv, plan.d, "v"))
    _same_device(plan, q, k, v)
    out = _out(q, out, plan.Tq, plan.Hq, plan.d, "out")
    lse = torch.empty((plan.Tq, plan.Hq), dtype=torch.float32, device=q.device) if want_lse else None
    if workspace is None and plan._workspace:
        workspace = torch.empty(plan._workspace, dtype=torch.uint8, device=q.device)
    host, size, dev = plan._at
    _check(load().sla_prompt_forward(
        _struct(q), _struct(k), _struct(v), _struct(out), None if lse is None else lse.data_ptr(), host, size, dev,
        None if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.numel(),
        torch.cuda.current_stream().cuda_stream), "sla_prompt_forward")
    return out, lse


def prompt_backward(q, k, v, o, lse, do, plan: PromptPlan, *, out=None, workspace=None, stream=None):
    """(dq, dk, dv): sla_prompt_backward for the upstream do of a prompt_forward's o and lse.
    out: a triple of tensors to write to. Gradient rows behind the plan's last token are
    zero, or with `out` as they were."""
    import torch

    from . import _check, load
    from .rope import _on

    on = _on(q, stream)
    if on is not None:
        with on:
            return prompt_backward(q, k, v, o, lse, do, plan, out=out, workspace=workspace)
    if not plan.grad:
        raise ValueError("the plan was made without the backward pass (grad=True)")
    Tq, Tk, Hq, Hkv, d = plan.Tq, plan.Tk, plan.Hq, plan.Hkv, plan.d
    rows = (q.shape[0], k.shape[0])
    q, k, v = _rows(q, Tq, Hq, d, "q"), _rows(k, Tk, Hkv, d, "k"), _rows(v, Tk, Hkv, d, "v")
    o, do = _rows(o, Tq, Hq, d, "o"), _rows(do, Tq, Hq, d, "do")
    _same_device(plan, q, k, v, o, do, lse)
    if lse.dtype != torch.float32 or tuple(lse.shape) != (Tq, Hq) or not lse.is_contiguous():
        raise ValueError(f"lse: prompt_forward's [{Tq}, {Hq}] float32")
    dq, dk, dv = (None, None, None) if out is None else out
    fresh = out is None
    dq, dk, dv = _out(q, dq, Tq, Hq, d, "dq"), _out(k, dk, Tk, Hkv, d, "dk"), _out(v, dv, Tk, Hkv, d, "dv")
    if workspace is None:
        workspace = torch.empty(plan._backward_workspace, dtype=torch.uint8, device=q.device)
    host, size, dev = plan._at
    _check(load().sla_prompt_backward(
        _struct(q), _struct(k), _struct(v), _struct(o), lse.data_ptr(), _struct(do), _struct(dq), _struct(dk),
        _struct(dv), host, size, dev, workspace.data_ptr(), workspace.numel(),
        torch.cuda.current_stream().cuda_stream), "sla_prompt_backward")
    if fresh:
        for t, n in ((dq, Tq), (dk, Tk), (dv, Tk)):
            if t.shape[0] > n:
                t[n:].zero_()
    return dq, dk, dv


_function = None


def _prompt_function():
    """The autograd function (made at the first use: the package imports torch late)."""
    global _function
    if _function is not None:
        return _function
    import torch

    class PromptAttention(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, plan):
            o, lse = prompt_forward(q, k, v, plan)
            ctx.plan = plan
            ctx.save_for_backward(q, k, v, o, lse)
            return o

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, do):
            return (*prompt_backward(*ctx.saved_tensors, do, ctx.plan), None)

    _function = PromptAttention
    return _function


def prompt_attention(q, k, v, plan: PromptPlan, *, stream=None):
    """O = softmax(scale Q K^T + mask) V for the plan's packed sequences, [rows of q, Hq, d].
    Differentiable in q, k and v (with a plan made for it)."""
    import torch

    from .rope import _on

    on = _on(q, stream)
    if on is not None:
        with on:
            return prompt_attention(q, k, v, plan)
    if torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad):
        if not plan.grad:
            raise ValueError("the plan was made without the backward pass (grad=True)")
        return _prompt_function().apply(q, k, v, plan)
    return prompt_forward(q, k, v, plan, want_lse=False)[0]
