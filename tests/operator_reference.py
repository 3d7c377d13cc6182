"""Float64 references of the operators beside the attention (rotary positions,
query / key norms, packed prompt attention), written from their definitions, with
the magnitudes that the tests' error bounds are made of. CPU torch only."""

import math

import torch

EPS32 = 2.0 ** -24  # half a float32 step, relative


def half_step(dtype):
    """Half a rounding step relative to the value (bf16 2^-8, fp16 2^-11, fp32 2^-24)."""
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half a step among the subnormals."""
    return torch.finfo(dtype).smallest_normal * half_step(dtype)


def pair_indices(rot, layout):
    i = torch.arange(rot // 2)
    return (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)


def angles(freqs, axis, pos):
    """pos [T] or [A, T] -> [T, pairs] float64."""
    f = torch.tensor(freqs, dtype=torch.float64)
    p = pos.double()
    if p.dim() == 1:
        return p[:, None] * f
    return p[torch.tensor(axis, dtype=torch.long)].t() * f


def rotate(x, ang, rot, layout, gain=1.0, sign=1.0):
    """x [..., T, d] float64, ang [T, rot / 2]."""
    a, b = pair_indices(rot, layout)
    c, s = torch.cos(ang) * gain, torch.sin(ang) * gain * sign
    y = x.clone()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def rotate_size(x, rot, layout, gain=1.0):
    """|u| + |v| of each value's pair: what the errors of a rotation are relative to."""
    a, b = pair_indices(rot, layout)
    y = x.abs().clone()
    both = (x[..., a].abs() + x[..., b].abs()) * abs(gain)
    y[..., a], y[..., b] = both, both
    return y


def rms_norm(x, w, eps):
    r = 1.0 / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps)
    return x * r * w, r


def norm_rope_grads(x, w, eps, dy, ang, rot, layout, gain):
    """(dx, dw, size of dx's terms, size of dw's terms); x, dy [..., T, d]."""
    _, r = rms_norm(x, w, eps)
    xh = x * r
    g = rotate(dy, ang, rot, layout, gain, -1.0)
    gs = rotate_size(dy, rot, layout, gain)
    gw = g * w
    dx = r * (gw - xh * (gw * xh).mean(-1, keepdim=True))
    over = tuple(range(x.dim() - 1))
    size_x = r * (gs * w.abs() + xh.abs() * (gs * w.abs() * xh.abs()).mean(-1, keepdim=True))
    return dx, (g * xh).sum(over), size_x, (gs * xh.abs()).sum(over)


def prompt(q, k, v, lens_q, lens_k, causal, scale=None, do=None):
    """Packed attention in float64: q [Tq, Hq, d], k, v [Tk, Hkv, d]. Returns a dict
    with o, lse and, for an upstream do, dq, dk, dv, beside what the error bounds need."""
    d, grp = q.shape[-1], q.shape[1] // k.shape[1]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    q, k, v = q.double(), k.double(), v.double()
    out = dict(o=torch.zeros_like(q), lse=torch.full(q.shape[:2], -math.inf, dtype=torch.float64),
               o_size=torch.zeros_like(q))
    if do is not None:
        do = do.double()
        for n, t in (("dq", q), ("dk", k), ("dv", v)):
            out[n], out[n + "_size"] = torch.zeros_like(t), torch.zeros_like(t)
    a = b = 0
    for lq, lk in zip(lens_q, lens_k):
        for h in range(q.shape[1]):
            if lq == 0 or lk == 0:
                continue
            qs, ks, vs = q[a:a + lq, h], k[b:b + lk, h // grp], v[b:b + lk, h // grp]
            see = torch.ones(lq, lk, dtype=torch.bool)
            if causal:
                see = torch.arange(lk)[None] <= torch.arange(lq)[:, None] + (lk - lq)
            s = (qs @ ks.t() * scale).masked_fill(~see, -math.inf)
            lse = torch.logsumexp(s, -1)
            p = torch.exp(s - lse.masked_fill(lse == -math.inf, 0.0)[:, None])
            o = p @ vs
            out["o"][a:a + lq, h], out["lse"][a:a + lq, h] = o, lse
            out["o_size"][a:a + lq, h] = p @ vs.abs()
            if do is not None:
                g = do[a:a + lq, h]
                dp = g @ vs.t()
                ds = p * (dp - (g * o).sum(-1, keepdim=True))
                # sizes of the terms that the kernels round: |P dP| + |P D|
                dsz = p * (g.abs() @ vs.abs().t() + (g.abs() * o.abs()).sum(-1, keepdim=True))
                out["dq"][a:a + lq, h] = ds @ ks * scale
                out["dq_size"][a:a + lq, h] = dsz @ ks.abs() * scale
                out["dk"][b:b + lk, h // grp] += ds.t() @ qs * scale
                out["dk_size"][b:b + lk, h // grp] += dsz.t() @ qs.abs() * scale
                out["dv"][b:b + lk, h // grp] += p.t() @ g
                out["dv_size"][b:b + lk, h // grp] += p.t() @ g.abs()
        a, b = a + lq, b + lk
    return out
