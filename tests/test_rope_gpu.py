"""Rotary positions and query / key norms on the GPU against float64."""

import math

import pytest
import torch

from tests import operator_reference as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def make(shape, dt, seed, form):
    """Values of a [B, H, N, d] tensor ("heads": read from token-major memory; "packed": [N, H, d])."""
    g = torch.Generator().manual_seed(seed)
    B, H, N, d = shape
    x = torch.randn(B, N, H, d, generator=g).to(dt)
    return x[0] if form == "packed" else x.transpose(1, 2)


def to_bhnd(x):
    return x.transpose(0, 1).unsqueeze(0) if x.dim() == 3 else x


def rope_bound(ref, size, dt):
    """One rounding of the result; two float32 products and a sum (3 half-steps) of cos and
    sin off by 2 steps each, and an angle off by 2^-25 of 2 pi in float32: 4e-7 covers them."""
    return R.half_step(dt) * ref.abs() * 1.01 + 1e-6 * size + R.tiny(dt)


CASES = [
    # dt, form, B, H, N, d, rot, layout, axes, scaling
    ("bf16", "heads", 1, 3, 65, 128, 128, "interleaved", 1, "none"),
    ("bf16", "heads", 2, 2, 33, 64, 64, "half", 1, "linear"),
    ("bf16", "packed", 1, 5, 1, 128, 128, "half", 1, "none"),
    ("fp16", "packed", 1, 7, 130, 128, 64, "half", 1, "yarn"),
    ("fp32", "heads", 2, 3, 31, 128, 128, "interleaved", 3, "none"),
    ("bf16", "heads", 1, 4, 100, 128, 128, "interleaved", 3, "none"),
    ("fp32", "packed", 1, 2, 77, 80, 40, "half", 1, "ntk"),
    ("bf16", "packed", 1, 2, 77, 80, 40, "half", 1, "ntk"),
    ("bf16", "packed", 1, 1, 5, 256, 256, "half", 1, "none"),
    ("fp32", "packed", 1, 1, 5, 256, 256, "half", 1, "none"),
    ("fp16", "heads", 1, 2, 9, 256, 254, "interleaved", 1, "none"),
    ("bf16", "packed", 1, 3, 6, 10, 6, "half", 1, "none"),
    ("bf16", "packed", 1, 3, 6, 2, 2, "interleaved", 1, "none"),
    ("bf16", "packed", 1, 40, 300, 96, 96, "half", 1, "none"),
    ("bf16", "packed", 1, 2, 9, 128, 0, "half", 1, "none"),
]


def table_of(sla, rot, layout, axes, scaling):
    kw = {}
    if axes == 3:
        a = rot // 2 // 3
        kw["sections"] = (rot // 2 - 2 * a, a, a)
    if scaling != "none":
        kw.update(scaling=scaling, factor=3.5, original=512 if scaling == "yarn" else 0)
    return sla.rope_table(rot, layout=layout, **kw)


def positions_of(axes, B, N, seed, form):
    g = torch.Generator().manual_seed(seed)
    shape = ([axes] if axes > 1 else []) + ([B] if B > 1 else []) + [N]
    return torch.randint(-5, 1_000_000, shape, generator=g)


def reference_angles(table, pos, axes, B, N):
    """[B][N, pairs]"""
    from sparse_linear_attention_pool_b200.rotary import RopeTable  # noqa: F401

    axis = None if table.axis is None else table.axis.cpu().tolist()
    out = []
    for b in range(B):
        p = pos
        if B > 1:
            p = pos[:, b] if axes > 1 else pos[b]
        out.append(R.angles(table.freqs, axis, p))
    return torch.stack(out)[:, None]  # [B, 1, N, pairs]


def rot64(x, ang, table, sign=1.0):
    rot = table.rot_dim
    a, b = R.pair_indices(rot, table.layout)
    c, s = torch.cos(ang) * table.gain, torch.sin(ang) * table.gain * sign
    y = x.clone()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("long_positions", [False, True])
def test_rope_and_its_gradient(cuda_lib, case, long_positions):
    sla = cuda_lib
    name, form, B, H, N, d, rot, layout, axes, scaling = case
    dt = DT[name]
    x = make((B, H, N, d), dt, 1, form)
    table = table_of(sla, rot, layout, axes, scaling)
    pos = positions_of(axes, B, N, 2, form)
    ang = reference_angles(table, pos, axes, B, N)
    pos = pos.cuda() if long_positions else pos.int().cuda()
    xg = x.cuda().requires_grad_(True)
    y = sla.rope(xg, table, pos)
    assert y.shape == x.shape and y.is_contiguous()
    x64 = to_bhnd(x).double()
    ref = rot64(x64, ang, table)
    size = R.rotate_size(x64, rot, layout, table.gain)
    err = (to_bhnd(y.detach().cpu()).double() - ref).abs()
    assert (err <= rope_bound(ref, size, dt)).all(), (err / rope_bound(ref, size, dt)).max()
    dy = make((B, H, N, d), dt, 3, form)
    (dx,) = torch.autograd.grad(y, xg, dy.cuda())
    dy64 = to_bhnd(dy).double()
    ref = rot64(dy64, ang, table, -1.0)
    size = R.rotate_size(dy64, rot, layout, table.gain)
    err = (to_bhnd(dx.cpu()).double() - ref).abs()
    assert (err <= rope_bound(ref, size, dt)).all()


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("w32", [False, True])
def test_qk_norm_rope_and_its_gradients(cuda_lib, case, w32):
    sla = cuda_lib
    name, form, B, H, N, d, rot, layout, axes, scaling = case
    dt = DT[name]
    Hk = max(1, H // 2)
    eps = 1e-5
    xs = [make((B, h, N, d), dt, 10 + i, form) for i, h in enumerate((H, Hk))]
    xs[0][..., 0, :] = 0  # a row (packed: a head) of zeros: its norm is sqrt(eps)
    g = torch.Generator().manual_seed(12)
    ws = [(1 + 0.3 * torch.randn(d, generator=g)).to(torch.float32 if w32 else dt) for _ in range(2)]
    table = table_of(sla, rot, layout, axes, scaling)
    pos = positions_of(axes, B, N, 13, form)
    ang = reference_angles(table, pos, axes, B, N)
    leaves = [t.cuda().requires_grad_(True) for t in xs + ws]
    ys = sla.qk_norm_rope(*leaves, table, pos.cuda(), eps=eps)
    dys = [make((B, h, N, d), dt, 20 + i, form) for i, h in enumerate((H, Hk))]
    grads = torch.autograd.grad(ys, leaves, [t.cuda() for t in dys])
    # the mean of d squares: d half-steps at most, and a few operations behind it
    rel = (d + 16) * R.EPS32
    for i in range(2):
        x64, w64, dy64 = to_bhnd(xs[i]).double(), ws[i].double(), to_bhnd(dys[i]).double()
        n64, _ = R.rms_norm(x64, w64, eps)
        ref = rot64(n64, ang, table)
        size = R.rotate_size(n64, rot, layout, table.gain)
        bound = rope_bound(ref, size, dt) + rel * size
        err = (to_bhnd(ys[i].detach().cpu()).double() - ref).abs()
        assert (err <= bound).all(), (err / bound).max()
        # gradients, formula by formula
        _, r = R.rms_norm(x64, w64, eps)
        xh = x64 * r
        gr = rot64(dy64, ang, table, -1.0)
        gs = R.rotate_size(dy64, rot, layout, table.gain)
        gw = gr * w64
        dx = r * (gw - xh * (gw * xh).mean(-1, keepdim=True))
        sx = r * (gs * w64.abs() + xh.abs() * (gs * w64.abs() * xh.abs()).mean(-1, keepdim=True))
        bound = R.half_step(dt) * dx.abs() * 1.01 + (3 * rel + 1e-6) * sx + R.tiny(dt)
        err = (to_bhnd(grads[i].cpu()).double() - dx).abs()
        assert (err <= bound).all(), (err / bound).max()
        dw, sw = (gr * xh).sum((0, 1, 2)), (gs * xh.abs()).sum((0, 1, 2))
        # sums of at most N B H float32 terms; every chain of additions is shorter than 1024
        bound = R.half_step(ws[i].dtype) * dw.abs() * 1.01 + (rel + 1e-6 + 1024 * R.EPS32) * sw + R.tiny(dt)
        err = (grads[2 + i].cpu().double() - dw).abs()
        assert (err <= bound).all(), (err / bound).max()


def test_gradient_against_differences(cuda_lib):
    """<grad, v> against the kernel's own central difference, in float32."""
    sla = cuda_lib
    torch.manual_seed(5)
    q, k = (torch.randn(1, h, 9, 64).cuda() for h in (3, 2))
    ws = [1 + 0.3 * torch.randn(64).cuda() for _ in range(2)]
    table = sla.rope_table(64, layout="half")
    dys = [torch.randn_like(q), torch.randn_like(k)]
    leaves = [t.requires_grad_(True) for t in (q, k, *ws)]
    grads = torch.autograd.grad(sla.qk_norm_rope(*leaves, table), leaves, dys)
    h = 2.0 ** -7
    with torch.no_grad():
        for i, t in enumerate(leaves):
            v = torch.randn_like(t)
            f = []
            for s in (1, -1):
                args = [x + s * h * v if j == i else x for j, x in enumerate(leaves)]
                f.append(sum((y.double() * g.double()).sum() for y, g in zip(sla.qk_norm_rope(*args, table), dys)))
            got, want = ((f[0] - f[1]) / (2 * h)).item(), (grads[i].double() * v.double()).sum().item()
            # rounding: every y is off by ~2^-22 of itself, n of them add like noise; / h.
            # truncation: h^2 / 6 of the third derivative, which is of the order of the terms
            n = sum(g.numel() for g in dys)
            assert abs(got - want) <= 8 * (2.0 ** -22 * math.sqrt(n) / h + h * h * math.sqrt(n)), (i, got, want)


def test_padded_rows_in_place_and_strides(cuda_lib):
    sla = cuda_lib
    g = torch.Generator().manual_seed(3)
    x = torch.randn(2, 3, 70, 128, generator=g).bfloat16().cuda()
    table = sla.rope_table(128, layout="interleaved")
    want = sla.rope(x, table)
    # N < rows: the rows behind N keep what they hold
    out = torch.full((2, 3, 128, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    sla.rope(x, table, N=65, out=out)
    assert torch.equal(out[:, :, :65], want[:, :, :65]) and (out[:, :, 65:] == 7.0).all()
    assert sla.rope(x, table, N=65, rows=128).shape == (2, 3, 128, 128)
    # in place
    y = x.clone()
    assert sla.rope(y, table, out=y) is y and torch.equal(y, want)
    # rows that start on odd addresses take the narrow path, with the same result
    wide = torch.zeros(2, 3, 70, 131, dtype=torch.bfloat16, device="cuda")
    wide[..., 1:129] = x
    assert torch.equal(sla.rope(wide[..., 1:129], table), want)
    # a last dimension that is not contiguous, and repeated rows
    assert torch.equal(sla.rope(x.transpose(2, 3).contiguous().transpose(2, 3), table), want)
    e = x[:, :1].expand(2, 3, 70, 128)
    assert torch.equal(sla.rope(e, table), sla.rope(e.contiguous(), table))
    # gradients of broadcast heads add up
    leaf = x[:, :1].float().clone().requires_grad_(True)
    dy = torch.randn(2, 3, 70, 128, device="cuda")
    (dx,) = torch.autograd.grad(sla.rope(leaf.expand(2, 3, 70, 128), table), leaf, dy)
    torch.testing.assert_close(dx, sla.rope(dy, table, inverse=True).sum(1, keepdim=True), rtol=1e-5, atol=1e-5)
    # gradient rows behind N are zero, and the upstream rows there are not read
    leaf = x.clone().requires_grad_(True)
    y = sla.rope(leaf, table, N=65, rows=128)
    gy = torch.randn(2, 3, 128, 128, device="cuda").bfloat16()
    gy[:, :, 65:] = float("nan")
    (dx,) = torch.autograd.grad(y, leaf, gy)
    assert (dx[:, :, 65:] == 0).all() and torch.isfinite(dx).all()


def test_rotation_keeps_scores_relative(cuda_lib):
    """Scores of rotated q and k depend on the difference of positions alone, at far positions too."""
    sla = cuda_lib
    g = torch.Generator().manual_seed(4)
    q, k = (torch.randn(1, 1, 1, 64, generator=g).cuda() for _ in range(2))
    table = sla.rope_table(64)

    def score(p, r):
        pq, pk = (torch.tensor([t], device="cuda") for t in (p, r))
        return (sla.rope(q, table, pq).double() * sla.rope(k, table, pk).double()).sum().item()

    size = (q.double().norm() * k.double().norm()).item()
    for far in (10 ** 3, 10 ** 6, 10 ** 9):
        assert abs(score(5 + far, far) - score(5, 0)) <= 1e-6 * size * 4 + far * 2.0 ** -52 * size


def test_empty_and_refused(cuda_lib):
    sla = cuda_lib
    table = sla.rope_table(64)
    x = torch.randn(2, 3, 8, 64, device="cuda")
    assert sla.rope(x[:, :, :0], table).shape == (2, 3, 0, 64)
    assert sla.rope(x[:0], table).shape == (0, 3, 8, 64)
    yq, yk = sla.qk_norm_rope(x[:, :, :0], x[:, :1, :0], torch.ones(64, device="cuda"), torch.ones(64, device="cuda"), table)
    assert yq.shape == (2, 3, 0, 64) and yk.shape == (2, 1, 0, 64)
    pos = torch.arange(8, device="cuda")
    for bad in (dict(positions=pos[:7]), dict(positions=pos.float()), dict(positions=pos.cpu()), dict(N=9), dict(N=-1),
                dict(N=8, rows=7), dict(positions=pos.expand(3, 8)), dict(out=x.half()), dict(out=x[:, :, :7])):
        with pytest.raises(ValueError):
            sla.rope(x, table, **bad)
    with pytest.raises(ValueError):
        sla.rope(x.double(), table)
    with pytest.raises(ValueError):
        sla.rope(x.clone().requires_grad_(True), table, out=torch.empty_like(x))
    with pytest.raises(ValueError):
        sla.rope(x, sla.rope_table(64, sections=(16, 16)), pos)
    with pytest.raises(sla.SLAError):
        sla.rope(x, sla.rope_table(66))  # wider than the head
    with pytest.raises(sla.SLAError):
        sla.rope(x, table, out=torch.empty(2, 1, 8, 64, device="cuda").expand(2, 3, 8, 64))
    w = torch.ones(64, device="cuda")
    with pytest.raises(ValueError):
        sla.qk_norm_rope(x, x[:, :, :4], w, w, table)
    with pytest.raises(ValueError):
        sla.qk_norm_rope(x, x, w, w.half(), table)
    with pytest.raises(ValueError):
        sla.qk_norm_rope(x, x, w[:32], w, table)


def test_offsets_beyond_32_bits(cuda_lib):
    sla = cuda_lib
    H, N, d = 40, 440_000, 128
    assert H * N * d > 2 ** 31
    x = torch.zeros(N, H, d, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(50, H, d, generator=torch.Generator().manual_seed(6)).bfloat16().cuda()
    x[-50:] = tail
    table = sla.rope_table(d)
    y = sla.rope(x, table)
    pos = torch.arange(N - 50, N, device="cuda")
    assert torch.equal(y[-50:], sla.rope(tail, table, pos)) and (y[:-50] == 0).all()
    hm = x.transpose(0, 1).unsqueeze(0)  # the same memory as [1, H, N, d]
    assert torch.equal(sla.rope(hm, table)[0, :, -50:].transpose(0, 1), y[-50:])


def test_streams_and_graphs(cuda_lib):
    sla = cuda_lib
    x = torch.randn(2, 3, 80, 128, device="cuda").bfloat16()
    k = torch.randn(2, 1, 80, 128, device="cuda").bfloat16()
    w = [torch.randn(128, device="cuda").bfloat16() for _ in range(2)]
    table = sla.rope_table(128)
    pos = torch.randint(0, 1000, (80,), device="cuda")
    want = sla.qk_norm_rope(x, k, *w, table, pos)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sla.qk_norm_rope(x, k, *w, table, pos, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    dy = [torch.randn_like(t) for t in want]
    ref = sla.qk_norm_rope_backward(x, k, *w, *dy, table, pos)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = sla.qk_norm_rope(x, k, *w, table, pos)
        g = sla.qk_norm_rope_backward(x, k, *w, *dy, table, pos)
    x.copy_(torch.randn_like(x))
    pos.add_(17)
    graph.replay()
    for a, b in zip(y, sla.qk_norm_rope(x, k, *w, table, pos)):
        assert torch.equal(a, b)
    for a, b in zip(g, sla.qk_norm_rope_backward(x, k, *w, *dy, table, pos)):
        assert torch.equal(a, b)
    assert not torch.equal(g[0], ref[0])
