"""The operators beside the attention run together, as a model uses them: norm and
rotation of queries and keys, then the sparse-linear or the prompt attention."""

import pytest
import torch

import workloads as W
from tests import operator_reference as R

pytestmark = pytest.mark.gpu


def randn(*shape, seed, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def test_attention_with_norm_and_rotation(cuda_lib):
    """sla.attention's own norm and rotation are the separate calls, forward and backward,
    on a video-shaped grid of three position axes with padded rows."""
    sla = cuda_lib
    B, H, d, f, h, w = 1, 2, 128, 3, 5, 7
    N = f * h * w
    Np = W.n_pad(N)
    x = randn(B, Np, 3, H, d, seed=1)
    x[:, N:] = float("nan")  # pad rows may hold anything
    wq, wk = (1 + 0.1 * randn(d, seed=s, dtype=torch.float32) for s in (2, 3))
    n = torch.arange(N, device="cuda")
    grid = torch.stack([n // (h * w), n // w % h, n % w])
    table = sla.rope_table(d, sections=(22, 21, 21))
    do = randn(B, H, Np, d, seed=4)
    kw = dict(N=N, variant="sla", k_crit=1, k_neg=0)

    def leaves():
        return [t.detach().requires_grad_(True) for t in (x[:, :, 0].transpose(1, 2), x[:, :, 1].transpose(1, 2),
                                                           x[:, :, 2].transpose(1, 2), wq, wk)]

    a = leaves()
    o = sla.attention(*a[:3], qk_norm=a[3:], norm_eps=1e-5, rotary=table, positions=grid, **kw)
    got = torch.autograd.grad(o, a, do)
    b = leaves()
    q2, k2 = sla.qk_norm_rope(*b[:2], *b[3:], table, grid, eps=1e-5, N=N)
    o2 = sla.attention(q2, k2, b[2], **kw)
    want = torch.autograd.grad(o2, b, do)
    assert torch.equal(o[:, :, :N], o2[:, :, :N]) and torch.isfinite(o[:, :, :N].float()).all()
    for g, h_ in zip(got, want):
        assert torch.equal(g, h_) and torch.isfinite(g.float()).all()
    # the rotation alone
    o3 = sla.attention(*(t.detach() for t in a[:3]), rotary=table, positions=grid, **kw)
    q3, k3 = (sla.rope(t.detach(), table, grid, N=N) for t in a[:2])
    assert torch.equal(o3[:, :, :N], sla.attention(q3, k3, a[2].detach(), **kw)[:, :, :N])
    with pytest.raises(ValueError):
        sla.attention(*(t.detach() for t in a[:3]), positions=grid, **kw)


def block(sla, x, w, plan, table, Hq, Hkv, d):
    """A prompt's attention block: one projection's heads, norm, rotation, attention."""
    qkv = x.view(-1, Hq + 2 * Hkv, d)
    q, k = sla.qk_norm_rope(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], *w, table, plan.positions())
    return sla.prompt_attention(q, k, qkv[:, Hq + Hkv:], plan)


def test_prompt_block_against_float64(cuda_lib):
    sla = cuda_lib
    Hq, Hkv, d, lens = 6, 2, 64, [90, 1, 150]
    plan = sla.prompt_plan(lens, Hq=Hq, Hkv=Hkv, d=d)
    table = sla.rope_table(d, layout="half")
    x = randn(sum(lens), (Hq + 2 * Hkv) * d, seed=5).requires_grad_(True)
    w = [(1 + 0.1 * randn(d, seed=s, dtype=torch.float32)).requires_grad_(True) for s in (6, 7)]
    do = randn(sum(lens), Hq, d, seed=8)
    o = block(sla, x, w, plan, table, Hq, Hkv, d)
    got = torch.autograd.grad(o, [x, *w], do)
    # the same in float64, through torch's autograd
    x64 = x.detach().cpu().double().requires_grad_(True)
    w64 = [t.detach().cpu().double().requires_grad_(True) for t in w]
    qkv = x64.view(-1, Hq + 2 * Hkv, d)
    ang = R.angles(table.freqs, None, plan.positions().cpu())
    q, k = (R.rotate(R.rms_norm(t, u, 1e-6)[0].transpose(0, 1), ang, d, "half").transpose(0, 1)
            for t, u in ((qkv[:, :Hq], w64[0]), (qkv[:, Hq:Hq + Hkv], w64[1])))
    v = qkv[:, Hq + Hkv:]
    outs, at = [], 0
    for n in lens:
        s = slice(at, at + n)
        at += n
        sc = torch.einsum("ihd,jhd->hij", q[s], k[s].repeat_interleave(Hq // Hkv, 1)) / d ** 0.5
        sc = sc.masked_fill(torch.ones(n, n, dtype=torch.bool).triu(1), float("-inf"))
        outs.append(torch.einsum("hij,jhd->ihd", torch.softmax(sc, -1), v[s].repeat_interleave(Hq // Hkv, 1)))
    ref = torch.cat(outs)
    want = torch.autograd.grad(ref, [x64, *w64], do.cpu().double())
    # relative 2-norm: at most eight bf16 roundings (q, k, P, O, dS, dq and dk of the attention, dx),
    # each 2^-8, doubled for the scores that the rounded q and k shift
    for g, h in zip((o.detach(), *got), (ref.detach(), *want)):
        rel = ((g.cpu().double() - h).norm() / h.norm()).item()
        assert rel <= 16 * 2.0 ** -8, rel


def test_prompt_block_in_a_graph(cuda_lib):
    """Forward and explicit backward of the block, captured and replayed on new inputs."""
    sla = cuda_lib
    Hq, Hkv, d, lens = 4, 2, 128, [130, 61]
    plan, table = sla.prompt_plan(lens, Hq=Hq, Hkv=Hkv, d=d), sla.rope_table(d)
    pos = plan.positions()
    x, do = randn(sum(lens), Hq + 2 * Hkv, d, seed=9), randn(sum(lens), Hq, d, seed=10)
    w = [torch.ones(d, device="cuda", dtype=torch.bfloat16) for _ in range(2)]

    def step():
        q0, k0, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        q, k = sla.qk_norm_rope(q0, k0, *w, table, pos)
        o, lse, rest = sla.prompt_forward(q, k, v, plan, want_rest=True)
        dq, dk, dv = sla.prompt_backward(q, k, v, o, lse, do, plan, rest=rest)
        return (o, dv, *sla.qk_norm_rope_backward(q0, k0, *w, dq, dk, table, pos))

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        made = step()
    for seed in (11, 12):
        x.copy_(randn(*x.shape, seed=seed))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(made, step()))


def test_autograd_in_a_graph(cuda_lib):
    """A training step captured through autograd, once no eager graph of its leaves is alive
    (torch ties a leaf to the stream of the oldest living graph, which a capture cannot wait
    for; the explicit backward calls have no such tie and are captured above)."""
    sla = cuda_lib
    Hq, Hkv, d, lens = 4, 2, 64, [100, 30]
    plan, table = sla.prompt_plan(lens, Hq=Hq, Hkv=Hkv, d=d), sla.rope_table(d)
    x = randn(sum(lens), (Hq + 2 * Hkv) * d, seed=13).requires_grad_(True)
    w = [torch.ones(d, device="cuda", requires_grad=True) for _ in range(2)]
    do = randn(sum(lens), Hq, d, seed=14)
    pos = plan.positions()

    def f():
        qkv = x.view(-1, Hq + 2 * Hkv, d)
        q, k = sla.qk_norm_rope(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], *w, table, pos)
        return torch.autograd.grad(sla.prompt_attention(q, k, qkv[:, Hq + Hkv:], plan), [x, *w], do)

    want = f()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        made = f()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(made, want))


def test_decoding_step_by_step_is_the_whole_prompt(cuda_lib):
    """Tokens one by one over a growing cache, each rotated at its own position, give the
    whole prompt's rows."""
    sla = cuda_lib
    Hq, Hkv, d, n = 4, 1, 128, 7
    table = sla.rope_table(d, layout="half")
    x = randn(n, Hq + 2 * Hkv, d, seed=15)
    w = [torch.ones(d, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    whole = sla.prompt_plan([n], Hq=Hq, Hkv=Hkv, d=d)
    q, k = sla.qk_norm_rope(x[:, :Hq], x[:, Hq:Hq + Hkv], *w, table, whole.positions())
    want = sla.prompt_attention(q, k, x[:, Hq + Hkv:], whole)
    cache_k, cache_v = torch.empty(n, Hkv, d, dtype=torch.bfloat16, device="cuda"), x[:, Hq + Hkv:].contiguous()
    for t in range(n):
        plan = sla.prompt_plan([1], [t + 1], Hq=Hq, Hkv=Hkv, d=d)
        row = x[t:t + 1]
        q1, k1 = sla.qk_norm_rope(row[:, :Hq], row[:, Hq:Hq + Hkv], *w, table, plan.positions())
        assert torch.equal(q1, q[t:t + 1])
        cache_k[t:t + 1] = k1
        o = sla.prompt_attention(q1, cache_k[:t + 1], cache_v[:t + 1], plan)
        # the same products in another tile: P and O rounded alike but for the order of the sums
        assert ((o - want[t:t + 1]).abs().float() <= 2 * 2.0 ** -8 * want[t:t + 1].abs().float() + 2.0 ** -8).all()


def test_second_derivatives_are_refused(cuda_lib):
    sla = cuda_lib
    plan = sla.prompt_plan([5], Hq=1, Hkv=1, d=64)
    q = randn(5, 1, 64, seed=16).requires_grad_(True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(sla.prompt_attention(q, q, q, plan).sum(), q, create_graph=True)
    one = torch.ones(64, device="cuda")
    with pytest.raises(RuntimeError):
        torch.autograd.grad(sla.qk_norm_rope(q, q, one, one)[0].sum(), q, create_graph=True)
    # a rotation is linear: its gradient's gradient is the rotation itself
    table = sla.rope_table(64)
    x, dy, v = (randn(5, 1, 64, seed=s, dtype=torch.float32).requires_grad_(True) for s in (17, 18, 19))
    (dx,) = torch.autograd.grad(sla.rope(x, table), x, dy, create_graph=True)
    (ddy,) = torch.autograd.grad(dx, dy, v.detach())
    assert torch.equal(ddy, sla.rope(v.detach(), table))
    # positions changed in place between forward and backward are noticed
    pos = torch.arange(5, device="cuda")
    y = sla.rope(x, table, pos)
    pos.add_(1)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(y, x, dy)
