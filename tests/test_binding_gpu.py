"""What the binding of the operators beside the attention owes its caller: derivatives
that are whole or refused, writes that autograd sees, memory that outlives the call,
sizes and scratch tensors that are checked before anything is launched."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def randn(*shape, seed, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def fill_free_memory_with_nan(*shapes, dtype=torch.float32):
    """The allocator's free blocks of these sizes hold NaN: what is not written shows."""
    for _ in range(2):
        kept = [torch.full(s, math.nan, dtype=dtype, device="cuda") for s in shapes for _ in range(8)]
        del kept


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("packed", [False, True])
def test_rope_gradient_rows_behind_N_with_a_graph(cuda_lib, packed, inverse):
    """With create_graph the gradient of a rotation is a rotation that is differentiable
    itself; its rows behind N are zero, as without the graph."""
    sla = cuda_lib
    N, n = 5, 9
    shape = (n, 2, 64) if packed else (2, 2, n, 64)
    tail = (slice(N, None),) if packed else (slice(None), slice(None), slice(N, None))
    table = sla.rope_table(64)
    x, dy, v = (randn(*shape, seed=s, dtype=torch.float32).requires_grad_(True) for s in (1, 2, 3))
    y = sla.rope(x, table, N=N, inverse=inverse)
    (want,) = torch.autograd.grad(y, x, dy.detach(), retain_graph=True)
    fill_free_memory_with_nan(shape)
    (dx,) = torch.autograd.grad(y, x, dy, create_graph=True)
    assert (dx[tail] == 0).all() and torch.equal(dx, want)
    fill_free_memory_with_nan(shape)
    (ddy,) = torch.autograd.grad(dx, dy, v)
    assert (ddy[tail] == 0).all()
    assert torch.equal(ddy.narrow(0 if packed else 2, 0, N),
                       sla.rope(v.detach(), table, N=N, inverse=inverse).narrow(0 if packed else 2, 0, N))


def test_memory_outlives_a_call_on_another_stream(cuda_lib):
    """Dropped right after a call on another stream, a plan, a table and the tensors given with
    `stream` keep their memory until that stream is done."""
    sla = cuda_lib
    side = torch.cuda.Stream()
    x = randn(6, 2, 64, seed=1)
    w = torch.ones(64, device="cuda", dtype=torch.bfloat16)
    grid = torch.arange(6, device="cuda").repeat(2, 1)
    made = lambda: sla.prompt_plan([6], Hq=2, Hkv=2, d=64)  # noqa: E731
    o, lse = sla.prompt_forward(x, x, x, made())

    def plan_in(f):
        p = made()
        kept = [p.device_bytes]
        f(p)
        return kept

    def table_in(f):
        t = sla.rope_table(64, sections=(16, 16))
        kept = [t.turns, t.axis]
        f(t)
        return kept

    def tensors(f, *ts):
        ts = [t.clone() for t in ts]
        f(*ts)
        return ts

    def on_side(f):
        with torch.cuda.stream(side):
            return f()

    def trained(p):
        leaf = x.clone().requires_grad_(True)
        on_side(lambda: sla.prompt_attention(leaf, x, x, p).float().sum().backward())

    table, plan = sla.rope_table(64), made()
    calls = [
        lambda: plan_in(lambda p: sla.prompt_forward(x, x, x, p, stream=side)),
        lambda: plan_in(lambda p: sla.prompt_attention(x, x, x, p, stream=side.cuda_stream)),
        lambda: plan_in(lambda p: on_side(lambda: sla.prompt_attention(x, x, x, p))),
        lambda: plan_in(lambda p: sla.prompt_backward(x, x, x, o, lse, x, p, stream=side)),
        lambda: plan_in(trained),
        lambda: table_in(lambda t: sla.rope(x, t, grid, stream=side)),
        lambda: table_in(lambda t: on_side(lambda: sla.rope(x, t, grid))),
        lambda: table_in(lambda t: sla.qk_norm_rope(x, x, w, w, t, grid, stream=side)),
        lambda: table_in(lambda t: sla.qk_norm_rope_backward(x, x, w, w, x, x, t, grid, stream=side)),
        lambda: tensors(lambda a, p, y: sla.rope(a, table, p, out=y, stream=side), x, grid[0].contiguous(), x),
        lambda: tensors(lambda a, b, u, v, y, z: sla.qk_norm_rope(a, b, u, v, table, out=(y, z), stream=side), x, x, w, w, x, x),
        lambda: tensors(lambda a, b, c, y: sla.prompt_forward(a, b, c, plan, out=y, stream=side), x, x, x, x),
        lambda: tensors(lambda a, b, c: sla.prompt_attention(a, b, c, plan, stream=side), x, x, x),
        lambda: tensors(lambda a, b, c, s: sla.prompt_backward(x, x, x, a, s, b, plan, out=(c, x.clone(), x.clone()), stream=side),
                        o, x, x, lse),
    ]
    for i, call in enumerate(calls):
        call()  # what a first call sets up
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(400_000_000)  # clocks: a fifth of a second
        kept = call()
        sizes = [(t.shape, t.dtype, t.data_ptr()) for t in kept]
        del kept
        again = [torch.empty(s, dtype=d, device="cuda") for s, d, _ in sizes for _ in range(64)]
        assert not side.query(), i  # else nothing was tested
        assert not {p for *_, p in sizes} & {t.data_ptr() for t in again}, i
        torch.cuda.synchronize()


def test_forward_mode_is_refused(cuda_lib):
    """There is no forward-mode derivative: a dual tensor is refused, not stripped of its tangent."""
    sla = cuda_lib
    fwd = torch.autograd.forward_ad
    x, t = randn(5, 2, 64, seed=1), randn(5, 2, 64, seed=2)
    w = torch.ones(64, device="cuda", dtype=torch.bfloat16)
    table, plan = sla.rope_table(64), sla.prompt_plan([5], Hq=2, Hkv=2, d=64)
    with fwd.dual_level():
        dual, dual_w = fwd.make_dual(x, t), fwd.make_dual(w, w)
        for call in (lambda: sla.rope(dual, table), lambda: sla.rope(x, table, out=fwd.make_dual(x.clone(), t)),
                     lambda: sla.qk_norm_rope(dual, x, w, w), lambda: sla.qk_norm_rope(x, dual, w, w),
                     lambda: sla.qk_norm_rope(x, x, dual_w, w), lambda: sla.qk_norm_rope(x, x, w, dual_w),
                     lambda: sla.prompt_attention(dual, x, x, plan), lambda: sla.prompt_attention(x, dual, x, plan),
                     lambda: sla.prompt_attention(x, x, dual, plan)):
            with pytest.raises(NotImplementedError):
                call()
        sla.rope(x, table), sla.prompt_attention(x, x, x, plan)  # others go on inside the level
    sla.rope(x, table)


def out_calls(sla):
    """(operator, its `out` tensors, the call) of every call that writes to the caller's tensors."""
    x, w = randn(5, 2, 64, seed=1), torch.ones(64, device="cuda", dtype=torch.bfloat16)
    table, plan = sla.rope_table(64), sla.prompt_plan([5], Hq=2, Hkv=2, d=64)
    o, lse = sla.prompt_forward(x, x, x, plan)
    new = lambda n: [torch.zeros_like(x) for _ in range(n)]  # noqa: E731
    return [("rope", new(1), lambda t: sla.rope(x, table, out=t[0])),
            ("qk_norm_rope", new(2), lambda t: sla.qk_norm_rope(x, x, w, w, table, out=tuple(t))),
            ("prompt_forward", new(1), lambda t: sla.prompt_forward(x, x, x, plan, out=t[0])),
            ("prompt_backward", new(3), lambda t: sla.prompt_backward(x, x, x, o, lse, x, plan, out=tuple(t)))]


def test_writes_to_out_are_seen_by_autograd(cuda_lib):
    """A tensor that another operation saved for its backward and that `out` overwrites is noticed."""
    sla = cuda_lib
    for name, outs, call in out_calls(sla):
        for i in range(len(outs)):
            leaf = torch.ones(5, 2, 64, device="cuda", dtype=torch.bfloat16, requires_grad=True)
            y = (leaf * outs[i]).sum()
            before = outs[i]._version
            call(outs)
            assert outs[i]._version > before, name
            with pytest.raises(RuntimeError, match="inplace"):
                y.backward()
    # in place: the input's own version
    x, table = randn(5, 2, 64, seed=1), sla.rope_table(64)
    before = x._version
    sla.rope(x, table, out=x)
    assert x._version > before
    # without autograd's bookkeeping there is none to keep
    with torch.inference_mode():
        y = torch.empty_like(x)
        sla.rope(x, table, out=y)
    sla.rope(x, table, out=y)


def test_out_that_requires_grad_is_refused(cuda_lib):
    sla = cuda_lib
    for name, outs, call in out_calls(sla):
        for i in range(len(outs)):
            some = [t.requires_grad_(True) if i == j else t for j, t in enumerate(torch.zeros_like(t) for t in outs)]
            with pytest.raises(ValueError, match="requires grad"):
                call(some)
            with torch.no_grad():
                before = some[i]._version
                call(some)
            assert some[i]._version > before, name


def test_counts_past_32_bits_are_refused(cuda_lib):
    """Views of one token or one head, repeated: no count is cut to its low 32 bits."""
    sla = cuda_lib
    table = sla.rope_table(2)
    w = torch.ones(2, device="cuda")
    one = torch.ones(1, 1, 2, device="cuda", dtype=torch.bfloat16)
    for x in (one.expand(2 ** 32 + 5, 1, 2), one[None].expand(1, 1, 2 ** 32 + 5, 2), one[None].expand(2 ** 32 + 1, 1, 1, 2),
              one.expand(1, 2 ** 32 + 1, 2)):
        for call in (lambda: sla.rope(x, table), lambda: sla.qk_norm_rope(x, x, w, w, table),
                     lambda: sla.qk_norm_rope_backward(x, x, w, w, x, x, table)):
            with pytest.raises(sla.SLAError) as e:
                call()
            assert e.value.status == sla.SLA_ERR_UNSUPPORTED
    # the first tokens of a long view are not many
    assert sla.rope(one.expand(2 ** 20, 1, 2), table, N=3, out=torch.empty(3, 1, 2, device="cuda", dtype=torch.bfloat16)).shape == (3, 1, 2)


def test_workspaces_are_checked(cuda_lib):
    """A workspace on the host, or one whose bytes are not in one piece, is refused before a launch."""
    sla = cuda_lib
    x, w = randn(6, 2, 64, seed=1), torch.ones(64, device="cuda", dtype=torch.bfloat16)
    k = torch.zeros(9000, 2, 64, device="cuda", dtype=torch.bfloat16)
    one, plan = sla.prompt_plan([1], [9000], Hq=2, Hkv=2, d=64), sla.prompt_plan([6], Hq=2, Hkv=2, d=64)
    assert one.workspace_size > 0
    o, lse = sla.prompt_forward(x, x, x, plan)
    for n, call in ((one.workspace_size, lambda ws: sla.prompt_forward(x[:1], k, k, one, workspace=ws)),
                    (plan.backward_workspace_size, lambda ws: sla.prompt_backward(x, x, x, o, lse, x, plan, workspace=ws)),
                    (1 << 20, lambda ws: sla.qk_norm_rope_backward(x, x, w, w, x, x, workspace=ws))):
        for bad in (torch.zeros(n, dtype=torch.uint8), torch.zeros(n, dtype=torch.uint8).pin_memory(),
                    torch.zeros(2 * n, dtype=torch.uint8, device="cuda")[::2],
                    torch.zeros(1, dtype=torch.uint8, device="cuda").expand(n)):
            with pytest.raises(ValueError, match="workspace"):
                call(bad)
        call(torch.zeros(n, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("rows", [None, 16])
def test_gradients_where_one_output_is_not_used(cuda_lib, rows):
    """The other output's gradient counts as zeros, of its own shape."""
    sla = cuda_lib
    table = sla.rope_table(64)
    q, k = randn(2, 4, 9, 64, seed=1), randn(2, 2, 9, 64, seed=2)
    w = [1 + 0.2 * randn(64, seed=s, dtype=torch.float32) for s in (3, 4)]
    dy = [randn(2, h, rows or 9, 64, seed=5 + h) for h in (4, 2)]
    for i in range(2):
        leaves = [t.detach().requires_grad_(True) for t in (q, k, *w)]
        y = sla.qk_norm_rope(*leaves, table, N=7, rows=rows)
        got = torch.autograd.grad(y[i], leaves, dy[i])
        zero = [g if i == j else torch.zeros_like(g) for j, g in enumerate(dy)]
        want = sla.qk_norm_rope_backward(q, k, *w, *zero, table, N=7)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert (got[1 - i] == 0).all() and (got[3 - i] == 0).all() and got[i].any() and got[2 + i].any()


FIRST_CALL = """
import torch
import sparse_linear_attention_pool_b200 as sla
x, w = torch.randn(40, 2, 64, device="cuda").bfloat16(), torch.ones(64, device="cuda", dtype=torch.bfloat16)
k = torch.zeros(9000, 2, 64, device="cuda", dtype=torch.bfloat16)
plan, table = sla.prompt_plan([40], Hq=2, Hkv=2, d=64), sla.rope_table(64)
one = sla.prompt_plan([1], [9000], Hq=2, Hkv=2, d=64)


def step():
    q, h = sla.qk_norm_rope(x, x, w, w, table)
    o, lse, rest = sla.prompt_forward(q, h, x, plan, want_rest=True)
    dq, dk, dv = sla.prompt_backward(q, h, x, o, lse, x, plan, rest=rest)
    return (o, dv, sla.rope(x, table), sla.prompt_attention(q[:1], k, k, one), *sla.qk_norm_rope_backward(x, x, w, w, dq, dk, table))


g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    made = step()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(made, step()))
print("same")
"""


def test_first_call_of_a_process_is_captured(cuda_lib):
    """A capture needs no call before it that loads the kernels."""
    import os
    import subprocess
    import sys

    r = subprocess.run([sys.executable, "-c", FIRST_CALL], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
