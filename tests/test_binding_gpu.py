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
