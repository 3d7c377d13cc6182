"""Packed prompt attention on the GPU against float64."""

import math

import pytest
import torch

from tests import operator_reference as R

pytestmark = pytest.mark.gpu

H8 = 2.0 ** -8  # half a bf16 step, relative

# lens_q, lens_k, Hq, Hkv, d, causal
CASES = [
    ([1], None, 1, 1, 64, True),
    ([1], None, 4, 1, 128, False),
    ([127, 1, 128, 129], None, 2, 2, 128, True),
    ([300, 17], None, 3, 1, 64, True),         # groups of 3: 42 tokens to a tile, 2 rows idle
    ([255, 513, 64], None, 4, 2, 128, True),
    ([100, 260], None, 5, 1, 128, False),
    ([33, 0, 65], None, 6, 3, 64, True),       # an empty sequence between two
    ([40], None, 65, 1, 64, True),             # one token to a tile, almost half of it idle
    ([9], None, 128, 1, 64, True),
    ([1, 1, 1], [1, 700, 129], 8, 2, 128, True),     # single tokens over caches
    ([1, 3], [5000, 4100], 4, 2, 128, True),         # long enough for split keys
    ([1], [20000], 7, 1, 64, False),
    ([50, 200], [450, 200], 4, 4, 64, True),         # a piece behind a cache
    ([130, 7], [60, 0], 2, 1, 128, True),            # rows that see nothing
    ([5], [0, ], 2, 1, 64, False),                   # no keys at all
    ([5, 4], [0, 3], 2, 1, 64, False),
    ([600], None, 2, 1, 128, True),
    ([1300, 900], None, 2, 2, 128, True),
    ([33, 1100], None, 4, 2, 64, False),
]
IDS = lambda c: f"{c[0]}-{c[1]}-{c[2]}x{c[3]}-{c[4]}-{'causal' if c[5] else 'full'}".replace(" ", "")  # noqa: E731


def make(case, seed=0, spread=1.0):
    lq, lk, Hq, Hkv, d, causal = case
    lk = lq if lk is None else lk
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(sum(lq), Hq, d, generator=g) * spread).bfloat16()
    k = torch.randn(sum(lk), Hkv, d, generator=g).bfloat16()
    v = torch.randn(sum(lk), Hkv, d, generator=g).bfloat16()
    do = torch.randn(sum(lq), Hq, d, generator=g).bfloat16()
    return q, k, v, do, lq, lk


def plan_of(sla, case, **kw):
    lq, lk, Hq, Hkv, d, causal = case
    return sla.prompt_plan(lq, lk, Hq=Hq, Hkv=Hkv, d=d, causal=causal, **kw)


def score_error(d, q, k, scale):
    """How far a score's exponent may be off: float32 sums of d products in any order (d half-steps of
    the sum of their sizes, twice for truncating adders), the float32 exponent's own rounding and 2^x's."""
    size = (q.abs().double().amax() * k.abs().double().amax() * d * scale).item() if k.numel() else 0.0
    return (2 * d + 4) * R.EPS32 * size + 2.0 ** -21


def check_forward(case, o, lse, ref, q, k, scale=None):
    d = case[4]
    e = score_error(d, q, k, 1 / math.sqrt(d) if scale is None else scale)
    # P rounded to bf16, off by e in the exponent (twice: P and the sum), O rounded to bf16
    bound = (H8 + 3 * e) * ref["o_size"] * 1.01 + H8 * ref["o"].abs() * 1.01 + 1e-30
    err = (o.cpu().double() - ref["o"]).abs()
    assert (err <= bound).all(), (err / bound).max()
    if lse is not None:
        got, want = lse.cpu().double(), ref["lse"]
        assert torch.equal(got == -math.inf, want == -math.inf)
        fin = want != -math.inf
        assert ((got[fin] - want[fin]).abs() <= 2 * e + 2.0 ** -21 * (1 + want[fin].abs())).all()


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(cuda_lib, case):
    sla = cuda_lib
    q, k, v, _, lq, lk = make(case)
    plan = plan_of(sla, case)
    o, lse = sla.prompt_forward(q.cuda(), k.cuda(), v.cuda(), plan)
    assert sla.read_device_status(plan.device_bytes) == 0
    check_forward(case, o, lse, R.prompt(q, k, v, lq, lk, case[5]), q, k)
    assert torch.equal(sla.prompt_attention(q.cuda(), k.cuda(), v.cuda(), plan), o)  # bit for bit, again


@pytest.mark.parametrize("case", [CASES[2], CASES[10], CASES[3]], ids=IDS)
@pytest.mark.parametrize("spread,scale", [(30.0, None), (1.0, 1e-4), (0.0, 1.0)])
def test_forward_of_peaked_and_flat_rows(cuda_lib, case, spread, scale):
    sla = cuda_lib
    q, k, v, _, lq, lk = make(case, seed=1, spread=spread)
    plan = plan_of(sla, case, softmax_scale=scale or 0.0)
    o, lse = sla.prompt_forward(q.cuda(), k.cuda(), v.cuda(), plan)
    check_forward(case, o, lse, R.prompt(q, k, v, lq, lk, case[5], scale), q, k, scale)


def test_growing_maxima(cuda_lib):
    """Scores that grow towards the first keys: the running maximum is raised in every block."""
    sla = cuda_lib
    case = ([700], None, 2, 1, 128, True)
    q, k, v, _, lq, lk = make(case, seed=2)
    q[..., 0], k[:, :, 0] = 8.0, torch.linspace(120.0, 0.0, 700)[:, None].bfloat16()
    o, lse = sla.prompt_forward(q.cuda(), k.cuda(), v.cuda(), plan_of(sla, case))
    check_forward(case, o, lse, R.prompt(q, k, v, lq, lk, True), q, k)
    case = ([700], None, 2, 1, 128, False)
    o, lse = sla.prompt_forward(q.cuda(), k.cuda(), v.cuda(), plan_of(sla, case))
    check_forward(case, o, lse, R.prompt(q, k, v, lq, lk, False), q, k)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
def test_more_items_than_sms(cuda_lib, d, causal):
    """Over a thousand items of two tiles, so that every SM takes several: second tiles that are not there,
    items without keys, rows that see nothing, last blocks of every length; another sequence's NaN."""
    sla = cuda_lib
    lens = [129, 1, 64, 200, 300, 5, 128, 63] * 13, [129, 40, 0, 500, 100, 260, 128, 63] * 13
    case = (*lens, 16, 8, d, causal)
    q, k, v, _, lq, lk = make(case, seed=5)
    plan = plan_of(sla, case)
    o, lse = sla.prompt_forward(q.cuda(), k.cuda(), v.cuda(), plan)
    assert sla.read_device_status(plan.device_bytes) == 0
    check_forward(case, o, lse, R.prompt(q, k, v, lq, lk, causal), q, k)
    bad, first = 51, (sum(lq[:51]), sum(lk[:51]))  # 500 keys
    k[first[1]:first[1] + lk[bad]], v[first[1]:first[1] + lk[bad]] = math.nan, math.inf
    p = sla.prompt_attention(q.cuda(), k.cuda(), v.cuda(), plan)
    rest = torch.ones(sum(lq), dtype=torch.bool)
    rest[first[0]:first[0] + lq[bad]] = False
    assert torch.equal(p.cpu()[rest], o.cpu()[rest]) and p.cpu()[~rest].isnan().all()


def test_strided_rows_and_rows_behind_the_last_sequence(cuda_lib):
    sla = cuda_lib
    case = ([70, 200, 33], None, 4, 2, 64, True)
    q, k, v, _, lq, _ = make(case)
    plan = plan_of(sla, case)
    want = sla.prompt_attention(q.cuda(), k.cuda(), v.cuda(), plan)
    # one projection's output with 41 more tokens of NaN behind the last sequence
    x = torch.full((sum(lq) + 41, 4 + 2 + 2, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    x[:sum(lq), :4], x[:sum(lq), 4:6], x[:sum(lq), 6:] = q.cuda(), k.cuda(), v.cuda()
    out = torch.full((sum(lq) + 41, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    sla.prompt_forward(x[:, :4], x[:, 4:6], x[:, 6:], plan, out=out)
    assert torch.equal(out[:sum(lq)], want) and (out[sum(lq):] == 5.0).all()
    # head-major memory, rows that are not 16-byte steps apart, a broadcast head
    hm = [t.cuda().transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v)]
    assert torch.equal(sla.prompt_attention(*hm, plan), want)
    odd = torch.zeros(sum(lq), 4, 67, dtype=torch.bfloat16, device="cuda")
    odd[..., 1:65] = q.cuda()
    assert torch.equal(sla.prompt_attention(odd[..., 1:65], k.cuda(), v.cuda(), plan), want)
    ke, ve = (t.cuda()[:, :1].expand(-1, 2, -1) for t in (k, v))
    assert torch.equal(sla.prompt_attention(q.cuda(), ke, ve, plan),
                       sla.prompt_attention(q.cuda(), ke.contiguous(), ve.contiguous(), plan))


@pytest.mark.parametrize("d", [64, 128])
def test_sequences_do_not_touch_each_other(cuda_lib, d):
    """NaN and infinities in one sequence stay in it."""
    sla = cuda_lib
    case = ([70, 150, 33], None, 3, 1, d, True)
    q, k, v, _, lq, _ = make(case, seed=3)
    plan = plan_of(sla, case)
    want = sla.prompt_attention(q.cuda(), k.cuda(), v.cuda(), plan)
    for bad in (float("nan"), float("inf")):
        ts = [t.clone() for t in (q, k, v)]
        for t in ts:
            t[70:220] = bad
        got = sla.prompt_attention(*(t.cuda() for t in ts), plan)
        keep = torch.ones(253, dtype=torch.bool)
        keep[70:220] = False
        assert torch.equal(got[keep], want[keep])
        assert not torch.isfinite(got[70:220].float()).any()


def test_future_keys_do_not_reach_the_past(cuda_lib):
    sla = cuda_lib
    case = ([500], None, 2, 1, 128, True)
    q, k, v, _, _, _ = make(case, seed=4)
    plan = plan_of(sla, case)
    want = sla.prompt_attention(q.cuda(), k.cuda(), v.cuda(), plan)
    k2, v2 = k.clone(), v.clone()
    k2[300:], v2[300:] = 100.0, -77.0
    got = sla.prompt_attention(q.cuda(), k2.cuda(), v2.cuda(), plan)
    assert torch.equal(got[:300], want[:300]) and not torch.equal(got[300:], want[300:])
    k2[300:] = float("nan")  # a score that the mask leaves out may be anything
    got = sla.prompt_attention(q.cuda(), k2.cuda(), v.cuda(), plan)
    assert torch.equal(got[:300], want[:300]) and torch.isnan(got[300:].float()).all()


def test_a_prompt_in_pieces_is_the_whole_prompt(cuda_lib):
    """Pieces and single tokens over the cache give the whole prompt's rows."""
    sla = cuda_lib
    case = ([260], None, 4, 2, 128, True)
    q, k, v, _, _, _ = make(case, seed=5)
    ref = R.prompt(q, k, v, [260], [260], True)
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    for a, b in ((0, 100), (100, 230), (230, 259), (259, 260)):
        plan = sla.prompt_plan([b - a], [b], Hq=4, Hkv=2, d=128)
        o, lse = sla.prompt_forward(q[a:b], k[:b], v[:b], plan)
        part = {n: t[a:b] for n, t in ref.items()}
        check_forward(case, o, lse, part, q.cpu(), k.cpu())


def test_streams_graphs_and_two_calls_of_one_plan(cuda_lib):
    sla = cuda_lib
    case = ([1, 2], [9000, 6000], 8, 2, 128, True)  # split keys: the calls have workspaces
    q, k, v, _, _, _ = make(case, seed=6)
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    plan = plan_of(sla, case)
    assert plan.workspace_size > 0
    want, want_lse = sla.prompt_forward(q, k, v, plan)
    q2 = q.flip(1).contiguous()
    want2, _ = sla.prompt_forward(q2, k, v, plan)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        a, _ = sla.prompt_forward(q, k, v, plan, stream=side)
        b, _ = sla.prompt_forward(q2, k, v, plan)
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want2)
    graphs = []
    for x in (q, q2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = sla.prompt_forward(x, k, v, plan)
        graphs.append((g, y))
    for _ in range(3):
        for g, y in graphs:
            y[0].zero_()
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1][0], want) and torch.equal(graphs[0][1][1], want_lse)
    assert torch.equal(graphs[1][1][0], want2)
    assert sla.read_device_status(plan.device_bytes) == 0


def test_from_a_fresh_thread(cuda_lib):
    """A thread that has made no CUDA call yet has no context current (autograd's threads, a server's)."""
    import threading

    sla = cuda_lib
    case = ([90, 20], None, 4, 2, 128, True)
    q, k, v, do, _, _ = make(case, seed=13)
    q, k, v, do = q.cuda(), k.cuda(), v.cuda(), do.cuda()
    plan = plan_of(sla, case)
    o, lse = sla.prompt_forward(q, k, v, plan)
    grads = sla.prompt_backward(q, k, v, o, lse, do, plan)
    out, dx = torch.empty_like(o), tuple(torch.empty_like(t) for t in (q, k, v))
    got = []

    def work(f):
        try:
            got.append(f())
        except Exception as e:  # noqa: BLE001
            got.append(e)

    for f in (lambda: sla.prompt_forward(q, k, v, plan, out=out),
              lambda: sla.prompt_backward(q, k, v, o, lse, do, plan, out=dx)):
        t = threading.Thread(target=work, args=(f,))
        t.start()
        t.join()
    assert not any(isinstance(x, Exception) for x in got), got
    assert torch.equal(out, o) and all(torch.equal(a, b) for a, b in zip(dx, grads))


def test_offsets_beyond_32_bits(cuda_lib):
    """A cache of more than 2^31 values: its last sequence is read where it is."""
    sla = cuda_lib
    first, last = 2_100_000, 300
    assert (first + last) * 8 * 128 > 2 ** 31
    k, v = (torch.zeros(first + last, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    case = ([1, 3], [first, last], 16, 8, 128, True)
    g = torch.Generator().manual_seed(14)
    q = torch.randn(4, 16, 128, generator=g).bfloat16()
    kl, vl = (torch.randn(last, 8, 128, generator=g).bfloat16() for _ in range(2))
    k[first:], v[first:] = kl.cuda(), vl.cuda()
    v[first - 1] = 3.0  # the first sequence: equal scores over zeros and one row of 3
    plan = plan_of(sla, case)
    o, lse = sla.prompt_forward(q.cuda(), k, v, plan)
    ref = R.prompt(q[1:], kl, vl, [3], [last], True)
    check_forward(case, o[1:], lse[1:], ref, q, kl)
    # 3 / n for every value, from a sum of 2 million equal weights in float32
    assert torch.allclose(o[0].float() * first, torch.full((16, 128), 3.0, device="cuda"), rtol=2.0 ** -7, atol=0)
    assert torch.allclose(lse[0], torch.full((16,), math.log(first), device="cuda"), rtol=0, atol=1e-4)


def test_refusals(cuda_lib):
    sla = cuda_lib
    case = ([10, 20], None, 4, 2, 64, True)
    q, k, v, _, _, _ = make(case)
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    plan = plan_of(sla, case)
    for bad in ((q[:29], k, v), (q, k[:29], v), (q[:, :3], k, v), (q, k, v[:, :1]), (q[..., :32], k, v),
                (q.float(), k, v), (q, k.half(), v), (q.cpu(), k, v), (q[0], k, v)):
        with pytest.raises(ValueError):
            sla.prompt_attention(*bad, plan)
    with pytest.raises(ValueError):
        sla.prompt_forward(q, k, v, plan, out=torch.empty(30, 4, 64, device="cuda"))
    with pytest.raises(sla.SLAError):
        sla.prompt_forward(q, k, v, plan, out=torch.empty(1, 4, 64, device="cuda", dtype=torch.bfloat16).expand(30, 4, 64))
    small = sla.prompt_plan([1], [9000], Hq=4, Hkv=2, d=64)
    kk = torch.zeros(9000, 2, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(sla.SLAError):
        sla.prompt_forward(q[:1], kk, kk, small, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


def check_grads(case, got, ref, q, k):
    """dV: P rounded to bf16. dK, dQ: dS rounded to bf16, its D from an O rounded to bf16 (both
    within the sizes |P dP| + |P| rowsum |dO O|); every exponent off by e; one rounding at the end."""
    e = score_error(case[4], q, k, 1 / math.sqrt(case[4]))
    for name, t in zip(("dq", "dk", "dv"), got):
        rounds = 1 if name == "dv" else 2
        bound = (rounds * H8 + 4 * e) * ref[name + "_size"] * 1.02 + H8 * ref[name].abs() * 1.02 + 1e-30
        err = (t.cpu().double() - ref[name]).abs()
        assert (err <= bound).all(), (name, (err / bound).max())


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(cuda_lib, case):
    sla = cuda_lib
    q, k, v, do, lq, lk = make(case, seed=7)
    plan = plan_of(sla, case, grad=True)
    ref = R.prompt(q, k, v, lq, lk, case[5], do=do)
    leaves = [t.cuda().requires_grad_(True) for t in (q, k, v)]
    o = sla.prompt_attention(*leaves, plan)
    grads = torch.autograd.grad(o, leaves, do.cuda())
    assert sla.read_device_status(plan.device_bytes) == 0
    check_forward(case, o.detach(), None, ref, q, k)
    check_grads(case, grads, ref, q, k)
    # bit for bit, again
    o, lse, rest = sla.prompt_forward(*(t.detach() for t in leaves), plan, want_rest=True)
    again = sla.prompt_backward(*(t.detach() for t in leaves), o, lse, do.cuda(), plan, rest=rest)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))
    # O + rest is the float32 O: two bf16 hold 16 bits of it
    e = score_error(case[4], q, k, 1 / math.sqrt(case[4]))
    err = (o.cpu().double() + rest.cpu().double() - ref["o"]).abs()
    assert (err <= (H8 + 3 * e) * ref["o_size"] * 1.01 + 2.0 ** -15 * ref["o"].abs() + 1e-30).all()
    # without the rest the gradients hold the same bounds
    check_grads(case, sla.prompt_backward(*(t.detach() for t in leaves), o, lse, do.cuda(), plan), ref, q, k)


def test_backward_with_split_query_tiles(cuda_lib):
    """Few key tiles that many query tiles see: their sums are split and joined."""
    sla = cuda_lib
    for case in (([2500], None, 4, 1, 64, True), ([3000], [140], 2, 1, 128, False)):
        q, k, v, do, lq, lk = make(case, seed=8)
        plan = plan_of(sla, case, grad=True)
        assert plan.backward_workspace_size > 256 + plan.Tq * plan.Hq * 8  # split sums have a place of their own
        ref = R.prompt(q, k, v, lq, lk, case[5], do=do)
        o, lse = sla.prompt_forward(q.cuda(), k.cuda(), v.cuda(), plan)
        check_grads(case, sla.prompt_backward(q.cuda(), k.cuda(), v.cuda(), o, lse, do.cuda(), plan), ref, q, k)


def test_backward_against_differences(cuda_lib):
    """<grad, w> against the kernel's own central difference."""
    sla = cuda_lib
    case = ([140, 9], None, 4, 2, 64, True)
    q, k, v, do, _, _ = make(case, seed=9)
    plan = plan_of(sla, case)
    leaves = [t.cuda().requires_grad_(True) for t in (q, k, v)]
    grads = torch.autograd.grad(sla.prompt_attention(*leaves, plan), leaves, do.cuda())
    g = torch.Generator().manual_seed(10)
    with torch.no_grad():
        for i, t in enumerate(leaves):
            # a step in the direction of the gradient: a large difference against the rounding of O
            w = (grads[i].float() / grads[i].float().norm() * 8).bfloat16()
            up, down = (t + w), (t - w)
            w2 = up.double() - down.double()  # the step that bf16 leaves
            f = [(sla.prompt_attention(*(x if j == i else y for j, y in enumerate(leaves)), plan).double()
                  * do.cuda().double()).sum() for x in (up, down)]
            got, want = (f[0] - f[1]).item(), (grads[i].double() * w2).sum().item()
            # rounding of O: half-steps of both, against dO, adding like noise
            noise = 2 * H8 * (do.double().norm() * 3).item()
            assert abs(got - want) <= 0.1 * abs(want) + noise, (i, got, want)


def test_backward_keeps_sequences_apart_and_rows_behind_them(cuda_lib):
    sla = cuda_lib
    for d in (64, 128):
        case = ([70, 150, 33], None, 3, 1, d, True)
        q, k, v, do, lq, _ = make(case, seed=11)
        plan = plan_of(sla, case)
        dev = [t.cuda() for t in (q, k, v, do)]

        def grads(ts):
            o, lse = sla.prompt_forward(*ts[:3], plan)
            return sla.prompt_backward(*ts[:3], o, lse, ts[3], plan)

        want = grads(dev)
        keep = torch.ones(253, dtype=torch.bool)
        keep[70:220] = False
        bad = [t.clone() for t in dev]
        for t in bad:
            t[70:220] = float("nan")
        for a, b in zip(grads(bad), want):
            assert torch.equal(a[keep], b[keep])
        # 19 more tokens of NaN behind the last sequence; gradients land in strided rows
        long = [torch.cat([t, torch.full((19, *t.shape[1:]), float("nan"), dtype=t.dtype, device="cuda")]) for t in dev]
        o, lse = sla.prompt_forward(*long[:3], plan)
        got = sla.prompt_backward(*long[:3], o, lse, long[3], plan)
        assert all(torch.equal(a[:253], b) and (a[253:] == 0).all() for a, b in zip(got, want))
        x = torch.full((272, 3 + 1 + 1, d), 9.0, dtype=torch.bfloat16, device="cuda")
        sla.prompt_backward(*long[:3], o, lse, long[3], plan, out=(x[:, :3], x[:, 3:4], x[:, 4:]))
        assert torch.equal(x[:253], torch.cat(want, 1)) and (x[253:] == 9.0).all()


def test_backward_graph_and_shared_leaves(cuda_lib):
    sla = cuda_lib
    case = ([90, 200], None, 4, 2, 128, True)
    q, k, v, do, _, _ = make(case, seed=12)
    q, k, v, do = q.cuda(), k.cuda(), v.cuda(), do.cuda()
    plan = plan_of(sla, case)
    o, lse = sla.prompt_forward(q, k, v, plan)
    want = sla.prompt_backward(q, k, v, o, lse, do, plan)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o2, lse2 = sla.prompt_forward(q, k, v, plan)
        got = sla.prompt_backward(q, k, v, o2, lse2, do, plan)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # k and v the same tensor, and broadcast heads: gradients add up
    kv = k.clone().requires_grad_(True)
    (dkv,) = torch.autograd.grad(sla.prompt_attention(q, kv, kv, plan), kv, do)
    o, lse, rest = sla.prompt_forward(q, k, k, plan, want_rest=True)
    _, dk, dv = sla.prompt_backward(q, k, k, o, lse, do, plan, rest=rest)
    assert torch.equal(dkv, dk + dv)
    one = k[:, :1].float().requires_grad_(True)
    (d1,) = torch.autograd.grad(sla.prompt_attention(q, one.bfloat16().expand(-1, 2, -1), v, plan), one, do)
    assert d1.shape == one.shape and torch.isfinite(d1).all()
    # plans for serving refuse the backward
    serve = sla.prompt_plan([3], [40], Hq=4, Hkv=2, d=128)
    with pytest.raises(ValueError):
        sla.prompt_attention(q[:3].clone().requires_grad_(True), k[:40], v[:40], serve)


def broken(plan, table, index, **fields):
    """The plan's device copy with some words of one of its items changed."""
    from tests import test_prompt as T

    h = T.read(plan)[0]
    names = dict(items=T.ITEM, rows=T.ITEM, joins=T.JOIN, keys=T.KEYS, kjoins=T.KJOIN)[table]
    words = plan.device_bytes.view(torch.int32)
    for name, value in fields.items():
        words[getattr(h, table) // 4 + index * len(names) + names.index(name)] = value
    return h


FORWARD_FAULTS = [("items", dict(head=2)), ("items", dict(head=-1)), ("items", dict(slot=0)), ("items", dict(nq=0)),
                  ("items", dict(q0=300)), ("items", dict(lk=1000))]


@pytest.mark.parametrize("table,fields", FORWARD_FAULTS, ids=str)
@pytest.mark.parametrize("lens,d", [([300], 64), ([129] * 700, 128)])
def test_items_out_of_range_are_refused_in_the_forward(cuda_lib, table, fields, lens, d):
    """An item whose rows, keys, head or slot are not the plan's is skipped and reported: its own CTA's
    first item, and one that a CTA takes behind another (700 sequences: several items to an SM)."""
    sla = cuda_lib
    case = (lens, None, 4, 2, d, True)
    q, k, v, _, lq, _ = make(case, seed=20)
    want = sla.prompt_attention(q.cuda(), k.cuda(), v.cuda(), plan_of(sla, case))
    plan = plan_of(sla, case)
    from tests.test_prompt import read

    items = read(plan)[1]
    at = len(items) - 1
    fields = {n: sum(lq) if n == "q0" else x for n, x in fields.items()}
    h = broken(plan, table, at, **fields)
    assert h.n_slots == 0 and (len(items) > 4 * 148) == (len(lens) > 1)
    out = torch.full_like(want, 7.0)
    sla.prompt_forward(q.cuda(), k.cuda(), v.cuda(), plan, out=out)
    assert sla.read_device_status(plan.device_bytes) == sla.SLA_ERR_DEVICE_CHECK
    it = items[at]
    rows, heads = slice(it["q0"], it["q0"] + it["nq"]), slice(it["head"] * 2, it["head"] * 2 + 2)
    assert (out[rows, heads] == 7.0).all()
    if len(lens) == 1:  # (behind a bad item a CTA takes no more: those run as blocks of their own)
        want[rows, heads] = 7.0
        assert torch.equal(out, want)


@pytest.mark.parametrize("table,fields", [("items", dict(slot=1 << 20)), ("items", dict(head=1)), ("joins", dict(head=1)),
                                          ("joins", dict(first=1)), ("joins", dict(n=1 << 20)), ("joins", dict(q0=-1))], ids=str)
def test_pieces_out_of_range_are_refused(cuda_lib, table, fields):
    sla = cuda_lib
    case = ([1], [9000], 8, 1, 128, True)
    q, k, v, _, _, _ = make(case, seed=21)
    plan = plan_of(sla, case)
    assert broken(plan, table, 0, **fields).n_joins == 1
    out = torch.full((1, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(plan.workspace_size, dtype=torch.uint8, device="cuda")  # a piece that is not written: weight 1, zeros
    sla.prompt_forward(q.cuda(), k.cuda(), v.cuda(), plan, out=out, workspace=ws)
    assert sla.read_device_status(plan.device_bytes) == sla.SLA_ERR_DEVICE_CHECK
    assert (out == 7.0).all() == (table == "joins")


@pytest.mark.parametrize("table,fields", [("keys", dict(head=2)), ("keys", dict(slot=1 << 20)), ("keys", dict(t1=1000)),
                                          ("keys", dict(t0=-1)), ("keys", dict(block=100)), ("rows", dict(head=2)), ("rows", dict(head=-1)),
                                          ("rows", dict(nq=0)), ("kjoins", dict(head=2)), ("kjoins", dict(first=-1)),
                                          ("kjoins", dict(n=1 << 20)), ("kjoins", dict(row=-1)), ("kjoins", dict(row=2500))], ids=str)
def test_items_out_of_range_are_refused_in_the_backward(cuda_lib, table, fields):
    from tests.test_prompt import read

    sla = cuda_lib
    case = ([2500], None, 4, 2, 64, True)
    q, k, v, do, _, _ = make(case, seed=22)
    q, k, v, do = q.cuda(), k.cuda(), v.cuda(), do.cuda()
    good = plan_of(sla, case)
    o, lse = sla.prompt_forward(q, k, v, good)
    ws = torch.zeros(good.backward_workspace_size, dtype=torch.uint8, device="cuda")
    want = sla.prompt_backward(q, k, v, o, lse, do, good, workspace=ws)
    plan = plan_of(sla, case)
    h = broken(plan, table, 0, **fields)
    assert h.n_kjoins > 0
    got = [torch.full_like(t, 7.0) for t in (q, k, v)]
    sla.prompt_backward(q, k, v, o, lse, do, plan, out=tuple(got), workspace=ws)
    assert sla.read_device_status(plan.device_bytes) == sla.SLA_ERR_DEVICE_CHECK
    _, _, _, keys, kjoins, rows = read(good)
    if table == "rows":
        it = rows[0]
        want[0][it["q0"]:it["q0"] + it["nq"], it["head"] * 2:it["head"] * 2 + 2] = 7.0
    elif table == "kjoins":
        it = kjoins[0]
        for t in want[1:]:
            t[it["row"]:it["row"] + it["nk"], it["head"]] = 7.0
    elif keys[0]["slot"] < 0:
        it = keys[0]
        for t in want[1:]:
            t[it["block"] * 128:it["block"] * 128 + 128, it["head"]] = 7.0
    # (a split key tile's piece that is skipped leaves what the call before left in its slot: the same sums)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("d", [64, 128])
def test_one_infinite_score_makes_its_rows_nan(cuda_lib, d):
    """Whatever column of a block the key stands in: softmax of an infinite score is NaN, not infinity."""
    sla = cuda_lib
    case = ([40], None, 2, 1, d, False)
    q, k, v, _, _, _ = make(case, seed=18)
    q[..., 0] = 1.0
    plan = plan_of(sla, case)
    for j in range(32):
        bad = k.clone()
        bad[j, 0, 0] = math.inf
        o, lse = sla.prompt_forward(q.cuda(), bad.cuda(), v.cuda(), plan)
        assert o.isnan().all() and not torch.isfinite(lse).any(), j


@pytest.mark.parametrize("d", [64, 128])
def test_a_nan_query_makes_its_keys_gradients_nan(cuda_lib, d):
    """dV of every key that the query sees, whatever column of the tile it stands in, and of no other."""
    sla = cuda_lib
    case = ([200], None, 1, 1, d, True)
    q, k, v, do, _, _ = make(case, seed=19)
    plan = plan_of(sla, case)

    def grads(q):
        o, lse = sla.prompt_forward(q, k.cuda(), v.cuda(), plan)
        return sla.prompt_backward(q, k.cuda(), v.cuda(), o, lse, do.cuda(), plan)

    clean = grads(q.cuda())
    for r in [*range(100, 116), 0, 127, 128, 199]:
        bad = q.cuda()
        bad[r] = math.nan
        dq, dk, dv = grads(bad)
        assert dq[r].isnan().all() and dk[:r + 1].isnan().all() and dv[:r + 1].isnan().all(), r
        assert torch.equal(dv[r + 1:], clean[2][r + 1:]), r


def scores_size(q, k, lq, lk, scale):
    """Per query row: the largest scale sum_i |q_i k_i| over its sequence's keys (what a score's rounding is relative to)."""
    out = torch.zeros(q.shape[:2], dtype=torch.float64)
    a = b = 0
    for n, m in zip(lq, lk):
        for h in range(q.shape[1]):
            if n and m:
                kh = k[b:b + m, h // (q.shape[1] // k.shape[1])].double().abs()
                out[a:a + n, h] = (q[a:a + n, h].double().abs() @ kh.t()).amax(-1) * scale
        a, b = a + n, b + m
    return out


def lse_bound(case, q, k, lse, scale=None):
    """Row by row. A score: float32 sums of d products, 2 d + 4 half-steps of its own size. The
    exponentials: the hardware's 2^-22 of each; at d = 64 a quarter of them by a cubic, 1.0e-4. Their
    sum: eight interleaved chains over the keys, half a step an addition, and a few to join them
    (split keys: fewer). log2 and the product with ln 2: 2^-22 of the result each."""
    lq, lk, _, _, d, _ = case
    lk = lq if lk is None else lk
    e = (2 * d + 4) * R.EPS32 * scores_size(q, k, lq, lk, 1 / math.sqrt(d) if scale is None else scale)
    return e + (1.05e-4 if d == 64 else 0.0) + 2.0 ** -22 + (max(lk) / 8 + 24) * R.EPS32 + 2.0 ** -21 * (1 + lse.abs())


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_lse_row_by_row(cuda_lib, case):
    sla = cuda_lib
    q, k, v, _, lq, lk = make(case, seed=15)
    _, lse = sla.prompt_forward(q.cuda(), k.cuda(), v.cuda(), plan_of(sla, case))
    want = R.prompt(q, k, v, lq, lk, case[5])["lse"]
    got, fin = lse.cpu().double(), want != -math.inf
    assert torch.equal(got == -math.inf, ~fin)
    err, bound = (got - want).abs()[fin], lse_bound(case, q, k, want)[fin]
    assert (err <= bound).all(), (err / bound).max()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tokens", [1, 3])
def test_every_key_at_the_edge_of_a_piece_counts_once(cuda_lib, d, tokens):
    """Long rows whose keys are split: query head i looks for one key, in turn the first and the
    last of each piece and the sequence's last. Left out, O is another row of V; counted twice,
    lse is off by ln 2."""
    from tests.test_prompt import read

    sla = cuda_lib
    n, H = 9000 + 37, 32
    case = ([tokens], [n], H, 1, d, False)
    plan = plan_of(sla, case)
    items = read(plan)[1]
    assert any(it["slot"] >= 0 for it in items)
    edges = sorted({min(n, e) - s for it in items for e, s in ((it["b0"] * 128, 0), (it["b1"] * 128, 1))} | {n - 1})
    g = torch.Generator().manual_seed(16)
    v = torch.randn(n, 1, d, generator=g).bfloat16()
    for at in range(0, len(edges), H):
        want = edges[at:at + H]
        # key want[i] is 32 along axis i, query head i 16 sqrt(d) / 16 along it: a score of 32 against 0
        q, k = torch.zeros(tokens, H, d), torch.zeros(n, 1, d)
        for i, j in enumerate(want):
            q[:, i, i], k[j, 0, i] = math.sqrt(d), 32.0
        q, k = q.bfloat16(), k.bfloat16()
        o, lse = sla.prompt_forward(q.cuda(), k.cuda(), v.cuda(), plan)
        ref = R.prompt(q, k, v, [tokens], [n], False)
        check_forward(case, o, None, ref, q, k)
        err = (lse.cpu().double() - ref["lse"]).abs()
        assert (err <= lse_bound(case, q, k, ref["lse"])).all(), err.max()
        # one key carries all but n e^-30 of the row
        for i, j in enumerate(want):
            assert ((o[:, i].cpu().float() - v[j, 0].float()).abs() <= 2.0 ** -8 * v[j, 0].float().abs() + 1e-6).all(), j


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", [([700], None, 2, 1, 64), ([1], [9000], 8, 1, 64), ([1], [9000], 8, 1, 128), ([3000], None, 8, 8, 64)],
                         ids=str)
def test_growing_maxima_in_every_form(cuda_lib, case, causal):
    """The running maximum raised in every block, where heads are of 64 (whose scores have columns
    of their own), where keys are split, and with one and two tiles to an item."""
    sla = cuda_lib
    case = (*case, causal)
    lk = case[1] or case[0]
    q, k, v, _, lq, lk = make(case, seed=17)
    q[..., 0], k[:, :, 0] = 8.0, torch.linspace(120.0, 0.0, lk[0])[:, None].bfloat16()
    o, lse = sla.prompt_forward(q.cuda(), k.cuda(), v.cuda(), plan_of(sla, case))
    ref = R.prompt(q, k, v, lq, lk, causal)
    check_forward(case, o, lse, ref, q, k)
    assert ((lse.cpu().double() - ref["lse"]).abs() <= lse_bound(case, q, k, ref["lse"])).all()


@pytest.mark.parametrize("case", [([3000], None, 8, 8, 64, True), ([3000], None, 8, 8, 128, True), ([300], None, 2, 2, 64, True),
                                  ([1], [9000], 2, 2, 64, True), ([4], [9000], 2, 2, 128, True)], ids=IDS)
def test_one_infinite_score_in_every_form(cuda_lib, case):
    """One and two tiles to an item, whole and split keys: the rows that see the key are NaN (their lse
    too), the others as they were."""
    sla = cuda_lib
    q, k, v, _, lq, lk = make(case, seed=23)
    q[..., 0] = 1.0
    plan = plan_of(sla, case)
    want = sla.prompt_forward(q.cuda(), k.cuda(), v.cuda(), plan)
    first = max(0, lk[0] - 2000)
    for j in range(first, first + 16):
        bad = k.clone()
        bad[j, 0, 0] = math.inf
        see = torch.zeros(case[2], sum(lq), dtype=torch.bool)
        see[0] = torch.arange(lq[0]) + lk[0] - lq[0] >= j
        o, lse = (t.cpu() for t in sla.prompt_forward(q.cuda(), bad.cuda(), v.cuda(), plan))
        assert o.transpose(0, 1)[see].isnan().all() and lse.t()[see].isnan().all(), j
        assert torch.equal(o.transpose(0, 1)[~see], want[0].cpu().transpose(0, 1)[~see])
        assert torch.equal(lse.t()[~see], want[1].cpu().t()[~see])
