"""Packed prompt attention without a GPU: the plan's work lists, the reference's
gradients against differences, and the calls that are refused."""

import ctypes
import random

import pytest
import torch

import sparse_linear_attention_pool_b200 as sla
from sparse_linear_attention_pool_b200 import build as sla_build
from tests import operator_reference as R


class Plan(ctypes.Structure):
    """Mirror of the plan's header (csrc/prompt.cuh)."""
    _fields_ = [("status", ctypes.c_int), ("magic", ctypes.c_uint)] + \
        [(n, ctypes.c_int) for n in ("n_seq", "Hq", "Hkv", "G", "d", "causal")] + \
        [("scale", ctypes.c_float), ("tiles", ctypes.c_int), ("few", ctypes.c_int), ("Tq", ctypes.c_longlong), ("Tk", ctypes.c_longlong)] + \
        [(n, ctypes.c_int) for n in ("n_items", "n_joins", "n_slots", "join_rows", "join_parts", "n_keys", "n_kjoins", "n_kslots", "n_rows",
                                     "row_tiles")] + \
        [(n, ctypes.c_ulonglong) for n in ("items", "joins", "keys", "kjoins", "rows", "total")]


ITEM = ("q0", "nq", "k0", "lk", "pos0", "head", "b0", "b1", "slot", "_1", "_2", "_3")
JOIN = ("q0", "nq", "head", "first", "n", "_1", "_2", "_3")
KEYS = ("k0", "lk", "q0", "lq", "block", "head", "t0", "t1", "slot", "_1", "_2", "_3")
KJOIN = ("row", "nk", "head", "first", "n", "_1", "_2", "_3")


def read(plan):
    raw = plan.host.raw
    h = Plan.from_buffer_copy(raw)

    def table(at, n, names):
        a = (ctypes.c_int * (n * len(names))).from_buffer_copy(raw, at)
        return [dict(zip(names, a[i * len(names):(i + 1) * len(names)])) for i in range(n)]

    return (h, table(h.items, h.n_items, ITEM), table(h.joins, h.n_joins, JOIN), table(h.keys, h.n_keys, KEYS),
            table(h.kjoins, h.n_kjoins, KJOIN), table(h.rows, h.n_rows, ITEM))


@pytest.fixture(scope="module")
def lib():
    sla_build.build()
    return sla.load()


def ceil(a, b):
    return -(-a // b)


CASES = [([1], None, 1, 1, True), ([7, 0, 300], None, 6, 2, True), ([1] * 8, [32768, 1025, 8000, 20001, 513, 16384, 4099, 65], 32, 8, True),
         ([5000], None, 4, 1, True), ([2500], None, 1, 1, False), ([130, 7], [60, 0], 2, 1, True), ([50], [9000], 65, 1, True),
         ([4096, 777, 8191, 1530], None, 32, 8, True), ([3, 2], [0, 0], 2, 2, False)]
rng = random.Random(1)
CASES += [([rng.randint(0, 600) + 1 for _ in range(rng.randint(1, 6))], None, g * h, h, rng.random() < 0.7)
          for g, h in ((1, 3), (3, 2), (8, 1), (5, 4))]


@pytest.mark.parametrize("lq,lk,Hq,Hkv,causal", CASES)
def test_plan_covers_every_row_and_key_once(lib, lq, lk, Hq, Hkv, causal):
    plan = sla.prompt_plan(lq, lk, Hq=Hq, Hkv=Hkv, d=64, causal=causal, grad=True, device="cpu")
    lk = lq if lk is None else lk
    h, items, joins, keys, kjoins, rows = read(plan)
    G = Hq // Hkv
    tpt = 128 // G
    assert (h.status, h.Hq, h.Hkv, h.G, h.Tq, h.Tk) == (0, Hq, Hkv, G, sum(lq), sum(lk))
    lens = [(ctypes.c_int32 * len(x))(*x) for x in (lq, lk)]
    assert h.total == len(plan.host.raw) <= lib.sla_prompt_plan_size(sla.PromptParams(
        len(lq), ctypes.addressof(lens[0]), ctypes.addressof(lens[1]), Hq, Hkv, 64, int(causal), 1, 0.0))

    def seen_blocks(pos):
        return ceil(max(0, min(pos + 1, lk_s)), 128) if causal else ceil(lk_s, 128)

    # forward and dQ items: every (token, key head) belongs to items that read all its key blocks, once
    for table, tiles in ((items, h.tiles), (rows, h.row_tiles)):
        at = {}
        for it in table:
            assert 0 <= it["q0"] and it["q0"] + it["nq"] <= h.Tq and 1 <= it["nq"] <= tiles * tpt
            at.setdefault((it["q0"], it["head"]), []).append(it)
        cost = [it["b1"] - it["b0"] for it in table]
        assert cost == sorted(cost, reverse=True)
        q0 = k0 = 0
        for lq_s, lk_s in zip(lq, lk):
            for head in range(Hkv):
                t = 0
                while t < lq_s:
                    group = sorted(at.pop((q0 + t, head)), key=lambda x: x["b0"])
                    nq = group[0]["nq"]
                    end = 0
                    for it in group:
                        assert (it["nq"], it["k0"], it["lk"], it["pos0"]) == (nq, k0, lk_s, lk_s - lq_s + t)
                        assert it["b0"] == end
                        end = it["b1"]
                    assert end == seen_blocks(lk_s - lq_s + t + nq - 1)
                    assert (len(group) == 1) == (group[0]["slot"] < 0)
                    t += nq
                assert t == lq_s
            q0, k0 = q0 + lq_s, k0 + lk_s
        assert not at
    # every slot is written once and joined once
    slots = sorted(it["slot"] for it in items if it["slot"] >= 0)
    assert slots == list(range(h.n_slots)) == sorted(s for j in joins for s in range(j["first"], j["first"] + j["n"]))
    by_slot = {it["slot"]: it for it in items}
    for j in joins:
        assert all((by_slot[s]["q0"], by_slot[s]["nq"], by_slot[s]["head"]) == (j["q0"], j["nq"], j["head"])
                   for s in range(j["first"], j["first"] + j["n"]))
    # key items: every key tile, over the query tiles that see it
    at = {}
    for it in keys:
        at.setdefault((it["k0"] + it["block"] * 128, it["head"]), []).append(it)
    q0 = k0 = 0
    for lq_s, lk_s in zip(lq, lk):
        for b in range(ceil(lk_s, 128)):
            for head in range(Hkv):
                group = sorted(at.pop((k0 + b * 128, head)), key=lambda x: x["t0"])
                first = max(0, b * 128 - (lk_s - lq_s)) if causal else 0
                tiles = ceil(lq_s, tpt)
                assert group[0]["t0"] == min(tiles, first // tpt) and group[-1]["t1"] == tiles
                for x, y in zip(group, group[1:]):
                    assert x["t1"] == y["t0"]
                assert all((x["k0"], x["lk"], x["q0"], x["lq"]) == (k0, lk_s, q0, lq_s) for x in group)
                assert (len(group) == 1) == (group[0]["slot"] < 0)
        q0, k0 = q0 + lq_s, k0 + lk_s
    assert not at
    slots = sorted(it["slot"] for it in keys if it["slot"] >= 0)
    assert slots == list(range(h.n_kslots)) == sorted(s for j in kjoins for s in range(j["first"], j["first"] + j["n"]))
    need = lib.sla_prompt_workspace_size(plan.host)
    assert (need > 0) == (h.n_slots > 0)
    assert lib.sla_prompt_backward_workspace_size(plan.host) >= h.Tq * Hq * 8


def test_plan_positions():
    plan = sla.prompt_plan([3, 2], [3, 7], Hq=1, Hkv=1, d=64, device="cpu")
    assert plan.positions().tolist() == [0, 1, 2, 5, 6] and plan.positions().dtype == torch.int32


def test_serving_plans_list_no_backward(lib):
    plan = sla.prompt_plan([1], [500], Hq=4, Hkv=2, d=128, device="cpu")
    h, _, _, keys, _, rows = read(plan)
    assert not keys and not rows and not plan.grad and lib.sla_prompt_backward_workspace_size(plan.host) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(Hq=3, Hkv=2), "INVALID_ARG"), (dict(Hq=0), "INVALID_ARG"), (dict(Hkv=0), "INVALID_ARG"),
    (dict(d=96), "UNSUPPORTED"), (dict(Hq=129, Hkv=1), "UNSUPPORTED"), (dict(lens_q=[0, 0]), "INVALID_ARG"),
    (dict(softmax_scale=-1.0), "INVALID_ARG"), (dict(softmax_scale=float("nan")), "INVALID_ARG"),
    (dict(lens_q=[2 ** 30, 2 ** 30]), "UNSUPPORTED"), (dict(lens_k=[2 ** 31 - 1]), "UNSUPPORTED"),
    (dict(lens_q=[2 ** 26], Hq=64, Hkv=64), "UNSUPPORTED"), (dict(lens_q=[1], lens_k=[2 ** 30], grad=True), "UNSUPPORTED"),
    (dict(softmax_scale=1e-35), "INVALID_ARG"),
])
def test_plan_refusals(lib, kw, code):
    a = dict(lens_q=[5], lens_k=None, Hq=4, Hkv=2, d=64, device="cpu")
    a.update(kw)
    lq, lk = a.pop("lens_q"), a.pop("lens_k")
    with pytest.raises(sla.SLAError) as e:
        sla.prompt_plan(lq, lk, **a)
    assert e.value.status == getattr(sla, "SLA_ERR_" + code)


def test_plan_argument_errors(lib):
    for lq, lk in (([], None), ([-1], None), ([5], [1, 2]), ([2 ** 31], None)):
        with pytest.raises(ValueError):
            sla.prompt_plan(lq, lk, Hq=1, Hkv=1, d=64, device="cpu")
    n = (ctypes.c_int32 * 1)(5)
    ok = dict(n_seq=1, len_q=ctypes.addressof(n), len_k=None, Hq=2, Hkv=1, d=64, causal=1, backward=0, softmax_scale=0.0)

    def status(**kw):
        return lib.sla_prompt_validate(sla.PromptParams(**{**ok, **kw}))

    assert status() == sla.SLA_OK
    for kw in (dict(n_seq=0), dict(len_q=None), dict(causal=2), dict(backward=-1)):
        assert status(**kw) == sla.SLA_ERR_INVALID_ARG
        assert lib.sla_prompt_plan_size(sla.PromptParams(**{**ok, **kw})) == 0
    assert lib.sla_prompt_validate(None) == sla.SLA_ERR_INVALID_ARG
    p = sla.PromptParams(**ok)
    size = lib.sla_prompt_plan_size(p)
    buf = (ctypes.c_longlong * (size // 8 + 1))()
    assert lib.sla_prompt_plan_used(None) == 0 == lib.sla_prompt_plan_used(buf)  # no plan there yet
    assert lib.sla_prompt_plan(p, None, size) == sla.SLA_ERR_INVALID_ARG
    assert lib.sla_prompt_plan(p, ctypes.addressof(buf) + 4, size) == sla.SLA_ERR_ALIGNMENT
    assert lib.sla_prompt_plan(p, buf, size) == sla.SLA_OK
    used = lib.sla_prompt_plan_used(buf)
    assert 0 < used <= size
    assert lib.sla_prompt_plan(p, buf, used - 1) == sla.SLA_ERR_WORKSPACE
    assert lib.sla_prompt_plan(p, buf, used) == sla.SLA_OK


def rows(base=0x10000, row=512, head=64):
    return sla.Rows(base, row, head)


CALLS = [
    (dict(plan=None), "INVALID_ARG"), (dict(size=16), "INVALID_ARG"), (dict(dev=None), "INVALID_ARG"),
    (dict(dev=0x100080), "ALIGNMENT"), (dict(q=None), "INVALID_ARG"), (dict(k=rows(base=None)), "INVALID_ARG"),
    (dict(q=rows(base=0x10008)), "ALIGNMENT"), (dict(v=rows(row=516)), "ALIGNMENT"), (dict(q=rows(head=68)), "ALIGNMENT"),
    (dict(q=rows(row=0)), "INVALID_ARG"), (dict(k=rows(head=-64)), "INVALID_ARG"), (dict(q=rows(row=1 << 39)), "UNSUPPORTED"),
]


@pytest.mark.parametrize("kw,code", CALLS + [
    (dict(o=None), "INVALID_ARG"), (dict(o=rows(row=64)), "INVALID_ARG"), (dict(o=rows(head=32)), "INVALID_ARG"),
    (dict(lse=0x2002), "ALIGNMENT"), (dict(rest=0x2008), "ALIGNMENT"),
])
def test_forward_refuses_on_the_host(lib, kw, code):
    """Fake device addresses: every call is refused before anything is enqueued."""
    plan = sla.prompt_plan([5, 90], Hq=4, Hkv=2, d=64, device="cpu")
    a = dict(q=rows(), k=rows(), v=rows(), o=rows(), lse=None, rest=None, plan=plan.host, size=len(plan.host.raw), dev=0x100000)
    a.update(kw)
    st = lib.sla_prompt_forward(a["q"], a["k"], a["v"], a["o"], a["lse"], a["rest"], a["plan"], a["size"], a["dev"], None, 0, None)
    assert st == getattr(sla, "SLA_ERR_" + code)


def test_forward_refuses_a_missing_workspace(lib):
    plan = sla.prompt_plan([1], [9000], Hq=4, Hkv=2, d=64, device="cpu")
    need = lib.sla_prompt_workspace_size(plan.host)
    assert need > 0
    r = rows()
    for ws, n in ((None, 1 << 30), (0x200080, 1 << 30), (0x200000, need - 1)):
        assert lib.sla_prompt_forward(r, r, r, r, None, None, plan.host, len(plan.host.raw), 0x100000, ws, n,
                                      None) == sla.SLA_ERR_WORKSPACE


@pytest.mark.parametrize("kw,code", CALLS + [
    (dict(o=None), "INVALID_ARG"), (dict(do=rows(base=0x10004)), "ALIGNMENT"), (dict(lse=None), "INVALID_ARG"),
    (dict(dq=rows(head=32)), "INVALID_ARG"), (dict(dk=None), "INVALID_ARG"), (dict(dv=rows(row=64)), "INVALID_ARG"),
    (dict(rest=0x2008), "ALIGNMENT"), (dict(ws=None), "WORKSPACE"), (dict(ws=0x200010), "WORKSPACE"), (dict(n=64), "WORKSPACE"),
    (dict(serve=True), "UNSUPPORTED"),
])
def test_backward_refuses_on_the_host(lib, kw, code):
    plan = sla.prompt_plan([5, 90], Hq=4, Hkv=2, d=64, grad=not kw.pop("serve", False), device="cpu")
    a = dict(q=rows(), k=rows(), v=rows(), o=rows(), lse=0x3000, rest=None, do=rows(), dq=rows(), dk=rows(), dv=rows(),
             plan=plan.host, size=len(plan.host.raw), dev=0x100000, ws=0x200000, n=1 << 30)
    a.update(kw)
    st = lib.sla_prompt_backward(a["q"], a["k"], a["v"], a["o"], a["lse"], a["rest"], a["do"], a["dq"], a["dk"], a["dv"],
                                 a["plan"], a["size"], a["dev"], a["ws"], a["n"], None)
    assert st == getattr(sla, "SLA_ERR_" + code)


def test_reference_gradients_against_differences():
    g = torch.Generator().manual_seed(0)
    q, k, v, do = (torch.randn(n, h, 8, generator=g).double() for n, h in ((9, 4), (12, 2), (12, 2), (9, 4)))
    args = ([4, 0, 5], [7, 2, 3], True)
    ref = R.prompt(q, k, v, *args, do=do)
    h = 1e-5
    for name, t in (("dq", q), ("dk", k), ("dv", v)):
        for _ in range(3):
            w = torch.randn(t.shape, generator=g).double()
            f = []
            for s in (1, -1):
                x = [y + s * h * w if y is t else y for y in (q, k, v)]
                f.append((R.prompt(*x, *args)["o"] * do).sum().item())
            assert (f[0] - f[1]) / (2 * h) == pytest.approx((ref[name] * w).sum().item(), abs=1e-6)


def test_binding_refuses_cpu_tensors():
    plan = sla.prompt_plan([5], Hq=1, Hkv=1, d=64, device="cpu")
    x = torch.zeros(5, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sla.prompt_attention(x, x, x, plan)


@pytest.mark.parametrize("kw", [dict(Hq=2 ** 32 + 4), dict(Hkv=2 ** 32 + 2), dict(d=2 ** 32 + 64), dict(Hq=2 ** 31), dict(Hq=-2 ** 33)], ids=str)
def test_plan_sizes_past_32_bits_are_refused(lib, kw):
    """No size is cut to its low 32 bits."""
    a = dict(Hq=4, Hkv=2, d=64, device="cpu")
    with pytest.raises(sla.SLAError) as e:
        sla.prompt_plan([5], **{**a, **kw})
    assert e.value.status == sla.SLA_ERR_UNSUPPORTED


@pytest.mark.parametrize("scale", [1e-46, -1e-46, 1e-31])
def test_a_scale_that_float32_rounds_to_nothing_is_refused(lib, scale):
    """It would select the default."""
    with pytest.raises(sla.SLAError) as e:
        sla.prompt_plan([5], Hq=4, Hkv=2, d=64, softmax_scale=scale, device="cpu")
    assert e.value.status == sla.SLA_ERR_INVALID_ARG


def test_binding_refuses_a_workspace_on_the_host():
    """Before anything else of the call: the library would take its address for the device's."""
    plan = sla.prompt_plan([5], Hq=1, Hkv=1, d=64, device="cpu")
    x, ws = torch.zeros(5, 1, 64, dtype=torch.bfloat16), torch.zeros(1 << 16, dtype=torch.uint8)
    lse = torch.zeros(5, 1)
    with pytest.raises(ValueError, match="workspace"):
        sla.prompt_forward(x, x, x, plan, workspace=ws)
    with pytest.raises(ValueError, match="workspace"):
        sla.prompt_backward(x, x, x, x, lse, x, plan, workspace=ws)
    w = torch.ones(64)
    with pytest.raises(ValueError, match="workspace"):
        sla.qk_norm_rope_backward(x, x, w, w, x, x, workspace=ws)
