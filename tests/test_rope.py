"""Rotary positions and query / key norms, without a GPU: the frequency tables,
the reference's gradients against differences, and the calls that are refused."""

import ctypes
import math
from fractions import Fraction

import pytest
import torch

import sparse_linear_attention_pool_b200 as sla
from sparse_linear_attention_pool_b200 import build as sla_build
from sparse_linear_attention_pool_b200.rotary import rope_frequencies
from tests import operator_reference as R


@pytest.fixture(scope="module")
def lib():
    sla_build.build()
    return sla.load()


def test_frequencies_and_scalings():
    f, axis, gain = rope_frequencies(8)
    assert axis == [0] * 4 and gain == 1.0
    assert f == pytest.approx([1.0, 0.1, 0.01, 0.001], rel=1e-14)
    f, _, _ = rope_frequencies(8, scaling="linear", factor=4.0)
    assert f == pytest.approx([0.25, 0.025, 0.0025, 0.00025], rel=1e-14)
    # ntk: the slowest pair is stretched by the factor, the fastest is kept
    f, _, _ = rope_frequencies(8, scaling="ntk", factor=4.0)
    assert f[0] == 1.0 and f[-1] == pytest.approx(0.001 / 4.0, rel=1e-12)
    # yarn: pairs that turn more than 32 times over the original length keep their frequency
    plain, _, _ = rope_frequencies(128)
    f, _, gain = rope_frequencies(128, scaling="yarn", factor=8.0, original=4096)
    assert gain == pytest.approx(0.1 * math.log(8.0) + 1.0)
    for x, y in zip(plain, f):
        turns = 4096 * x / (2 * math.pi)
        if turns > 40:
            assert y == x
        elif turns < 0.8:
            assert y == pytest.approx(x / 8.0, rel=1e-14)
        else:
            assert x / 8.0 * (1 - 1e-12) <= y <= x
    f, axis, _ = rope_frequencies(128, sections=(22, 21, 21))
    assert axis == [0] * 22 + [1] * 21 + [2] * 21
    assert f[0] == f[22] == f[43] == 1.0 and f[23] == pytest.approx(10000.0 ** (-1 / 21))
    assert rope_frequencies(0) == ([], [], 1.0)


@pytest.mark.parametrize("pos", [0, 1, 131071, 10 ** 7, -5, 2 ** 40])
def test_turn_table_gives_the_angle_at_any_position(pos):
    """p turns mod 2^64, as the kernel forms it, against exact rational arithmetic."""
    table = sla.rope_table(64, device="cpu", freqs=[0.37 ** i * (7.3 if i == 0 else 1.0) for i in range(32)])
    two_pi = Fraction(2 * math.pi)  # the float64 that the table divides by
    for f, t in zip(table.freqs, table.turns.tolist()):
        got = Fraction((t * pos) % (1 << 64), 1 << 64)
        want = (Fraction(f) / two_pi * pos) % 1
        off = abs(got - want)
        # the quotient f / 2 pi is rounded to float64 once: half a step of it, times p
        assert min(off, 1 - off) <= abs(pos) * (Fraction(f) / two_pi * Fraction(1, 1 << 53) + Fraction(1, 1 << 64))


def test_table_refusals():
    for kw in (dict(rot_dim=7), dict(rot_dim=-2), dict(rot_dim=8, sections=(1, 1)), dict(rot_dim=8, sections=(5, -1)),
               dict(rot_dim=8, scaling="other"), dict(rot_dim=8, theta=0.0), dict(rot_dim=8, scaling="linear", factor=0.0),
               dict(rot_dim=8, scaling="yarn", factor=2.0), dict(rot_dim=8, layout="both"),
               dict(rot_dim=8, freqs=[1.0]), dict(rot_dim=8, freqs=[1.0, 2.0, float("inf"), 0.0]),
               dict(rot_dim=8, freqs=[1.0] * 4, theta=5.0), dict(rot_dim=8, gain=float("nan"))):
        with pytest.raises(ValueError):
            sla.rope_table(device="cpu", **kw)


def test_reference_gradients_against_differences():
    torch.manual_seed(0)
    x, w, dy = torch.randn(2, 3, 5, 12).double(), torch.randn(12).double(), torch.randn(2, 3, 5, 12).double()
    ang = torch.rand(5, 4).double() * 6
    for layout in ("half", "interleaved"):
        def f(x_, w_):
            return (R.rotate(R.rms_norm(x_, w_, 1e-3)[0], ang, 8, layout, 1.3) * dy).sum()

        dx, dw, _, _ = R.norm_rope_grads(x, w, 1e-3, dy, ang, 8, layout, 1.3)
        h = 1e-5
        for t, g in ((x, dx), (w, dw)):
            for _ in range(3):
                v = torch.randn_like(t)
                up, down = (f(x + s * h * v, w) if t is x else f(x, w + s * h * v) for s in (1, -1))
                # central difference: error h^2 f''' / 6 ~ 1e-9, rounding 1e-16 / h ~ 1e-11 per unit
                assert (up - down) / (2 * h) == pytest.approx((g * v).sum().item(), abs=1e-6)


def heads(base=0x10000, H=2, sb=0, sh=128, sn=256):
    return sla.Heads(base, H, sb, sh, sn)


def spec(**kw):
    s = sla.RopeSpec(0x1000, None, None, 0, 0, 0, 1.0, 32, 128, 1, 1)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


@pytest.mark.parametrize("what,code", [
    (dict(B=0), "INVALID_ARG"), (dict(N=0), "INVALID_ARG"), (dict(d=0), "INVALID_ARG"), (dict(dtype=3), "INVALID_ARG"),
    (dict(d=127), "UNSUPPORTED"), (dict(d=258), "UNSUPPORTED"), (dict(B=2 ** 20, N=2 ** 11), "UNSUPPORTED"),
    (dict(x=None), "INVALID_ARG"), (dict(y=None), "INVALID_ARG"), (dict(rope=None), "INVALID_ARG"),
    (dict(x=heads(base=None)), "INVALID_ARG"), (dict(x=heads(H=0)), "INVALID_ARG"), (dict(x=heads(sn=-1)), "INVALID_ARG"),
    (dict(y=heads(H=3)), "INVALID_ARG"), (dict(x=heads(base=0x10001)), "ALIGNMENT"),
    (dict(x=heads(base=0x10002), dtype=2), "ALIGNMENT"),
    (dict(y=heads(sn=0)), "INVALID_ARG"), (dict(y=heads(sh=0)), "INVALID_ARG"), (dict(y=heads(sn=130)), "INVALID_ARG"),
    (dict(y=heads(sh=64)), "INVALID_ARG"), (dict(B=2), "INVALID_ARG"),  # y's batches in the same place
    (dict(rope=spec(rot_dim=130)), "INVALID_ARG"), (dict(rope=spec(rot_dim=3)), "INVALID_ARG"),
    (dict(rope=spec(layout=2)), "INVALID_ARG"), (dict(rope=spec(turns=None)), "INVALID_ARG"),
    (dict(rope=spec(n_axes=0)), "INVALID_ARG"), (dict(rope=spec(gain=float("inf"))), "INVALID_ARG"),
    (dict(rope=spec(turns=0x1004)), "ALIGNMENT"), (dict(rope=spec(pos=0x2000, pos_bits=16)), "INVALID_ARG"),
    (dict(rope=spec(pos=0x2002)), "ALIGNMENT"), (dict(rope=spec(pos=0x2000, pos_n=-1)), "INVALID_ARG"),
])
def test_rope_refuses_on_the_host(lib, what, code):
    """Fake device addresses: every call is refused before anything is enqueued."""
    a = dict(x=heads(), y=heads(), B=1, N=7, d=128, dtype=0, rope=spec())
    a.update(what)
    st = lib.sla_rope(a["x"], a["y"], a["B"], a["N"], a["d"], a["dtype"], a["rope"], 0, None)
    assert st == getattr(sla, "SLA_ERR_" + code)


@pytest.mark.parametrize("what,code", [
    (dict(k=None), "INVALID_ARG"), (dict(wq=None), "INVALID_ARG"), (dict(eps=-1.0), "INVALID_ARG"),
    (dict(eps=float("nan")), "INVALID_ARG"), (dict(wk=0x3001), "ALIGNMENT"), (dict(wk=0x3002, w_f32=1), "ALIGNMENT"),
    (dict(yk=heads(H=3)), "INVALID_ARG"), (dict(yk=heads(sn=0)), "INVALID_ARG"), (dict(d=300), "UNSUPPORTED"),
    (dict(rope=spec(rot_dim=-2)), "INVALID_ARG"),
])
def test_qk_norm_rope_refuses_on_the_host(lib, what, code):
    a = dict(q=heads(), k=heads(), wq=0x3000, wk=0x3100, w_f32=0, eps=1e-6, yq=heads(), yk=heads(), B=1, N=7, d=128,
             dtype=0, rope=spec())
    a.update(what)
    st = lib.sla_qk_norm_rope(a["q"], a["k"], a["wq"], a["wk"], a["w_f32"], a["eps"], a["yq"], a["yk"], a["B"], a["N"],
                              a["d"], a["dtype"], a["rope"], None)
    assert st == getattr(sla, "SLA_ERR_" + code)
    # the backward refuses the same, and its own
    st = lib.sla_qk_norm_rope_backward(a["q"], a["k"], a["wq"], a["wk"], a["w_f32"], a["eps"], heads(), heads(),
                                       a["yq"], a["yk"], None, None, a["B"], a["N"], a["d"], a["dtype"], a["rope"],
                                       0x100000, 1 << 30, None)
    assert st == getattr(sla, "SLA_ERR_" + code)


def test_backward_workspace(lib):
    need = lib.sla_qk_norm_rope_backward_workspace_size(1, 1000, 4, 2, 128)
    assert need > 0
    assert lib.sla_qk_norm_rope_backward_workspace_size(0, 1000, 4, 2, 128) == 0
    assert lib.sla_qk_norm_rope_backward_workspace_size(1, 1000, 0, 2, 128) == 0
    h = heads()

    def call(ws, n, dwq=None, dwk=None, dyq=h):
        return lib.sla_qk_norm_rope_backward(h, h, 0x3000, 0x3100, 0, 1e-6, dyq, h, h, h, dwq, dwk, 1, 7, 128, 0, None,
                                             ws, n, None)

    small = lib.sla_qk_norm_rope_backward_workspace_size(1, 7, 2, 2, 128)
    assert call(None, 1 << 30) == sla.SLA_ERR_WORKSPACE
    assert call(0x100008, 1 << 30) == sla.SLA_ERR_WORKSPACE
    assert call(0x100000, small - 1) == sla.SLA_ERR_WORKSPACE
    assert call(0x100000, 1 << 30, dwq=0x4000) == sla.SLA_ERR_INVALID_ARG
    assert call(0x100000, 1 << 30, dwq=0x4001, dwk=0x4000) == sla.SLA_ERR_ALIGNMENT
    assert call(0x100000, 1 << 30, dyq=heads(H=3)) == sla.SLA_ERR_INVALID_ARG


def test_binding_refuses_cpu_tensors():
    table = sla.rope_table(8, device="cpu")
    x = torch.zeros(1, 1, 4, 8, dtype=torch.bfloat16)
    for bad in (x, x[0, 0]):
        with pytest.raises(ValueError):
            sla.rope(bad, table)
    with pytest.raises(ValueError):
        sla.qk_norm_rope(x, x, torch.ones(8), torch.ones(8), table)


def test_struct_sizes_match_the_header():
    assert ctypes.sizeof(sla.Heads) == 40 and ctypes.sizeof(sla.RopeSpec) == 72


def test_yarn_scales_cos_and_sin_only_for_longer_contexts():
    """The factor on cos and sin is 0.1 ln(factor) + 1 above 1, and 1 where nothing is stretched."""
    for factor, gain in ((8.0, 0.1 * math.log(8.0) + 1.0), (1.0, 1.0), (0.5, 1.0), (0.01, 1.0)):
        f, _, g = rope_frequencies(128, scaling="yarn", factor=factor, original=4096)
        assert g == pytest.approx(gain, rel=1e-15)
        assert sla.rope_table(128, scaling="yarn", factor=factor, original=4096, device="cpu").gain == g


# 2 pi to 60 digits
TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459")


def test_turn_table_is_rounded_once():
    """Every entry is 2^64 f / 2 pi to the nearest whole number, of the float64 f and of pi itself."""
    for f in ([0.37 ** i * (7.3 if i == 0 else 1.0) for i in range(32)], rope_frequencies(64)[0],
              [-1.0, 0.0, 1e-300, 2.0 ** -60, 123456.789, -1e15, 1e300, 0.5]):
        table = sla.rope_table(2 * len(f), device="cpu", freqs=f)
        for x, t in zip(f, table.turns.tolist()):
            off = abs(Fraction(t) - Fraction(x) / TWO_PI * (1 << 64)) % (1 << 64)
            # (the digits of pi above are off by 1e-61 of it: at 1e300 the turns' fraction is beyond them)
            assert abs(x) > 1e30 or min(off, (1 << 64) - off) <= Fraction(1, 2) + Fraction(1, 1 << 40), x


def test_a_stream_of_another_device_is_refused():
    """The call would run on the tensors' device, in no order with that stream."""
    class Stream:
        cuda_stream, device = 1, torch.device("cuda", 1)

    from sparse_linear_attention_pool_b200.rotary import on_stream

    with pytest.raises(ValueError, match="stream"):
        on_stream(Stream(), torch.device("cuda", 0))
    x, w = torch.zeros(4, 1, 64, dtype=torch.bfloat16), torch.ones(64)
    table, plan = sla.rope_table(64, device="cpu"), sla.prompt_plan([4], Hq=1, Hkv=1, d=64, device="cpu")
    for call in (lambda s: sla.rope(x, table, stream=s), lambda s: sla.qk_norm_rope(x, x, w, w, stream=s),
                 lambda s: sla.qk_norm_rope_backward(x, x, w, w, x, x, stream=s),
                 lambda s: sla.prompt_attention(x, x, x, plan, stream=s), lambda s: sla.prompt_forward(x, x, x, plan, stream=s),
                 lambda s: sla.prompt_backward(x, x, x, x, torch.zeros(4, 1), x, plan, stream=s)):
        with pytest.raises(ValueError, match="stream"):
            call(Stream())
