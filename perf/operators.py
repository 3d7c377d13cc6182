"""Cases of the operators that stand before and beside the sparse-linear attention:
rotary positions, the norm of every query and key head with the rotation in the
same pass, and exact attention over packed prompts with grouped heads.

Each case names an operator ("op") and its sizes. `run` computes it either in its
plain form (elementary torch operations in 32 bits, angles in 64) or, when `own`
is true, by the calls that a user makes of the package. `exact` gives the same
outputs in 64 bits, from the definitions.

The operators:

  rope    y = x rotated by the angle p * f_i in every pair i, p the token's position
          (one position per axis; each pair belongs to one axis)
  qknorm  q, k -> rope(q / rms(q) * w_q), rope(k / rms(k) * w_k), per head
  prompt  O = softmax(scale Q K^T + mask) V for packed sequences, causal with the
          last query at the last key; query heads in groups that share a key head

With "grad" a pass is a training step: outputs and the gradients of every input.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one new token for each of 32 running sequences, at their own far positions
        dict(name="rope_token", op="rope", form="packed", T=32, H=32, d=128, rot=128, layout="half", axes=1,
             scaling="none", factor=1.0, original=0, dtype="bf16", positions="far", grad=False),
        # queries of a 480p video latent (21 x 30 x 52 tokens, 12 heads), three axes,
        # read from the projection's token-major output into the attention's head-major layout
        dict(name="rope_video", op="rope", form="heads", T=21 * 30 * 52, H=12, d=128, rot=128, layout="interleaved",
             axes=3, f=21, h=30, w=52, scaling="none", factor=1.0, original=0, dtype="bf16", positions="grid",
             grad=False),
        # a training step's rotation of half of each head, stretched to a long context, odd length
        dict(name="rope_stretched_grad", op="rope", form="packed", T=16411, H=16, d=128, rot=64, layout="half",
             axes=1, scaling="yarn", factor=8.0, original=4096, dtype="bf16", positions="packed", grad=True),
        # single tokens of 16 sequences, grouped heads
        dict(name="qknorm_token", op="qknorm", form="packed", T=16, Hq=32, Hk=8, d=128, rot=128, layout="half",
             axes=1, scaling="none", factor=1.0, original=0, dtype="bf16", positions="far", grad=False),
        # queries and keys of a 720p video latent (21 x 45 x 80 = 75600 tokens, 40 heads)
        dict(name="qknorm_video", op="qknorm", form="heads", T=21 * 45 * 80, Hq=40, Hk=40, d=128, rot=128,
             layout="interleaved", axes=3, f=21, h=45, w=80, scaling="none", factor=1.0, original=0, dtype="bf16",
             positions="grid", grad=False),
        # a training step on a packed batch, grouped heads, with the weights' gradients
        dict(name="qknorm_train", op="qknorm", form="packed", T=16381, Hq=16, Hk=4, d=128, rot=128, layout="half",
             axes=1, scaling="none", factor=1.0, original=0, dtype="bf16", positions="packed", grad=True),
        # many short prompts, small heads: latency and ragged ends
        dict(name="prompt_short", op="prompt", lens_q="1,7,64,129,33,250,2,96,128,61,17,200", lens_k="", Hq=12, Hk=4,
             d=64, causal=True, grad=False),
        # a serving batch of prompts of mixed length, eight query heads to four key heads
        dict(name="prompt_packed", op="prompt", lens_q="4096,777,8191,1530,2049,310", lens_k="", Hq=32, Hk=8, d=128,
             causal=True, grad=False),
        # one long sequence, no sharing
        dict(name="prompt_long", op="prompt", lens_q="32768", lens_k="", Hq=12, Hk=12, d=128, causal=True, grad=False),
        # single tokens over long caches
        dict(name="prompt_tokens", op="prompt", lens_q="1,1,1,1,1,1,1,1",
             lens_k="32768,1025,8000,20001,513,16384,4099,65", Hq=32, Hk=8, d=128, causal=True, grad=False),
        # training steps: a small batch with groups of three, and a long one
        dict(name="prompt_train_small", op="prompt", lens_q="511,1024,130,67", lens_k="", Hq=12, Hk=4, d=64,
             causal=True, grad=True),
        dict(name="prompt_train", op="prompt", lens_q="8192,4001,2500", lens_k="", Hq=16, Hk=4, d=128, causal=True,
             grad=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


MAX_ROPE_VALUES = 75600 * 40 * 128       # values of one tensor, the largest listed rotation
MAX_PROMPT_FLOPS = 3.2e12                # the largest listed attention


def draw(rng):
    op = rng.choice(["rope", "qknorm", "prompt", "prompt"])
    return _draw_prompt(rng) if op == "prompt" else _draw_rope(rng, op)


def _draw_rope(rng, op):
    while True:
        c = dict(op=op)
        c["grad"] = rng.random() < 0.4
        c["dtype"] = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        c["d"] = rng.choice([64, 128, 128, 80, 96, 256])
        c["layout"] = rng.choice(["half", "interleaved"])
        kind = rng.choice(["far", "packed", "grid"])
        c["positions"] = kind
        if kind == "grid":
            c["axes"] = 3
            c["f"], c["h"], c["w"] = rng.randint(1, 21), _log_int(rng, 1, 45), _log_int(rng, 1, 80)
            c["T"] = c["f"] * c["h"] * c["w"]
            c["rot"] = c["d"]
            c["scaling"], c["factor"], c["original"] = "none", 1.0, 0
        else:
            c["axes"] = 1
            c["T"] = _log_int(rng, 1, 256 if kind == "far" else 75600)
            c["rot"] = rng.choice([c["d"], c["d"], c["d"] // 2])
            c["scaling"] = rng.choice(["none", "none", "linear", "ntk", "yarn"])
            c["factor"] = 1.0 if c["scaling"] == "none" else round(rng.uniform(1.5, 16.0), 2)
            c["original"] = 4096 if c["scaling"] == "yarn" else 0
        c["form"] = rng.choice(["packed", "heads"])
        if op == "rope":
            c["H"] = rng.choice([1, 2, 5, 8, 12, 16, 32, 40])
            values = c["T"] * c["H"] * c["d"]
        else:
            c["Hk"] = rng.choice([1, 2, 3, 4, 8, 12])
            c["Hq"] = c["Hk"] * rng.choice([1, 1, 2, 3, 4, 8])
            values = c["T"] * (c["Hq"] + c["Hk"]) * c["d"]
        if values * (2.5 if c["grad"] else 1) * (2 if c["dtype"] == "fp32" else 1) <= MAX_ROPE_VALUES:
            return c


def _draw_prompt(rng):
    while True:
        c = dict(op="prompt")
        c["d"] = rng.choice([64, 128])
        c["Hk"] = rng.choice([1, 2, 4, 8, 12])
        c["Hq"] = c["Hk"] * rng.choice([1, 1, 2, 3, 4, 5, 8])
        c["causal"] = rng.random() < 0.8
        form = rng.choice(["whole", "whole", "train", "train", "tokens", "piece"])
        c["grad"] = form == "train"
        n = _log_int(rng, 1, 24)
        if form in ("whole", "train"):
            lq = [_log_int(rng, 1, rng.choice([300, 4000, 30000])) for _ in range(n)]
            lk = None
        elif form == "tokens":  # single tokens over caches
            lq, lk = [1] * n, [_log_int(rng, 1, 60000) for _ in range(n)]
        else:  # a piece of a prompt after what is in the cache already
            lq = [_log_int(rng, 1, 2000) for _ in range(n)]
            lk = [a + rng.choice([0, _log_int(rng, 1, 20000)]) for a in lq]
        c["lens_q"] = ",".join(map(str, lq))
        c["lens_k"] = "" if lk is None else ",".join(map(str, lk))
        # the plain form holds a sequence's whole score matrix of one key head's group
        most = max(a * b for a, b in zip(lq, lk or lq)) * (c["Hq"] // c["Hk"])
        if work(c)["flops"] <= MAX_PROMPT_FLOPS and most <= 32768 * 32768:
            return c


def _lens(c):
    lq = [int(x) for x in c["lens_q"].split(",")]
    lk = [int(x) for x in c["lens_k"].split(",")] if c["lens_k"] else list(lq)
    return lq, lk


def _pairs(c):
    """Query-key pairs that the mask leaves, of one head."""
    total = 0
    for a, b in zip(*_lens(c)):
        if not c["causal"]:
            total += a * b
        else:  # query i sees keys 0 .. b - a + i
            first = max(0, a - b)      # queries before this one see nothing
            m = a - first
            total += m * (b - a + first + 1) + m * (m - 1) // 2
    return total


def work(c):
    if c["op"] == "prompt":
        lq, lk = _lens(c)
        pairs = _pairs(c)
        tq, tk = sum(lq), sum(lk)
        io = 2 * c["d"] * (2 * tq * c["Hq"] + 2 * tk * c["Hk"])
        flops = 4.0 * pairs * c["Hq"] * c["d"]
        if c["grad"]:  # reads dO, writes dQ, dK, dV; five products instead of two
            io += 2 * c["d"] * (2 * tq * c["Hq"] + 2 * tk * c["Hk"])
            flops += 10.0 * pairs * c["Hq"] * c["d"]
        return {"bytes": float(io), "flops": flops}
    size = 4 if c["dtype"] == "fp32" else 2
    heads = c["H"] if c["op"] == "rope" else c["Hq"] + c["Hk"]
    values = c["T"] * heads * c["d"]
    moved = 2 * values * size + 4 * c["T"] * c["axes"]
    flops = 3.0 * c["T"] * heads * c["rot"]
    if c["op"] == "qknorm":
        flops += 4.0 * values
        moved += 4 * c["d"] * size
    if c["grad"]:
        moved += 2 * values * size
        flops = 2 * flops + (8.0 * values if c["op"] == "qknorm" else 0.0)
        if c["op"] == "qknorm":
            moved += 4 * c["d"] * size  # q and k are read once for the pass, the weights' gradients written
    return {"bytes": float(moved), "flops": flops}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _gen(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed))
    return g


def _positions(c, g, device):
    """int32 positions: [T], or [3, T] for three axes."""
    T = c["T"]
    if c["positions"] == "grid":
        n = torch.arange(T, device=device)
        hw = c["h"] * c["w"]
        return torch.stack([n // hw, n % hw // c["w"], n % c["w"]]).to(torch.int32)
    if c["positions"] == "far":
        return torch.randint(0, 131072, (T,), generator=g, device=device).to(torch.int32)
    # packed sequences: positions start again at random places
    starts = (torch.rand(T, generator=g, device=device) < 1.0 / 2000).long()
    starts[0] = 1
    n = torch.arange(T, device=device)
    first = torch.cummax(n * starts, 0).values
    return (n - first).to(torch.int32)


def _sections(c):
    """Pairs of each axis: the first axis takes what three equal parts leave over."""
    pairs = c["rot"] // 2
    if c["axes"] == 1:
        return [pairs]
    a = pairs // 3
    return [pairs - 2 * a, a, a]



def prepare(case, seed):
    c = case
    device = _device()
    g = _gen(seed, device)
    s = {"case": c}
    if c["op"] == "prompt":
        lq, lk = _lens(c)
        d, hq, hk = c["d"], c["Hq"], c["Hk"]
        dt = torch.bfloat16
        rnd = lambda *shape: torch.randn(*shape, generator=g, device=device).to(dt)  # noqa: E731
        tq, tk = sum(lq), sum(lk)
        if c["lens_k"] == "":
            # one projection's output: the heads of q, k and v side by side in each token's row
            x = rnd(tq, hq + 2 * hk, d)
            s["q"], s["k"], s["v"] = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
        else:  # keys and values come from a cache of their own
            s["q"], s["k"], s["v"] = rnd(tq, hq, d), rnd(tk, hk, d), rnd(tk, hk, d)
        if c["grad"]:
            s["do"] = rnd(tq, hq, d)
            s["leaves"] = [s[n].detach().requires_grad_(True) for n in "qkv"]
        s["lq"], s["lk"] = lq, lk
        if own:
            import sparse_linear_attention_pool_b200 as sla

            s["plan"] = sla.prompt_plan(lq, None if c["lens_k"] == "" else lk, Hq=hq, Hkv=hk, d=d,
                                        causal=c["causal"], device=device)
        return s
    dt = DTYPES[c["dtype"]]
    d, T = c["d"], c["T"]
    heads = (c["H"],) if c["op"] == "rope" else (c["Hq"], c["Hk"])
    x = torch.randn(T, sum(heads), d, generator=g, device=device).to(dt)  # a projection's output, token-major
    parts = torch.split(x, list(heads), dim=1)
    dys = [torch.randn(T, h, d, generator=g, device=device).to(dt) for h in heads] if c["grad"] else []
    if c["form"] == "heads":  # [1, H, T, d], as the sparse-linear attention takes them
        parts = [p.transpose(0, 1).unsqueeze(0) for p in parts]
        dys = [p.transpose(0, 1).unsqueeze(0).contiguous() for p in dys]
    s["x"], s["dy"] = list(parts), dys
    s["w"] = []
    if c["op"] == "qknorm":
        s["w"] = [(1.0 + 0.2 * torch.randn(d, generator=g, device=device)).to(dt) for _ in range(2)]
    s["pos"] = _positions(c, g, device)
    if c["grad"]:
        s["leaves"] = [t.detach().requires_grad_(True) for t in s["x"] + s["w"]]
    if own:
        import sparse_linear_attention_pool_b200 as sla

        s["table"] = sla.rope_table(c["rot"], layout=c["layout"],
                                    sections=_sections(c) if c["axes"] > 1 else None, scaling=c["scaling"],
                                    factor=c["factor"], original=c["original"], device=device)
    else:
        s["freq"], s["axis"], s["gain"] = _frequencies(c, device)
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

THETA = 10000.0


def _frequencies(c, device):
    """(radians per position of every pair, its axis, the factor on cos and sin), in 64 bits."""
    freq, axis, gain = [], [], 1.0
    for a, n in enumerate(_sections(c)):
        r = 2 * n
        theta = THETA
        if c["scaling"] == "ntk" and r > 2:
            theta = THETA * c["factor"] ** (r / (r - 2.0))
        f = [theta ** (-2.0 * i / r) for i in range(n)]
        if c["scaling"] == "linear":
            f = [x / c["factor"] for x in f]
        elif c["scaling"] == "yarn":
            turn = lambda b: r * math.log(c["original"] / (b * 2 * math.pi)) / (2 * math.log(THETA))  # noqa: E731
            lo, hi = max(0, math.floor(turn(32.0))), min(r - 1, math.ceil(turn(1.0)))
            width = max(hi - lo, 0.001)
            for i in range(n):
                ramp = min(1.0, max(0.0, (i - lo) / width))
                f[i] = f[i] / c["factor"] * ramp + f[i] * (1.0 - ramp)
            gain = 0.1 * math.log(c["factor"]) + 1.0
        freq += f
        axis += [a] * n
    return (torch.tensor(freq, dtype=torch.float64, device=device), torch.tensor(axis, device=device), gain)


def _cos_sin(s):
    """[T, rot / 2] in 32 bits, from angles in 64."""
    pos = s["pos"].double()
    angle = (pos[s["axis"]].t() if pos.dim() == 2 else pos[:, None]) * s["freq"]
    return (torch.cos(angle) * s["gain"]).float(), (torch.sin(angle) * s["gain"]).float()


def _rotate(x, cos, sin, c):
    """x [T, H, d] or [1, H, T, d] in 32 bits."""
    r = c["rot"]
    if x.dim() == 3:
        cos, sin = cos[:, None], sin[:, None]
    y = x.clone()
    if c["layout"] == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y[..., :r // 2] = a * cos - b * sin
        y[..., r // 2:r] = b * cos + a * sin
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2] = a * cos - b * sin
        y[..., 1:r:2] = b * cos + a * sin
    return y


EPS = 1e-6


def _plain_rope(s):
    c = s["case"]
    cos, sin = _cos_sin(s)
    dt = DTYPES[c["dtype"]]
    if c["op"] == "rope":
        out = [_rotate(s["x"][0].float(), cos, sin, c).to(dt)]
        if c["grad"]:
            out.append(_rotate(s["dy"][0].float(), cos, -sin, c).to(dt))
        return out
    out, grads, dws = [], [], []
    for i in range(2):
        x, w = s["x"][i].float(), s["w"][i].float()
        rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        xhat = x * rstd
        out.append(_rotate(xhat * w, cos, sin, c).to(dt))
        if c["grad"]:
            g = _rotate(s["dy"][i].float(), cos, -sin, c)
            dws.append((g * xhat).sum(dim=tuple(j for j in range(x.dim() - 1))).to(dt))
            g = g * w
            grads.append((rstd * (g - xhat * (g * xhat).mean(-1, keepdim=True))).to(dt))
    return out + grads + dws


def _plain_prompt(s):
    c = s["case"]
    q, k, v = s["q"], s["k"], s["v"]
    d, hk, grp = c["d"], c["Hk"], c["Hq"] // c["Hk"]
    scale = 1.0 / math.sqrt(d)
    o = torch.zeros(q.shape, dtype=q.dtype, device=q.device)
    if c["grad"]:
        dq, dk, dv = (torch.zeros(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, v))
    at_q = at_k = 0
    for lq, lk in zip(s["lq"], s["lk"]):
        sq, sk = slice(at_q, at_q + lq), slice(at_k, at_k + lk)
        at_q, at_k = at_q + lq, at_k + lk
        for h in range(hk):
            hs = slice(h * grp, (h + 1) * grp)
            qf = q[sq, hs].float().transpose(0, 1)      # [group, lq, d]
            kf, vf = k[sk, h].float(), v[sk, h].float()  # [lk, d]
            p = torch.matmul(qf, kf.t()).mul_(scale)
            if c["causal"]:
                seen = torch.arange(lk, device=q.device)[None] <= torch.arange(lq, device=q.device)[:, None] + (lk - lq)
                p.masked_fill_(~seen, float("-inf"))
            m = p.amax(-1, keepdim=True)
            m.masked_fill_(m == float("-inf"), 0.0)      # rows that see nothing
            p.sub_(m).exp_()
            total = p.sum(-1, keepdim=True)
            p.div_(total.masked_fill_(total == 0.0, 1.0))
            of = torch.matmul(p, vf)
            o[sq, hs] = of.transpose(0, 1).to(o.dtype)
            if c["grad"]:
                gf = s["do"][sq, hs].float().transpose(0, 1)
                dv[sk, h] = torch.matmul(p.reshape(-1, lk).t(), gf.reshape(-1, d)).to(dv.dtype)
                dp = torch.matmul(gf, vf.t())
                dp.sub_((gf * of).sum(-1, keepdim=True)).mul_(p).mul_(scale)
                dq[sq, hs] = torch.matmul(dp, kf).transpose(0, 1).to(dq.dtype)
                dk[sk, h] = torch.matmul(dp.reshape(-1, lk).t(), qf.reshape(-1, d)).to(dk.dtype)
                del dp
            del p
    return [o, dq, dk, dv] if c["grad"] else [o]


def _own_rope(s):
    import sparse_linear_attention_pool_b200 as sla

    c = s["case"]
    if c["op"] == "rope":
        if not c["grad"]:
            return [sla.rope(s["x"][0], s["table"], s["pos"])]
        y = sla.rope(s["leaves"][0], s["table"], s["pos"])
        return [y.detach()] + list(torch.autograd.grad([y], s["leaves"], s["dy"]))
    if not c["grad"]:
        return list(sla.qk_norm_rope(s["x"][0], s["x"][1], s["w"][0], s["w"][1], s["table"], s["pos"], eps=EPS))
    leaves = s["leaves"]
    y = sla.qk_norm_rope(leaves[0], leaves[1], leaves[2], leaves[3], s["table"], s["pos"], eps=EPS)
    return [t.detach() for t in y] + list(torch.autograd.grad(y, leaves, s["dy"]))


def _own_prompt(s):
    import sparse_linear_attention_pool_b200 as sla

    if not s["case"]["grad"]:
        return [sla.prompt_attention(s["q"], s["k"], s["v"], s["plan"])]
    o = sla.prompt_attention(*s["leaves"], s["plan"])
    return [o.detach()] + list(torch.autograd.grad([o], s["leaves"], [s["do"]]))


def run(state):
    if state["case"]["op"] == "prompt":
        return _own_prompt(state) if own else _plain_prompt(state)
    return _own_rope(state) if own else _plain_rope(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_prompt(s) if case["op"] == "prompt" else _exact_rope(s)


def _exact_rope(s):
    """Pairs as complex numbers, turned by exp(i angle); the gradients through autograd in 64 bits."""
    c = s["case"]
    r, half = c["rot"], c["layout"] == "half"
    base, gain, turns = 10000.0, 1.0, []
    for axis, n in enumerate(_sections(c)):
        i = torch.arange(n, dtype=torch.float64, device=s["pos"].device)
        b = base * c["factor"] ** (n / (n - 1.0)) if c["scaling"] == "ntk" and n > 1 else base
        f = torch.exp(-i / n * math.log(b))
        if c["scaling"] == "linear":
            f = f / c["factor"]
        if c["scaling"] == "yarn":
            # pairs that turn more than 32 times over the original length keep their
            # frequency, those that turn less than once are stretched, a ramp between
            where = [2 * n * math.log(c["original"] / (2 * math.pi * b_)) / (2 * math.log(base)) for b_ in (32.0, 1.0)]
            lo, hi = max(math.floor(where[0]), 0), min(math.ceil(where[1]), 2 * n - 1)
            ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
            f = f * (1.0 - ramp + ramp / c["factor"])
            gain = 1.0 + 0.1 * math.log(c["factor"])
        p = s["pos"][axis] if c["axes"] > 1 else s["pos"]
        turns.append(p.double()[:, None] * f[None])
    turn = torch.polar(torch.full_like(torch.cat(turns, 1), gain), torch.cat(turns, 1))  # [T, rot / 2]

    def one(x, w):
        if w is not None:
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / c["d"] + EPS) * w
        z = torch.complex(x[..., :r // 2], x[..., r // 2:r]) if half else torch.complex(x[..., 0:r:2], x[..., 1:r:2])
        z = z * (turn[:, None] if c["form"] == "packed" else turn)
        front = torch.cat([z.real, z.imag], -1) if half else torch.stack([z.real, z.imag], -1).flatten(-2)
        return torch.cat([front, x[..., r:]], -1)

    ys, dxs, dws = [], [], []
    heads_axis = 1
    for i, x in enumerate(s["x"]):
        w = s["w"][i].double() if s["w"] else None
        if not c["grad"]:
            # a few heads at a time: 64-bit complex copies of the largest case are large
            ys.append(torch.cat([one(p.double(), w) for p in torch.split(x, 4, dim=heads_axis)], heads_axis))
            continue
        dw = None if w is None else torch.zeros_like(w)
        y_parts, dx_parts = [], []
        for p, dy in zip(torch.split(x, 4, dim=heads_axis), torch.split(s["dy"][i], 4, dim=heads_axis)):
            leaf = p.double().detach().requires_grad_(True)
            wl = None if w is None else w.detach().requires_grad_(True)
            y = one(leaf, wl)
            got = torch.autograd.grad(y, [leaf] + ([] if wl is None else [wl]), dy.double())
            y_parts.append(y.detach())
            dx_parts.append(got[0])
            if wl is not None:
                dw += got[1]
        ys.append(torch.cat(y_parts, heads_axis))
        dxs.append(torch.cat(dx_parts, heads_axis))
        if dw is not None:
            dws.append(dw)
    return ys + dxs + dws


def _exact_prompt(s):
    """Rows in pieces; softmax by log-sum-exp; the gradients by the chain rule."""
    c = s["case"]
    q, k, v = s["q"], s["k"], s["v"]
    d, group = c["d"], c["Hq"] // c["Hk"]
    # 64-bit products of the largest cases stay within seconds on the GPU, not on a CPU
    if q.device.type == "cpu" and work(c)["flops"] > 2e11:
        return None
    out = {n: torch.zeros(t.shape, dtype=torch.float64, device=t.device) for n, t in (("o", q), ("q", q), ("k", k), ("v", v))}
    bq = bk = 0
    for nq, nk in zip(s["lq"], s["lk"]):
        for head in range(c["Hq"]):
            kd, vd = k[bk:bk + nk, head // group].double(), v[bk:bk + nk, head // group].double()
            for r0 in range(0, nq, 4096):
                r1 = min(nq, r0 + 4096)
                last = min(nk, nk - nq + r1) if c["causal"] else nk  # keys past this one are seen by no row here
                if last <= 0:
                    continue
                x = q[bq + r0:bq + r1, head].double()
                score = x @ kd[:last].t() / math.sqrt(d)
                hidden = None
                if c["causal"]:
                    row = torch.arange(r0, r1, device=q.device) + (nk - nq)
                    hidden = torch.arange(last, device=q.device)[None, :] > row[:, None]
                    score = torch.where(hidden, -math.inf, score)
                lse = torch.logsumexp(score, -1, keepdim=True)
                prob = torch.exp(score - torch.where(lse == -math.inf, 0.0, lse))
                del score
                y = prob @ vd[:last]
                out["o"][bq + r0:bq + r1, head] = y
                if c["grad"]:
                    gy = s["do"][bq + r0:bq + r1, head].double()
                    out["v"][bk:bk + last, head // group] += prob.t() @ gy
                    ds = prob * (gy @ vd[:last].t() - (gy * y).sum(-1, keepdim=True)) / math.sqrt(d)
                    out["q"][bq + r0:bq + r1, head] = ds @ kd[:last]
                    out["k"][bk:bk + last, head // group] += ds.t() @ x
        bq, bk = bq + nq, bk + nk
    return [out["o"], out["q"], out["k"], out["v"]] if c["grad"] else [out["o"]]
