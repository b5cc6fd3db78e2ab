"""Normed rotary heads, attention over packed sequences and linears with a full epilogue, as cases to measure.

Each case is one pass through an operator. `own` is False: its plain form, elementary torch operations in
32 bits (angles in 64). `own` is True: the library's calls. Both take what prepare() makes: activations,
weights, the sequences' boundaries, the rotary plan's parameters."""

import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}
EPS = 1e-6


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one row's heads normed and turned: the smallest call, where the launch counts
        dict(name="heads-1-row", op="heads", B=1, T=1, Hq=24, Hk=24, d=128, widths="16,56,56", layout="pairs", x="bf16",
             grad=False, packed=True),
        # q and k of the 1024 x 1024 image's rows out of the packed QKV product
        dict(name="heads-1024sq", op="heads", B=1, T=4224, Hq=24, Hk=24, d=128, widths="16,56,56", layout="pairs", x="bf16",
             grad=False, packed=True),
        # an odd batch in fp32 with few key heads, three quarters of the head turned in halves
        dict(name="heads-odd", op="heads", B=3, T=1111, Hq=6, Hk=2, d=64, widths="48", layout="halves", x="fp32",
             grad=False, packed=False),
        # the gradient of the 1024 x 1024 image's heads
        dict(name="heads-grad-1024sq", op="heads", B=1, T=4224, Hq=24, Hk=24, d=128, widths="16,56,56", layout="pairs",
             x="bf16", grad=True, packed=True),
        # the gradient of an odd fp32 batch with few key heads
        dict(name="heads-grad-odd", op="heads", B=3, T=1111, Hq=6, Hk=2, d=64, widths="48", layout="halves", x="fp32",
             grad=True, packed=False),
        # one new row over the keys of a 512 x 512 image and its text: the smallest call
        dict(name="attend-1-row", op="attend", H=24, Hk=24, d=128, segs=1, q=1, k=1088, ragged=0, mask="full", cap=0.0,
             bias=False, packed=False),
        # the guided and the unguided sequence of a 1024 x 1024 image, their texts of unlike length, in one call
        dict(name="attend-1024sq-two", op="attend", H=24, Hk=24, d=128, segs=2, q=4224, k=4224, ragged=11, mask="full",
             cap=0.0, bias=False, packed=True),
        # images of many sizes with capped scores and grouped key heads; texts see texts alone, padding rows nothing
        dict(name="attend-sizes-capped", op="attend", H=16, Hk=4, d=64, segs=9, q=2100, k=2100, ragged=5, mask="prefix",
             cap=50.0, bias=False, packed=True),
        # single new rows of 64 sequences over long caches of unlike length, nearer keys preferred
        dict(name="attend-64-caches", op="attend", H=32, Hk=8, d=128, segs=64, q=1, k=8192, ragged=3, mask="full", cap=0.0,
             bias=True, packed=False),
        # one row through the modulation linear with its bias
        dict(name="linear-1-modulation", op="linear", M=1, K=3072, N=18432, act="none", out="bf16", residual=False, gate=0),
        # sizes no tile divides, fp32 residual rows and gates of three images
        dict(name="linear-ragged-gated", op="linear", M=333, K=1000, N=777, act="none", out="fp32", residual=True, gate=3),
        # the first linear of a GELU MLP over the rows of a 1024 x 1024 image: the largest product
        dict(name="linear-1024sq-gelu", op="linear", M=4224, K=3072, N=12288, act="gelu_tanh", out="bf16", residual=False,
             gate=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["heads", "attend", "attend", "linear"])
    if op == "heads":
        d = rng.choice([32, 64, 80, 96, 128, 256])
        widths = rng.choice([str(d), str(d // 4 * 2), str(3 * d // 8 * 2), "%d,%d,%d" % (d // 8, d // 32 * 14, d // 32 * 14)])  # even ones
        while True:
            B, T, Hq = rng.choice([1, 1, 2, 3, 5]), _log(rng, 1, 20000), rng.choice([1, 3, 6, 8, 12, 24, 32])
            Hk = rng.choice([h for h in (1, 2, 3, 4, 8, 24) if h <= Hq])
            if B * T * (Hq + Hk) * d <= 2.6e7:
                return dict(op=op, B=B, T=T, Hq=Hq, Hk=Hk, d=d, widths=widths, layout=rng.choice(["pairs", "halves"]),
                            x=rng.choice(["bf16", "bf16", "fp32"]), grad=rng.random() < 0.5, packed=rng.random() < 0.5)
    if op == "attend":
        while True:
            Hk, G = rng.choice([1, 2, 3, 4, 8, 24]), rng.choice([1, 1, 2, 3, 4, 6, 8])
            segs, few = rng.choice([1, 1, 2, 3, 7, 20, 64]), rng.random() < 0.4
            k = _log(rng, 1, 16000)
            q = min(k, rng.choice([1, 1, 1, 2, 5, 17])) if few else k
            d = rng.choice([64, 128])
            if segs * q * k * Hk * G * d <= 4.3e10 and segs * k * Hk * d <= 5.5e8 and segs * max(q, 64) * Hk * G * k <= 1.0e9:
                return dict(op=op, H=Hk * G, Hk=Hk, d=d, segs=segs, q=q, k=k, ragged=rng.choice([0, _log(rng, 1, 1000)]),
                            mask=rng.choice(["full", "full", "causal", "prefix", "frames"]), cap=rng.choice([0.0, 0.0, 30.0, 50.0]),
                            bias=rng.random() < 0.3, packed=not few and rng.random() < 0.7)
    while True:
        M, K, N = _log(rng, 1, 6000), _log(rng, 8, 14000) // 8 * 8, _log(rng, 8, 20000)
        if rng.random() < 0.5:  # half of them at widths a model has
            K, N = max(64, K // 64 * 64), max(128, N // 128 * 128)
        if M * K * N <= 1.5e11 and M * N <= 6.0e7 and K * N <= 6.0e7:
            return dict(op=op, M=M, K=K, N=N, act=rng.choice(["none", "silu", "gelu", "gelu_tanh"]), out=rng.choice(["bf16", "fp32"]),
                        residual=rng.random() < 0.5, gate=rng.choice([0, 0, 1, 3]))


# ------------------------------------------------------------------------------------- heads: plain form
def _frequencies(widths):
    """Angle per position of each pair (64 bits) and the axis of each pair."""
    f, axis = [], []
    for a, w in enumerate(widths):
        f.append(10000.0 ** (-2.0 * torch.arange(w // 2, dtype=torch.float64) / w))
        axis += [a] * (w // 2)
    return torch.cat(f), axis


def _turn(x, cos, sin, dim, pairs):
    """x [B, T, H, d]; cos, sin [B, T, 1, dim / 2]."""
    r = x[..., :dim]
    a, b = (r[..., 0::2], r[..., 1::2]) if pairs else (r[..., :dim // 2], r[..., dim // 2:])
    u, v = a * cos - b * sin, a * sin + b * cos
    y = torch.stack([u, v], -1).flatten(-2) if pairs else torch.cat([u, v], -1)
    return torch.cat([y, x[..., dim:]], -1)


def _heads_plain(st):
    case = st["case"]
    angle = st["pos"].double()[..., st["axis"]] * st["freq"]
    cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]
    dim, pairs = 2 * len(st["freq"]), case["layout"] == "pairs"
    out = {}
    for n in ("q", "k"):
        x, w = st[n].float(), st[n + "_norm"]
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        if not case["grad"]:
            st[n + "_out"].copy_(_turn(x * r * w, cos, sin, dim, pairs))
            out[n] = st[n + "_out"]
            continue
        g = _turn(st["d" + n].float(), cos, -sin, dim, pairs)
        xr = x * r
        st[n + "_out"].copy_(r * (g * w - xr * (g * w * xr).mean(-1, keepdim=True)))
        out[n] = st[n + "_out"]
        out[n + "_norm"] = (g * xr).double().sum((0, 1, 2)).float()
    return out


# ----------------------------------------------------------------------------------- attention: its layout
def _layout(case):
    """Lengths of the sequences' queries and keys and, per sequence, the keys each query sees (None: all)."""
    rng = random.Random(case["ragged"])
    ql, kl, seen = [], [], []
    for s in range(case["segs"]):
        k = case["k"] if not case["ragged"] else max(1, int(case["k"] * rng.uniform(0.25, 1.0)))
        q = k if case["q"] == case["k"] else min(case["q"], k)
        ql.append(q)
        kl.append(k)
        i = torch.arange(q) + (k - q)  # a query's place among the keys
        if case["mask"] == "full":
            seen.append(None)
        elif case["mask"] == "causal":
            seen.append(i + 1)
        elif case["mask"] == "frames":  # frames of 256 rows, each sees itself and the ones before
            seen.append(((i // 256 + 1) * 256).clamp(max=k))
        else:  # a text in front that sees itself alone, the last rows padding
            text, pad = min(k, rng.randint(1, 128)), rng.randint(0, 7) if k > 200 and q == k else 0
            v = torch.where(i < text, text, k - pad)
            seen.append(torch.where(i >= k - pad, 0, v))
    return ql, kl, seen


def _starts(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def _attend(q, k, v, seen, scale, cap, slope, one, zero):
    """One sequence: q [nq, H, d], k, v [nk, Hk, d] in the type to compute in -> o [nq, H, d], lse [H, nq]."""
    nq, H, d = q.shape
    nk, Hk = k.shape[0], k.shape[1]
    G = H // Hk
    o, lse = q.new_empty(nq, H, d), q.new_empty(H, nq)
    heads = min(Hk, max(1, 2 ** 28 // (G * nq * nk)))  # key heads and rows taken at a time
    step = min(nq, max(1, 2 ** 28 // (G * nk)))
    j = torch.arange(nk, device=q.device)
    for h in range(0, Hk, heads):
        n = min(heads, Hk - h)
        kt, vh, g = k[:, h:h + n].permute(1, 2, 0), v[:, h:h + n].transpose(0, 1), slice(h * G, (h + n) * G)
        for r in range(0, nq, step):
            rows = slice(r, min(nq, r + step))
            m = rows.stop - r
            s = q[rows, g].transpose(0, 1).reshape(n, G * m, d) @ kt * scale
            if cap > 0:
                s = torch.tanh(s / cap) * cap
            s = s.view(n * G, m, nk)
            i = torch.arange(r, rows.stop, device=q.device)
            if slope is not None:
                s = s - slope[g].to(q.dtype)[:, None, None] * (i[:, None] + (nk - nq) - j).abs().to(q.dtype)
            if seen is not None:
                s = s.masked_fill(j >= seen[rows, None], -math.inf)
            top = s.amax(-1, keepdim=True)
            top = torch.where(top == -math.inf, zero, top)
            e = torch.exp(s - top)
            total = e.sum(-1, keepdim=True)
            y = (e.view(n, G * m, nk) @ vh).view(n * G, m, d) / torch.where(total == 0, one, total)
            o[rows, g] = y.transpose(0, 1)
            lse[g, rows] = (torch.log(total) + top)[..., 0]
    return o, lse


def _attend_all(st, dtype):
    one, zero = torch.ones((), dtype=dtype, device="cuda"), torch.zeros((), dtype=dtype, device="cuda")
    case = st["case"]
    o = torch.empty(st["q"].shape, dtype=dtype, device="cuda")
    lse = torch.empty(case["H"], o.shape[0], dtype=dtype, device="cuda")
    for s in range(case["segs"]):
        a, b = slice(st["qs"][s], st["qs"][s + 1]), slice(st["ks"][s], st["ks"][s + 1])
        seen = None if st["visible"] is None else st["visible"][a]
        o[a], lse[:, a] = _attend(st["q"][a].to(dtype), st["k"][b].to(dtype), st["v"][b].to(dtype), seen,
                                  case["d"] ** -0.5, case["cap"], st["slope"], one, zero)
    return o, lse


# ------------------------------------------------------------------------------------- linear: plain form
def _act(y, name):
    if name == "silu":
        return y / (1 + torch.exp(-y))
    if name == "gelu":
        return 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    return y


def _linear(st, dtype):
    y = st["a"].to(dtype) @ st["w"].to(dtype).t() + st["bias"].to(dtype)
    y = _act(y, st["case"]["act"])
    if st["gate"] is not None:
        y = y * st["gate"].to(dtype)[st["map"].long()]
    return y if st["residual"] is None else st["residual"].to(dtype) + y


# ------------------------------------------------------------------------------------------------ inputs
def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    rn = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    st = {"case": case}
    if case["op"] == "heads":
        B, T, Hq, Hk, d = (case[n] for n in ("B", "T", "Hq", "Hk", "d"))
        dt = TYPES[case["x"]]
        # heads and rows of unlike size, as a projection leaves them; norm weights near one
        make = lambda h: (rn(B, T, h, d) * torch.exp(0.5 * rn(B, T, h, 1))).to(dt)  # noqa: E731
        for n in (("", "d") if case["grad"] else ("",)):
            if case["packed"]:  # columns of one QKV product's rows (or of its gradient's)
                qkv = make(Hq + 2 * Hk)
                st[n + "q"], st[n + "k"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
            else:
                st[n + "q"], st[n + "k"] = make(Hq), make(Hk)
        st["q_norm"], st["k_norm"] = 1 + 0.2 * rn(d), 1 + 0.2 * rn(d)
        axes = len(case["widths"].split(","))
        st["pos"] = torch.randint(-(T // 8), T + 4, (B, T, axes), device="cuda", generator=g, dtype=torch.int32)
        st["q_out"] = torch.empty(B, T, Hq, d, dtype=dt, device="cuda")
        st["k_out"] = torch.empty(B, T, Hk, d, dtype=dt, device="cuda")
    elif case["op"] == "attend":
        ql, kl, seen = _layout(case)
        H, Hk, d = case["H"], case["Hk"], case["d"]
        st["qs"], st["ks"] = _starts(ql), _starts(kl)
        nq, nk = st["qs"][-1], st["ks"][-1]
        # scores a few units wide; past the cap's linear part where there is one
        gain = 8.0 if case["cap"] else 2.0
        if case["packed"]:
            qkv = rn(nq, H + 2 * Hk, d).bfloat16()
            qkv[:, :H] *= gain
            st["q"], st["k"], st["v"] = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
        else:
            st["q"], st["k"], st["v"] = (gain * rn(nq, H, d)).bfloat16(), rn(nk, Hk, d).bfloat16(), rn(nk, Hk, d).bfloat16()
        st["q_start"] = torch.tensor(st["qs"], dtype=torch.int32, device="cuda")
        st["k_start"] = torch.tensor(st["ks"], dtype=torch.int32, device="cuda")
        st["visible"] = None if seen[0] is None else torch.cat(seen).to(torch.int32).cuda()
        st["slope"] = torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H) if case["bias"] else None
        st["o"] = torch.empty(nq, H, d, dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.empty(H, nq, device="cuda")
    else:
        M, K, N = case["M"], case["K"], case["N"]
        st["a"], st["w"] = rn(M, K).bfloat16(), (rn(N, K) / math.sqrt(K)).bfloat16()
        st["bias"] = 0.5 * rn(N)
        st["gate"] = 0.5 * rn(case["gate"], N) if case["gate"] else None
        st["map"] = torch.randint(0, case["gate"], (M,), device="cuda", generator=g, dtype=torch.int32) if case["gate"] else None
        st["residual"] = rn(M, N).to(TYPES[case["out"]]) if case["residual"] else None
        st["out"] = torch.empty(M, N, dtype=TYPES[case["out"]], device="cuda")
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        import diffusion_transformer_gb300 as D
        ws = lambda n: torch.empty(max(256, n), dtype=torch.uint8, device="cuda")  # noqa: E731
    if case["op"] == "heads":
        widths = [int(w) for w in case["widths"].split(",")]
        if own:
            st["plan"] = D.RotaryPlan(widths=widths, layout=case["layout"], theta=10000.0)
            if case["grad"]:
                st["ws"] = ws(D.dit_qknorm_rotary_backward_workspace_bytes(case["d"]))
                st["q_norm_grad"], st["k_norm_grad"] = torch.empty_like(st["q_norm"]), torch.empty_like(st["k_norm"])
        else:
            f, axis = _frequencies(widths)
            st.update(freq=f.cuda(), axis=torch.tensor(axis, device="cuda"))
    elif own and case["op"] == "attend":
        st["ws"] = ws(D.dit_attention_packed_workspace_bytes(st["q"].shape[0], st["k"].shape[0], case["segs"], case["H"],
                                                             case["Hk"], case["d"]))
    elif own:
        st["ws"] = ws(D.dit_linear_epilogue_workspace_bytes(case["M"], case["N"], case["K"]))
    return st


# ------------------------------------------------------------------------------------------------ one pass
def run(st):
    case = st["case"]
    if not own:
        if case["op"] == "heads":
            return _heads_plain(st)
        if case["op"] == "attend":
            o, lse = _attend_all(st, torch.float32)
            st["o"].copy_(o)
            st["lse"].copy_(lse)
            return {"o": st["o"], "lse": st["lse"]}
        st["out"].copy_(_linear(st, torch.float32))
        return st["out"]
    import diffusion_transformer_gb300 as D
    if case["op"] == "heads":
        if not case["grad"]:
            D.dit_qknorm_rotary(st["plan"], st["q"], st["k"], st["pos"], st["q_norm"], st["k_norm"], st["q_out"], st["k_out"],
                                eps=EPS)
            return {"q": st["q_out"], "k": st["k_out"]}
        D.dit_qknorm_rotary_backward(st["plan"], st["q"], st["k"], st["dq"], st["dk"], st["pos"], st["q_norm"], st["k_norm"],
                                     st["q_out"], st["k_out"], st["q_norm_grad"], st["k_norm_grad"], st["ws"], eps=EPS)
        return {"q": st["q_out"], "q_norm": st["q_norm_grad"], "k": st["k_out"], "k_norm": st["k_norm_grad"]}
    if case["op"] == "attend":
        D.dit_attention_packed(st["q"], st["k"], st["v"], st["o"], st["q_start"], st["k_start"], visible=st["visible"],
                               cap=case["cap"], slope=st["slope"], lse=st["lse"], ws=st["ws"])
        return {"o": st["o"], "lse": st["lse"]}
    D.dit_linear_epilogue(st["a"], st["w"], st["out"], bias=st["bias"], activation=case["act"], gate=st["gate"],
                          gate_map=st["map"], residual=st["residual"], ws=st["ws"])
    return st["out"]


def work(case):
    if case["op"] == "heads":
        n = case["B"] * case["T"] * (case["Hq"] + case["Hk"]) * case["d"]
        pos = case["B"] * case["T"] * len(case["widths"].split(",")) * 4
        return {"bytes": (3 if case["grad"] else 2) * n * SIZE[case["x"]] + pos, "flops": (16 if case["grad"] else 8) * n}
    if case["op"] == "attend":
        ql, kl, seen = _layout(case)
        pairs = sum(q * k if v is None else int(v.sum()) for q, k, v in zip(ql, kl, seen))
        rows = 2 * sum(ql) * case["H"] * case["d"] * 2 + 4 * sum(ql) * case["H"]
        return {"bytes": rows + 2 * sum(kl) * case["Hk"] * case["d"] * 2, "flops": 4 * pairs * case["H"] * case["d"]}
    M, N, K, s = case["M"], case["N"], case["K"], SIZE[case["out"]]
    return {"bytes": 2 * K * (M + N) + M * N * s * (2 if case["residual"] else 1), "flops": 2 * M * N * K}


# --------------------------------------------------------------------------------------------- in 64 bits
def _exact_heads(st):
    case = st["case"]
    f, axis = _frequencies([int(w) for w in case["widths"].split(",")])
    dim, half = 2 * len(f), len(f)
    at = st["pos"].double()[..., torch.tensor(axis, device="cuda")] * f.cuda()
    re = torch.arange(0, dim, 2) if case["layout"] == "pairs" else torch.arange(half)
    im = re + (1 if case["layout"] == "pairs" else half)

    def turned(x, angle):
        z = torch.complex(x[..., re], x[..., im]) * torch.polar(torch.ones_like(angle), angle)[:, :, None]
        y = x.clone()
        y[..., re], y[..., im] = z.real, z.imag
        return y

    res = {}
    for n in ("q", "k"):
        x, w = st[n].double(), st[n + "_norm"].double()
        size = torch.sqrt(torch.square(x).sum(-1, keepdim=True) / x.shape[-1] + EPS)
        unit = x / size
        if not case["grad"]:
            res[n] = turned(unit * w, at)
            continue
        g = turned(st["d" + n].double(), -at)
        along = (unit * g * w).sum(-1, keepdim=True) / x.shape[-1]
        res[n] = (g * w - unit * along) / size
        res[n + "_norm"] = torch.einsum("bthd,bthd->d", g, unit)
    return res


def exact(case, seed):
    st = _inputs(case, seed)
    if case["op"] == "heads":
        return _exact_heads(st)
    if case["op"] == "linear":
        out = torch.empty(case["M"], case["N"], dtype=torch.float64, device="cuda")
        w = st["w"].double().t().contiguous()
        for r in range(0, case["M"], 512):
            y = torch.addmm(st["bias"].double(), st["a"][r:r + 512].double(), w)
            if case["act"] == "silu":
                y = y * torch.sigmoid(y)
            elif case["act"] == "gelu":
                y = y * torch.special.ndtr(y)
            elif case["act"] == "gelu_tanh":
                y = y * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3))
            if st["gate"] is not None:
                y = y * st["gate"].double()[st["map"][r:r + 512].long()]
            out[r:r + 512] = y if st["residual"] is None else y + st["residual"][r:r + 512].double()
        return out
    H, G = case["H"], case["H"] // case["Hk"]
    o = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full((H, o.shape[0]), -math.inf, dtype=torch.float64, device="cuda")
    for s in range(case["segs"]):
        q0, q1, k0, k1 = st["qs"][s], st["qs"][s + 1], st["ks"][s], st["ks"][s + 1]
        nq, nk = q1 - q0, k1 - k0
        far = (torch.arange(nq, device="cuda")[:, None] + nk - nq - torch.arange(nk, device="cuda")).abs().double()
        for h in range(H):
            k, v = st["k"][k0:k1, h // G].double(), st["v"][k0:k1, h // G].double()
            for r in range(0, nq, 4096):
                e = min(nq, r + 4096)
                y = torch.einsum("id,jd->ij", st["q"][q0 + r:q0 + e, h].double(), k) / math.sqrt(case["d"])
                if case["cap"]:
                    y = case["cap"] * torch.tanh(y / case["cap"])
                if st["slope"] is not None:
                    y = y - float(st["slope"][h]) * far[r:e]
                if st["visible"] is not None:
                    y = torch.where(torch.arange(nk, device="cuda") < st["visible"][q0 + r:q0 + e, None], y, -math.inf)
                z = torch.logsumexp(y, 1)
                lse[h, q0 + r:q0 + e] = z
                o[q0 + r:q0 + e, h] = torch.exp(y - torch.where(z == -math.inf, 0.0, z)[:, None]) @ v
    return {"o": o, "lse": lse}
