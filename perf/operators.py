"""The 4-bit linears and the rotary positions of the block library, as cases to measure.

Each case is one pass through an operator. `own` is False: its plain form, elementary torch operations in
32 bits (angles in 64). `own` is True: the library's calls. Both take what prepare() makes: activations,
weights already quantised into the library's documented layout, the rotary plan's parameters."""

import math

import torch

own = False

NV, MX = 0, 1            # 4-bit formats: blocks of 16 with e4m3 scales and a row scale; blocks of 32 with 2^e
BLOCK = {NV: 16, MX: 32}
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one row through a 4-bit linear: the modulation linear (6 x hidden) of one denoise step
        dict(name="linear-1-modulation", op="linear", M=1, K=3072, N=18432, fmt="nv", x="bf16", out="bf16"),
        # a prompt's text rows through the QKV linear (512 x 512 image, 64 text rows)
        dict(name="linear-64-text-qkv", op="linear", M=64, K=3072, N=9216, fmt="nv", x="bf16", out="bf16"),
        # sizes no tile divides, fp32 residual rows in and fp32 out: a projection of another encoder's features
        dict(name="linear-ragged", op="linear", M=333, K=1000, N=777, fmt="nv", x="fp32", out="fp32"),
        # the 512 x 512 block's down linear with power-of-two block scales
        dict(name="linear-512sq-down", op="linear", M=1088, K=12288, N=3072, fmt="mx", x="bf16", out="bf16"),
        # the 1024 x 1024 block's up linear: the largest product of the block
        dict(name="linear-1024sq-up", op="linear", M=4224, K=3072, N=24576, fmt="nv", x="bf16", out="bf16"),
        # a few rows of an odd width, quantised and read back: what a check of a layer's error does
        dict(name="quant-small-odd", op="quant", R=5, K=1003, fmt="nv", x="fp32", out="fp32"),
        # the SwiGLU output of the 1024 x 1024 block, quantised per token and read back
        dict(name="quant-1024sq-act", op="quant", R=4224, K=12288, fmt="nv", x="bf16", out="bf16"),
        # a checkpoint's fp32 QKV weight turned into power-of-two blocks and read back
        dict(name="quant-qkv-weight-mx", op="quant", R=9216, K=3072, fmt="mx", x="fp32", out="fp32"),
        # one row's heads turned: the smallest call, where the launch counts
        dict(name="rotary-1-row", op="rotary", B=1, T=1, Hq=24, Hk=24, d=128, widths="16,56,56", layout="pairs", x="bf16",
             scaling="none", factor=1.0, far=4096, inverse=False, packed=True),
        # q and k of the 1024 x 1024 block, out of the packed QKV rows, written head-major
        dict(name="rotary-1024sq", op="rotary", B=1, T=4224, Hq=24, Hk=24, d=128, widths="16,56,56", layout="pairs", x="bf16",
             scaling="none", factor=1.0, far=4224, inverse=False, packed=True),
        # gradient rows in fp32, odd length, half layout over the whole head
        dict(name="rotary-grad-odd", op="rotary", B=3, T=1111, Hq=6, Hk=2, d=64, widths="64", layout="halves", x="fp32",
             scaling="linear", factor=4.0, far=1111, inverse=True, packed=False),
        # long sequences at positions far beyond the trained length, three quarters of the head, few key heads
        dict(name="rotary-long-yarn", op="rotary", B=2, T=65536, Hq=8, Hk=2, d=128, widths="96", layout="halves", x="bf16",
             scaling="yarn", factor=16.0, far=1000000, inverse=False, packed=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "quant", "rotary"])
    fmt, x, out = rng.choice(["nv", "nv", "mx"]), rng.choice(["bf16", "bf16", "fp32"]), rng.choice(["bf16", "fp32"])
    if op == "linear":
        while True:
            M, K, N = _log(rng, 1, 6000), _log(rng, 32, 14000), _log(rng, 16, 26000)
            if rng.random() < 0.5:  # half of them at widths a model has
                K, N = max(64, K // 64 * 64), max(128, N // 128 * 128)
            if M * K * N <= 3.0e11 and M * N <= 1.0e8 and K * N <= 7.5e7:
                return dict(op=op, M=M, K=K, N=N, fmt=fmt, x=x, out=out)
    if op == "quant":
        while True:
            R, K = _log(rng, 1, 25000), _log(rng, 1, 14000)
            if R * K <= 5.0e7:
                return dict(op=op, R=R, K=K, fmt=fmt, x=x, out=out)
    d = rng.choice([32, 64, 80, 96, 128, 256])
    widths = rng.choice([str(d), str(d // 4 * 2), str(3 * d // 8 * 2), "%d,%d,%d" % (d // 8, d // 16 * 7, d // 16 * 7)])
    while True:
        B, T, Hq = rng.choice([1, 1, 2, 3, 5]), _log(rng, 1, 70000), rng.choice([1, 3, 6, 8, 12, 24, 32])
        Hk = rng.choice([h for h in (1, 2, 3, 4, 8, 24) if h <= Hq])
        if B * T * (Hq + Hk) * d <= 1.6e8:
            break
    return dict(op=op, B=B, T=T, Hq=Hq, Hk=Hk, d=d, widths=widths, layout=rng.choice(["pairs", "halves"]), x=x,
                scaling=rng.choice(["none", "linear", "ntk", "yarn"]), factor=rng.choice([2.0, 4.0, 16.0]),
                far=_log(rng, max(16, T), 2000000), inverse=rng.random() < 0.3, packed=rng.random() < 0.5)


# ------------------------------------------------------------------------------------- 4-bit plain form
def _fmt(case):
    return NV if case["fmt"] == "nv" else MX


def _blocks(v, n):
    """[R, K] as [R, ceil(K / n), n], the last block filled with zeros."""
    R, K = v.shape
    nb = -(-K // n)
    if nb * n != K:
        v = torch.cat([v, v.new_zeros(R, nb * n - K)], 1)
    return v.view(R, nb, n)


def _pow2(e):
    """2^e in fp32 for whole e from -127 to 127."""
    return torch.where(e < -126, torch.full_like(e, 1 << 22), (e + 127) << 23).view(torch.float32)


def _e2m1(a):
    """Index of the nearest of VALUES to a >= 0 (ties to the even index)."""
    return ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)).to(torch.uint8)


def _quantise(x, fmt):
    """x [R, K] -> code indices with a sign bit [R, nb, n] uint8, block scales [R, nb] fp32, row scales [R] fp32."""
    b = _blocks(x.float(), BLOCK[fmt])
    amax_b = b.abs().amax(2)
    if fmt == NV:
        amax = amax_b.amax(1)
        live = amax >= 2.0 ** -100
        top = torch.where(live, amax, torch.ones_like(amax))
        s = (amax_b * (torch.full_like(top, 448.0) / top)[:, None]).clamp(max=448.0).to(torch.float8_e4m3fn).float()
        s = torch.where(live[:, None], s, torch.zeros_like(s))
        inv = torch.where(s > 0, (torch.full_like(top, 2688.0) / top)[:, None] / s, torch.zeros_like(s))
        row = torch.where(live, amax / torch.full_like(amax, 2688.0), torch.zeros_like(amax))
    else:
        e = (torch.frexp(amax_b)[1] - 3).clamp(-127, 127)
        e = torch.where(amax_b > 0, e, torch.full_like(e, -127))
        s, inv = _pow2(e), _pow2(-e)
        row = torch.ones(x.shape[0], device=x.device)
    y = b * inv[:, :, None]
    return _e2m1(y.abs()) | (y < 0).to(torch.uint8) << 3, s, row


def _values(idx, s, row, K):
    table = torch.tensor(VALUES + tuple(-v for v in VALUES), device=s.device)
    v = table[idx.long()] * s[:, :, None] * row[:, None, None]
    return v.flatten(1)[:, :K]


def _scale_place(R, nb, device):
    """Where block scale (r, b) stands: tiles of 128 rows x 4 blocks, 512 bytes each, row r % 128 of a tile at byte
    16 (r % 32) + 4 (r % 128 // 32)."""
    r, b = torch.arange(R, device=device)[:, None], torch.arange(nb, device=device)[None]
    tiles = -(-nb // 4)
    return ((r // 128) * tiles + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4


def _pack(idx, s, fmt, K):
    """The library's layout: codes [R, 16 ceil(K / 32)] (even k in the low half of a byte) and scale bytes."""
    R, nb, n = idx.shape
    wide = -(-K // 32) * 32
    flat = idx.flatten(1)
    flat = torch.cat([flat, flat.new_zeros(R, wide - flat.shape[1])], 1) if flat.shape[1] < wide else flat[:, :wide]
    codes = flat[:, 0::2] | flat[:, 1::2] << 4
    scales = torch.zeros(-(-R // 128) * -(-nb // 4) * 512, dtype=torch.uint8, device=s.device)
    by = s.to(torch.float8_e4m3fn).view(torch.uint8) if fmt == NV else (torch.frexp(s)[1] + 126).to(torch.uint8)
    scales[_scale_place(R, nb, s.device)] = by
    return codes.contiguous(), scales


def _unpack(codes, scales, fmt, R, K):
    idx = torch.stack([codes & 15, codes >> 4], 2).flatten(1)
    n, nb = BLOCK[fmt], -(-K // BLOCK[fmt])
    idx = idx[:, :nb * n] if idx.shape[1] >= nb * n else torch.cat([idx, idx.new_zeros(R, nb * n - idx.shape[1])], 1)
    by = scales[_scale_place(R, nb, scales.device)]
    s = by.view(torch.float8_e4m3fn).float() if fmt == NV else _pow2(by.int() - 127)
    return idx.reshape(R, nb, n), s


# -------------------------------------------------------------------------------------- rotary plain form
def _frequencies(case):
    """Angle per position of each pair (64 bits), the axis of each pair, the amplitude of cos and sin."""
    theta, f, L0 = 10000.0, case["factor"], 4096
    out, axis, amp = [], [], 1.0
    for a, w in enumerate(int(v) for v in case["widths"].split(",")):
        k = torch.arange(w // 2, dtype=torch.float64)
        base = theta * f ** (w / (w - 2.0)) if case["scaling"] == "ntk" and w > 2 else theta
        fr = base ** (-2.0 * k / w)
        if case["scaling"] == "linear":
            fr = fr / f
        elif case["scaling"] == "yarn":
            at = lambda turns: w * math.log(L0 / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
            lo, hi = max(0, math.floor(at(32.0))), min(w // 2 - 1, math.ceil(at(1.0)))
            ramp = ((k - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
            fr = fr * (1 - ramp) + fr / f * ramp
            amp = 0.1 * math.log(f) + 1.0
        out.append(fr)
        axis += [a] * (w // 2)
    return torch.cat(out), axis, amp


def _turn(x, cos, sin, dim, pairs):
    """x [B, T, H, d]; cos, sin [B, T, 1, dim / 2]."""
    r = x[..., :dim]
    a, b = (r[..., 0::2], r[..., 1::2]) if pairs else (r[..., :dim // 2], r[..., dim // 2:])
    u, v = a * cos - b * sin, a * sin + b * cos
    y = torch.stack([u, v], -1).flatten(-2) if pairs else torch.cat([u, v], -1)
    return torch.cat([y, x[..., dim:]], -1)


# ------------------------------------------------------------------------------------------------ inputs
def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    rn = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    if case["op"] == "rotary":
        B, T, Hq, Hk, d = (case[k] for k in ("B", "T", "Hq", "Hk", "d"))
        dt = TYPES[case["x"]]
        if case["packed"]:  # q and k are columns of one QKV product's rows
            qkv = rn(B, T, Hq + 2 * Hk, d).to(dt)
            q, k = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
        else:
            q, k = rn(B, T, Hq, d).to(dt), rn(B, T, Hk, d).to(dt)
        axes = len(case["widths"].split(","))
        pos = torch.randint(-(case["far"] // 8), case["far"], (B, T, axes), device="cuda", generator=g, dtype=torch.int32)
        return q, k, pos
    R = case["M"] if case["op"] == "linear" else case["R"]
    K = case["K"]
    # activations with a few wide channels and rows of unlike size, as behind a norm and a modulation
    x = rn(R, K) * (1 + 20 * (torch.rand(K, device="cuda", generator=g) < 0.01)) * torch.exp(0.5 * rn(R, 1))
    if R > 2:
        x[R // 2] = 0  # a padding row
    x = x.to(TYPES[case["x"]])
    w = rn(case["N"], K).mul_(0.02).bfloat16() if case["op"] == "linear" else None
    return x, w


def prepare(case, seed):
    st = {"case": case}
    if case["op"] == "rotary":
        q, k, pos = _inputs(case, seed)
        B, T, Hq, d = q.shape
        st.update(q=q, k=k, pos=pos, qo=torch.empty(B, Hq, T, d, dtype=q.dtype, device="cuda"),
                  ko=torch.empty(B, k.shape[2], T, d, dtype=q.dtype, device="cuda"))
        if own:
            import diffusion_transformer_gb300 as D
            st["plan"] = D.RotaryPlan(widths=[int(v) for v in case["widths"].split(",")], layout=case["layout"],
                                      theta=10000.0, scaling=case["scaling"], factor=case["factor"], original=4096)
        else:
            f, axis, amp = _frequencies(case)
            st.update(freq=f.cuda(), axis=torch.tensor(axis, device="cuda"), amp=amp)
        return st
    x, w = _inputs(case, seed)
    fmt, R, K = _fmt(case), x.shape[0], case["K"]
    st.update(x=x)
    cols = case["N"] if case["op"] == "linear" else K
    st["out"] = torch.empty(R, cols, dtype=TYPES[case["out"]], device="cuda")
    if w is not None:
        idx, s, row = _quantise(w, fmt)
        codes, scales = _pack(idx, s, fmt, K)
        del idx
        st.update(codes=codes, scales=scales, row=row if fmt == NV else None)
    if own:
        import diffusion_transformer_gb300 as D
        if w is not None:
            st["w"] = D.Fp4Matrix(fmt, case["N"], K, codes, scales, st["row"])
            st["ws"] = torch.empty(D.dit_linear_fp4_workspace_bytes(fmt, R, case["N"], K), dtype=torch.uint8, device="cuda")
        else:
            st["m"] = D.Fp4Matrix.empty(fmt, R, K, device="cuda")
    return st


# ------------------------------------------------------------------------------------------------ one pass
def run(st):
    case = st["case"]
    if own:
        import diffusion_transformer_gb300 as D
        if case["op"] == "linear":
            D.dit_linear_fp4(st["x"], st["w"], st["out"], st["ws"])
            return st["out"]
        if case["op"] == "quant":
            D.dit_fp4_quantize(st["x"], st["m"])
            D.dit_fp4_dequantize(st["m"], st["out"])
            return st["out"]
        D.dit_rotary(st["plan"], st["q"], st["k"], st["pos"], st["qo"].transpose(1, 2), st["ko"].transpose(1, 2),
                     inverse=case["inverse"])
        return {"q": st["qo"], "k": st["ko"]}
    if case["op"] == "rotary":
        angle = st["pos"].double()[..., st["axis"]] * st["freq"]
        cos, sin = (angle.cos() * st["amp"]).float()[:, :, None], (angle.sin() * st["amp"]).float()[:, :, None]
        if case["inverse"]:
            sin = -sin
        dim, pairs = 2 * len(st["freq"]), case["layout"] == "pairs"
        st["qo"].copy_(_turn(st["q"].float(), cos, sin, dim, pairs).transpose(1, 2))
        st["ko"].copy_(_turn(st["k"].float(), cos, sin, dim, pairs).transpose(1, 2))
        return {"q": st["qo"], "k": st["ko"]}
    fmt, K = _fmt(case), case["K"]
    idx, s, row = _quantise(st["x"], fmt)
    v = _values(idx, s, row, K)
    if case["op"] == "linear":
        widx, ws = _unpack(st["codes"], st["scales"], fmt, case["N"], K)
        w = _values(widx, ws, st["row"] if fmt == NV else torch.ones(case["N"], device="cuda"), K)
        v = v @ w.t()
    st["out"].copy_(v)
    return st["out"]


def work(case):
    size = {"bf16": 2, "fp32": 4}
    if case["op"] == "rotary":
        n = case["B"] * case["T"] * (case["Hq"] + case["Hk"])
        axes = len(case["widths"].split(","))
        dim = sum(int(v) for v in case["widths"].split(","))
        return {"bytes": 2 * n * case["d"] * size[case["x"]] + case["B"] * case["T"] * axes * 4, "flops": 3 * n * dim}
    q = 0.5 + 1.0 / BLOCK[_fmt(case)]
    if case["op"] == "quant":  # the matrix in, its 4-bit form out, that in again and the values out
        n = case["R"] * case["K"]
        return {"bytes": n * (size[case["x"]] + 2 * q + size[case["out"]]), "flops": 2 * n}
    M, N, K = case["M"], case["N"], case["K"]
    return {"bytes": M * K * size[case["x"]] + N * K * q + M * N * size[case["out"]], "flops": 2 * M * N * K}


# --------------------------------------------------------------------------------------------- in 64 bits
def _near(y):
    """y >= 0 rounded to the 4-bit values: steps of 1/2 below 2, of 1 below 4, of 2 above, ties to even; at most 6."""
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0)).double()
    return (torch.round(y / step) * step).clamp(max=6.0)


def _exact_values(x, fmt):
    """The values that the 4-bit form of x stands for, in 64 bits; where the definition rounds to 32 bits, so does this."""
    R, K = x.shape
    n = BLOCK[fmt]
    f32 = lambda v: v.float().double()  # noqa: E731
    power = lambda e: ((e.long() + 1023) << 52).view(torch.float64)  # noqa: E731
    v = _blocks(x.double(), n)
    mag = v.abs().amax(2)
    if fmt == NV:
        top = mag.amax(1)
        dead = top < 2.0 ** -100
        top = torch.where(dead, 1.0, top)
        t = f32(mag * f32(torch.full_like(top, 448.0) / top)[:, None]).clamp(max=448.0)
        quantum = power(torch.frexp(t.clamp(min=2.0 ** -6))[1] - 4)
        s = torch.round(t / quantum) * quantum
        inv = torch.where(s > 0, f32(f32(torch.full_like(top, 2688.0) / top)[:, None] / s.clamp(min=2.0 ** -9)), 0.0)
        g = torch.where(dead, 0.0, f32(top / torch.full_like(top, 2688.0)))
        s = torch.where(dead[:, None], 0.0, s)
    else:
        e = torch.where(mag > 0, torch.frexp(mag)[1] - 3, -127).clamp(-127, 127)
        s, inv, g = power(e), power(-e), torch.ones(R, dtype=torch.float64, device=x.device)
    y = f32(v * inv[:, :, None])
    return (torch.sign(y) * _near(y.abs()) * s[:, :, None] * g[:, None, None]).flatten(1)[:, :K]


def exact(case, seed):
    if case["op"] == "rotary":
        q, k, pos = _inputs(case, seed)
        f, axis, amp = _frequencies(case)
        dim, half = 2 * len(f), len(f)
        at = pos.double()[..., torch.tensor(axis, device="cuda")] * f.cuda()
        if case["inverse"]:
            at = -at
        turn = torch.polar(torch.full_like(at, amp), at)[:, :, None]
        res = {}
        for name, x in (("q", q), ("k", k)):
            y = x.double().contiguous()
            re = torch.arange(0, dim, 2) if case["layout"] == "pairs" else torch.arange(half)
            im = re + (1 if case["layout"] == "pairs" else half)
            z = torch.complex(y[..., re], y[..., im]) * turn
            y[..., re], y[..., im] = z.real, z.imag
            res[name] = y.transpose(1, 2)
        return res
    x, w = _inputs(case, seed)
    fmt = _fmt(case)
    v = _exact_values(x, fmt)
    if case["op"] == "quant":
        return v
    out = torch.empty(v.shape[0], w.shape[0], dtype=torch.float64, device="cuda")
    wv = _exact_values(w, fmt)
    for r in range(0, v.shape[0], 1024):
        out[r:r + 1024] = v[r:r + 1024] @ wv.t()
    return out
