"""The 4-bit block through the C ABI against the oracle (oracle/fp4.py), and a run of the 4-bit linear,
the rotary operator and the attention together.

Gates. An activation entering a 4-bit linear is rounded to bf16 and then to a code whose neighbours are a
quarter of it away. Downstream of the attention, whose bf16 output is off by about 2^-9 of itself, a
fraction p of about 2^-9 / 2 / (1/4) = 2^-8 of the codes flips by one step (1/4 of the value), and of the
block scales, a ninth apart, about a hundredth, each moving its codes by a tenth: sqrt(2^-8) / 4 + sqrt(1/100)
/ 10 = 0.026 of the out linear's product, RMS. The next linears see that as a perturbation of their own
inputs, of about the same effect again: gate 8e-2 RMS of the block's change of x, 2e-1 of RMS(out) at most.
With the attention's gate zero the MLP's inputs agree to fp32 rounding and flips are rare: the bf16 block's
1e-2."""

import numpy as np
import pytest
import torch

import dit_inputs as DI
import diffusion_transformer_gb300 as D
import oracle as O
from tests.gpu_util import bf16_f64, dev, dims_of, max_abs, modulation_dev, opt_dev, rms, rope_dev, workspace
from tests.test_gpu_block import _sample_rows

pytestmark = pytest.mark.gpu

NV, MX = D.DIT_FP4_NV, D.DIT_FP4_MX
FMT = pytest.mark.parametrize("fmt", [NV, MX], ids=["nv", "mx"])


def _weights(inp, fmt):
    """The four weights quantised by the library, and the values they stand for as it reads them back."""
    mats, vals = [], []
    for w in (inp.wqkv, inp.wout, inp.wup, inp.wdown):
        x = dev(O.bf16_to_f64(w).astype(np.float32))
        m = D.Fp4Matrix.empty(fmt, *x.shape)
        D.dit_fp4_quantize(x, m)
        v = torch.empty_like(x)
        D.dit_fp4_dequantize(m, v)
        mats.append(m)
        vals.append(v.cpu().numpy())
    return D.Fp4BlockWeights(mats, opt_dev(inp.norm1), opt_dev(inp.norm2), opt_dev(inp.q_norm), opt_dev(inp.k_norm)), vals


def _run(inp, w, tables=None):
    sh = inp.shape
    dims = dims_of(sh)
    txt, img = dev(inp.txt) if sh.L else None, dev(inp.img)
    tc, ts, ic, is_ = tables or rope_dev(sh)
    ws = workspace(D.dit_block_fp4_workspace_bytes(dims, w.format, sh.L, sh.N))
    ws.fill_(255)
    D.dit_block_forward_fp4(dims, w, txt, img, tc, ts, ic, is_, modulation_dev(inp), ws)
    D.dit_check()
    return np.concatenate([txt.cpu().numpy(), img.cpu().numpy()] if sh.L else [img.cpu().numpy()]).astype(np.float64)


def _oracle(inp, vals, fmt, rows=None, cos_sin=None):
    sh = inp.shape
    x = np.concatenate([inp.txt, inp.img]).astype(np.float64)
    cos, sin = cos_sin or O.rope_tables(O.positions(sh.L, sh.grid_h, sh.grid_w), sh.head_dim)
    return O.block_forward_fp4_rows(x, vals, fmt, inp.mod, inp.mod_map, cos, sin, sh.heads, sh.head_dim, rows=rows,
                                    norm1=inp.norm1, norm2=inp.norm2, q_norm=inp.q_norm, k_norm=inp.k_norm, eps=sh.eps,
                                    qk_eps=sh.qk_eps)


def _check(got, ref, x, gate_rms, gate_max, label):
    e = rms(got - ref) / rms(ref - x)
    m = max_abs(got, ref) / rms(ref)
    print(f"{label}: delta RMS error {e:.3e}, max {m:.3e}")
    assert e <= gate_rms and m <= gate_max, (label, e, m)


@FMT
@pytest.mark.parametrize("shape", ["tiny", "512sq"])
def test_block(shape, fmt):
    inp = DI.block_inputs(shape)
    sh = inp.shape
    w, vals = _weights(inp, fmt)
    rows = np.arange(sh.R) if sh.R < 512 else _sample_rows(sh, seed=5)
    got = _run(inp, w)
    x = np.concatenate([inp.txt, inp.img]).astype(np.float64)
    _check(got[rows], _oracle(inp, vals, fmt, rows), x[rows], 8e-2, 2e-1, f"fp4 block {shape}")
    assert np.array_equal(got, _run(inp, w))  # the same bits again, whatever the workspace held


@FMT
def test_mlp_branch(fmt):
    inp = DI.block_inputs("512sq")
    inp.mod[:, 2, :] = 0.0  # attention gate: x reaches the second norm unchanged
    w, vals = _weights(inp, fmt)
    rows = _sample_rows(inp.shape, seed=6)
    x = np.concatenate([inp.txt, inp.img]).astype(np.float64)
    _check(_run(inp, w)[rows], _oracle(inp, vals, fmt, rows), x[rows], 1e-2, 2e-2, "fp4 MLP branch")


def test_block_with_scaled_tables():
    # dit_rotary_tables with a scaling for grids beyond the trained one feeds the block
    inp = DI.block_inputs("tiny")
    sh = inp.shape
    widths = [8, 28, 28] if sh.head_dim == 64 else [16, 56, 56]
    spec = dict(widths=widths, scaling="yarn", factor=2.0, original=64)
    pos = np.asarray(O.positions(sh.L, sh.grid_h, sh.grid_w), np.int32).reshape(sh.R, 3)
    c, s = (torch.empty(sh.R, sh.head_dim // 2, device="cuda") for _ in range(2))
    D.dit_rotary_tables(D.RotaryPlan(**spec), dev(pos), c, s)
    f, ax, amp = O.rotary_frequencies(**spec)
    L = sh.L
    w, vals = _weights(inp, NV)
    got = _run(inp, w, (c[:L].contiguous(), s[:L].contiguous(), c[L:].contiguous(), s[L:].contiguous()))
    x = np.concatenate([inp.txt, inp.img]).astype(np.float64)
    _check(got, _oracle(inp, vals, NV, cos_sin=O.rotary_tables(pos, f, ax, amp)), x, 8e-2, 2e-1, "fp4 block, scaled tables")


@FMT
@pytest.mark.parametrize("H,heads,F,L,N", [(256, 4, 128, 0, 1), (256, 2, 384, 3, 130), (512, 8, 640, 17, 300),
                                           (1280, 10, 128, 5, 60), (3328, 26, 128, 2, 41)])
def test_block_sizes(fmt, H, heads, F, L, N):
    # odd row counts, an empty text, head widths 128 and 64: against the same linears called one by one.
    # The attention is torch's in fp32 at the narrow sizes and the library's own at the wide ones: a code flips
    # with probability e / (1/4) for an input off by e of itself and moves it by 1/4, sqrt(e / 4) RMS, so what the
    # attentions differ by (0.026 of the out linear, a fifth of the residual at width 3328, e = 0.005) is 0.036 of
    # the up linear's input, 0.05 of the SwiGLU's two factors and 0.11 after the down linear's quantiser: past
    # the gate through no fault of the linears. With one attention the inputs agree to fp32 rounding.
    g = np.random.default_rng(H + N)
    R, d = L + N, H // heads
    dims = D.DitDims(H, heads, d, F)
    bf = lambda *s: torch.from_numpy((g.standard_normal(s) * 0.05).astype(np.float32)).bfloat16().cuda()  # noqa: E731
    shapes = [(3 * H, H), (H, H), (2 * F, H), (H, F)]
    mats = []
    for s in shapes:
        m = D.Fp4Matrix.empty(fmt, *s)
        D.dit_fp4_quantize(bf(*s), m)
        mats.append(m)
    w = D.Fp4BlockWeights(mats)
    x = torch.from_numpy(g.standard_normal((R, H)).astype(np.float32)).cuda()
    mod = D.Modulation(torch.from_numpy((g.standard_normal((2, 6, H)) * 0.1).astype(np.float32)).cuda(),
                       torch.from_numpy(g.integers(0, 2, R).astype(np.int32)).cuda())
    ang = torch.from_numpy(g.uniform(-3, 3, (R, d // 2)).astype(np.float32)).cuda()
    c, s = ang.cos(), ang.sin()
    txt, img = x[:L].clone(), x[L:].clone()
    ws = workspace(D.dit_block_fp4_workspace_bytes(dims, fmt, L, N))
    D.dit_block_forward_fp4(dims, w, txt if L else None, img, c[:L].contiguous() if L else None,
                            s[:L].contiguous() if L else None, c[L:].contiguous(), s[L:].contiguous(), mod, ws)
    D.dit_check()
    # the plain composition, fp32 torch between the library's linears
    rows = mod.tensors[0][mod.tensors[1].long()]
    lws = workspace(max(D.dit_linear_fp4_workspace_bytes(fmt, R, n, k) for n, k in shapes))

    def lin(i, t):
        o = torch.empty(R, shapes[i][0], device="cuda")
        D.dit_linear_fp4(t.bfloat16(), mats[i], o, lws)
        return o

    def norm(t, which):
        return t * torch.rsqrt(t.pow(2).mean(-1, keepdim=True) + 1e-6) * (1 + rows[:, which + 1]) + rows[:, which]

    qkv = lin(0, norm(x, 0)).view(R, 3, heads, d)
    q, k = (t * torch.rsqrt(t.pow(2).mean(-1, keepdim=True) + 1e-6) for t in (qkv[:, 0], qkv[:, 1]))
    rot = lambda t: torch.stack([t[..., ::2] * c[:, None] - t[..., 1::2] * s[:, None],  # noqa: E731
                                 t[..., ::2] * s[:, None] + t[..., 1::2] * c[:, None]], -1).flatten(-2)
    q, k, v = (t.bfloat16().float().transpose(0, 1) for t in (rot(q), rot(k), qkv[:, 2]))
    if H < 1024:
        o = (torch.softmax(q @ k.transpose(1, 2) / d ** 0.5, -1) @ v).transpose(0, 1).reshape(R, H)
    else:
        vt = torch.zeros(heads, d, D.dit_vt_stride(R), dtype=torch.bfloat16, device="cuda")
        vt[:, :, :R] = v.bfloat16().transpose(1, 2)
        o = torch.empty(R, H, dtype=torch.bfloat16, device="cuda")
        D.dit_attention_qknorm(dims, R, q.bfloat16().contiguous(), k.bfloat16().contiguous(), vt, None, None, o)
    y = x + rows[:, 2] * lin(1, o)
    u = lin(2, norm(y, 3))
    y = y + rows[:, 5] * lin(3, torch.nn.functional.silu(u[:, ::2]) * u[:, 1::2])
    got = torch.cat([txt, img])
    _check(got.cpu().numpy().astype(np.float64), y.cpu().numpy().astype(np.float64), x.cpu().numpy().astype(np.float64),
           8e-2 if H < 1024 else 1e-2, 2e-1, f"fp4 block {H} {heads} {F} {L}+{N}")


def _small(g, H, heads, F, R, fmt, rope_split=False, weights=False):
    d = H // heads
    dims = D.DitDims(H, heads, d, F, rope_split=rope_split)
    t = lambda *s: torch.from_numpy(g.standard_normal(s).astype(np.float32)).cuda()  # noqa: E731
    mats = []
    for s in ((3 * H, H), (H, H), (2 * F, H), (H, F)):
        m = D.Fp4Matrix.empty(fmt, *s)
        D.dit_fp4_quantize((t(*s) * 0.05).bfloat16(), m)
        mats.append(m)
    nw = [1 + 0.2 * t(n) for n in (H, H, d, d)] if weights else [None] * 4
    ang = t(R, 3 * d // 8 if rope_split else d // 2) * 2
    return dims, mats, nw, t(R, H), t(3, 6, H) * 0.1, torch.from_numpy(g.integers(0, 3, R).astype(np.int32)).cuda(), ang


@FMT
@pytest.mark.parametrize("heads", [2, 4])
def test_block_with_norm_weights_and_split_halves(fmt, heads):
    # the first linear's epilogue against dit_qkv_rope's on the same values: the bf16 linear of the dequantised
    # weights, from a residual stream whose 4-bit codes lose nothing (h a multiple of the grid)
    H, R, d = 256, 150, 256 // heads
    g = np.random.default_rng(heads)
    for rope_split in (False, True):
        dims, mats, nw, x, rows, mp, ang = _small(g, H, heads, 256, R, fmt, rope_split, True)
        w = D.Fp4BlockWeights(mats, *nw)
        c, s = ang.cos(), ang.sin()
        img, ws = x.clone(), workspace(D.dit_block_fp4_workspace_bytes(dims, fmt, 0, R))
        D.dit_block_forward_fp4(dims, w, None, img, None, None, c, s, D.Modulation(rows, mp), ws)
        D.dit_check()
        # step by step: the library's norm, 4-bit linears, attention; torch for what lies between
        m = rows[mp.long()]
        lws = workspace(max(D.dit_linear_fp4_workspace_bytes(fmt, R, a.rows, a.cols) for a in mats))

        def lin(i, t):
            o = torch.empty(R, mats[i].rows, device="cuda")
            D.dit_linear_fp4(t, mats[i], o, lws)
            return o

        def norm(t, which, wn):
            return (t * torch.rsqrt(t.pow(2).mean(-1, keepdim=True) + 1e-6) * wn * (1 + m[:, which + 1]) + m[:, which]).bfloat16()

        qkv = lin(0, norm(x, 0, nw[0])).view(R, 3, heads, d)
        q, k = (t * torch.rsqrt(t.pow(2).mean(-1, keepdim=True) + 1e-6) * wn for t, wn in ((qkv[:, 0], nw[2]), (qkv[:, 1], nw[3])))

        def rot(t):
            cc, ss = c[:, None], s[:, None]
            if rope_split:
                n = 3 * d // 8
                a, b = t[..., :n], t[..., n:2 * n]
                return torch.cat([a * cc - b * ss, a * ss + b * cc, t[..., 2 * n:]], -1)
            a, b = t[..., ::2], t[..., 1::2]
            return torch.stack([a * cc - b * ss, a * ss + b * cc], -1).flatten(-2)

        q, k = (rot(t).bfloat16().transpose(0, 1).contiguous() for t in (q, k))
        vt = torch.zeros(heads, d, D.dit_vt_stride(R), dtype=torch.bfloat16, device="cuda")
        vt[:, :, :R] = qkv[:, 2].bfloat16().permute(1, 2, 0)
        o = torch.empty(R, H, dtype=torch.bfloat16, device="cuda")
        D.dit_attention_qknorm(dims, R, q, k, vt, nw[2], nw[3], o)
        y = x + m[:, 2] * lin(1, o)
        u = lin(2, norm(y, 3, nw[1]))
        y = y + m[:, 5] * lin(3, (torch.nn.functional.silu(u[:, ::2]) * u[:, 1::2]).bfloat16())
        f64 = lambda t: t.cpu().numpy().astype(np.float64)  # noqa: E731
        _check(f64(img), f64(y), f64(x), 8e-2, 2e-1, f"fp4 block weights split={rope_split} d={d}")


def test_block_on_16_byte_boundaries():
    # residual rows, tables and modulation rows that start on 16 bytes and not on 32: the same bits
    g = np.random.default_rng(9)
    R, L = 140, 9
    dims, mats, nw, x, rows, mp, ang = _small(g, 256, 2, 128, R, NV, weights=True)
    w = D.Fp4BlockWeights(mats, *nw)

    def at(t, shift):
        mem = torch.empty(t.numel() + 16, dtype=t.dtype, device="cuda")
        v = mem[shift:shift + t.numel()].view(t.shape)
        v.copy_(t)
        return v

    def run(shift):
        c, s = ang.cos(), ang.sin()
        parts = [at(t, shift) for t in (c[:L], s[:L], c[L:], s[L:])]
        txt, img, mod = at(x[:L], shift), at(x[L:], shift), D.Modulation(at(rows, shift), mp)
        ws = workspace(D.dit_block_fp4_workspace_bytes(dims, NV, L, R - L))
        D.dit_block_forward_fp4(dims, w, txt, img, *parts, mod, ws)
        D.dit_check()
        return torch.cat([txt, img])

    assert torch.equal(run(0), run(4))


def test_linear_rotary_attention_linear_together():
    # modulated norm -> 4-bit QKV -> rotary, head-major -> attention -> 4-bit output projection
    R, heads, d = 200, 4, 64
    H = heads * d
    g = np.random.default_rng(8)
    dims = D.DitDims(H, heads, d, 256)
    x = torch.from_numpy(g.standard_normal((R, H)).astype(np.float32)).cuda()
    mod = D.Modulation(torch.from_numpy((g.standard_normal((1, 6, H)) * 0.1).astype(np.float32)).cuda(), None)
    h = torch.empty(R, H, dtype=torch.bfloat16, device="cuda")
    D.dit_modnorm(dims, None, x, None, mod, 0, h)
    ws, mats = [], []
    for n, k in ((3 * H, H), (H, H)):
        w = torch.from_numpy((g.standard_normal((n, k)) * 0.06).astype(np.float32)).bfloat16().cuda()
        m = D.Fp4Matrix.empty(NV, n, k)
        D.dit_fp4_quantize(w, m)
        mats.append(m)
        ws.append(workspace(D.dit_linear_fp4_workspace_bytes(NV, R, n, k)))
    qkv = torch.empty(R, 3 * H, dtype=torch.bfloat16, device="cuda")
    D.dit_linear_fp4(h, mats[0], qkv, ws[0])
    plan = D.RotaryPlan([48], layout="halves", scaling="linear", factor=2.0)
    pos = torch.arange(R, dtype=torch.int32, device="cuda")[:, None].contiguous()
    q, k = (torch.empty(heads, R, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rows = qkv.view(R, 3, heads, d)
    D.dit_rotary(plan, rows[:, 0], rows[:, 1], pos, q.transpose(0, 1), k.transpose(0, 1))
    vt = torch.zeros(heads, d, D.dit_vt_stride(R), dtype=torch.bfloat16, device="cuda")
    vt[:, :, :R] = rows[:, 2].permute(1, 2, 0)
    o, out = torch.empty(R, H, dtype=torch.bfloat16, device="cuda"), torch.empty(R, H, device="cuda")
    D.dit_attention(dims, R, q, k, vt, o)
    D.dit_linear_fp4(o, mats[1], out, ws[1])
    D.dit_check()
    # each step in 64 bits from the step before it, as the GPU left that
    vals = []
    for m in mats:
        t = torch.empty(m.rows, m.cols, device="cuda")
        D.dit_fp4_dequantize(m, t)
        vals.append(t.cpu().numpy())
    S = np.abs(O.fp4_linear_f(np.abs(bf16_f64(h)), np.abs(vals[0]), NV))
    ref = O.fp4_linear_f(bf16_f64(h), vals[0], NV)
    got = bf16_f64(qkv)
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + (H / 64 + 2) * 2.0 ** -23 * S).all()
    f, ax, amp = O.rotary_frequencies([48], scaling="linear", factor=2.0)
    c, s = O.rotary_tables(pos.cpu().numpy(), f, ax, amp)
    qr, kr = (O.rotary_apply(got.reshape(R, 3, heads, d)[:, i], c, s, True) for i in (0, 1))
    for t, r in ((q, qr), (k, kr)):
        assert np.abs(bf16_f64(t).transpose(1, 0, 2) - r).max() <= 2.0 ** -8 * np.abs(r).max() + 2.0 ** -20 * np.abs(r).max()
    qh, kh, vh = bf16_f64(q), bf16_f64(k), got.reshape(R, 3, heads, d)[:, 2].transpose(1, 0, 2)
    sc = qh @ kh.transpose(0, 2, 1) / np.sqrt(d)
    pr = np.exp(sc - sc.max(-1, keepdims=True))
    ref_o = (pr / pr.sum(-1, keepdims=True) @ vh).transpose(1, 0, 2).reshape(R, H)
    assert rms(bf16_f64(o) - ref_o) <= 1e-2 * rms(ref_o)  # probabilities and output in bf16
    ref = O.fp4_linear_f(bf16_f64(o), vals[1], NV)
    S = O.fp4_linear_f(np.abs(bf16_f64(o)), np.abs(vals[1]), NV)
    assert (np.abs(out.cpu().numpy() - ref) <= (H / 64 + 2) * 2.0 ** -23 * S + 1e-30).all()


def test_block_refusals():
    dims = D.DitDims(256, 4, 64, 128)
    mk = lambda fmt, s: D.Fp4Matrix.empty(fmt, *s)  # noqa: E731
    shapes = [(768, 256), (256, 256), (256, 256), (256, 128)]
    x, c = torch.zeros(5, 256, device="cuda"), torch.zeros(5, 32, device="cuda")
    mod = D.Modulation(torch.zeros(1, 6, 256, device="cuda"), None)
    ws = workspace(D.dit_block_fp4_workspace_bytes(dims, NV, 0, 5))

    def call(mats, ws=ws):
        D.dit_block_forward_fp4(dims, D.Fp4BlockWeights(mats), None, x, None, None, c, c, mod, ws)

    good = [mk(NV, s) for s in shapes]
    for bad, why in (([good[0], good[1], good[2], mk(MX, shapes[3])], -1), ([good[0], good[1], good[2], good[1]], -1)):
        with pytest.raises(D.DitError) as e:
            call(bad)
        assert e.value.status == why
    with pytest.raises(D.DitError) as e:
        call(good, ws[:-256])
    assert e.value.status == -3
    assert D.dit_block_fp4_workspace_bytes(dims, 2, 0, 5) == 0 and D.dit_block_fp4_workspace_bytes(dims, NV, 0, 0) == 0


@FMT
@pytest.mark.parametrize("heads,part", [(h, p) for h in (2, 4) for p in range(8)])
def test_every_part_of_a_head_shows(fmt, heads, part, monkeypatch):
    # As test_block_with_norm_weights_and_split_halves (both rotary layouts), with head-norm weights of zero but for an
    # eighth of the head's columns and without the MLP, so that a wrong weight, angle or place in any of the columns
    # changes the scores by about their own size. Both sides share the attention and differ by fp32 rounding ahead of it:
    # 2^-22 of q and k, which moves 2^-13 of their bf16 values by 2^-8, a score by less than 2^-13, and the attention's
    # output, rounded to bf16, by about 2^-12 of itself. Codes are a quarter apart: sqrt(2^-12) / 2 = 0.008 of the out
    # linear, and 0.005 for the block scales that turn over (9 2^-12 of them, by a tenth). Gate: three times their root sum.
    import sys
    here = sys.modules[__name__]
    small, check = here._small, here._check

    def weights(*a):
        dims, mats, nw, x, rows, mp, ang = small(*a)
        n = len(nw[2]) // 8
        for w in nw[2:]:
            keep = w[part * n:(part + 1) * n] * 8 ** 0.5
            w.zero_()
            w[part * n:(part + 1) * n] = keep
        rows[:, 5] = 0
        return dims, mats, nw, x, rows, mp, ang

    monkeypatch.setattr(here, "_small", weights)
    monkeypatch.setattr(here, "_check", lambda got, ref, x, _, top, label: check(got, ref, x, 3e-2, top, label))
    test_block_with_norm_weights_and_split_halves(fmt, heads)
