"""Rotary positions on the GPU against the oracle in 64 bits (oracle/rotary.py).

Gate. cos and sin carry 2^-23 or less (sincospif is within one unit, the angle's residual of at most an
eighth turn is rounded to 24 bits: pi/4 2^-24; the amplitude's product half a unit): 2^-22 of 1 in all,
times the amplitude. A turned value is two products and a sum: |error| <= (2^-22 + 2 2^-23) (|a| + |b|) amp in
fp32, plus half a step of the output type (2^-8 of the value in bf16). Passed values are equal bit for bit."""

import numpy as np
import pytest
import torch

import diffusion_transformer_gb300 as D
import oracle as O
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu

SPECS = {
    "image": (dict(widths=[16, 56, 56]), 128),
    "image-pass": (dict(widths=[8, 28, 28], layout="pairs"), 80),
    "halves": (dict(widths=[128], layout="halves"), 128),
    "three-quarters": (dict(widths=[96], layout="halves", scaling="yarn", factor=16.0, original=4096), 128),
    "odd-pairs": (dict(widths=[6, 4], layout="pairs", scaling="linear", factor=4.0), 13),
    "odd-halves": (dict(widths=[14], layout="halves", scaling="ntk", factor=2.0), 17),
    "one-pair": (dict(widths=[2], layout="halves"), 2),
    "wide": (dict(widths=[128, 128], layout="pairs", theta=1e6), 256),
    "grid-yarn": (dict(widths=[16, 56, 56], scaling="yarn", factor=2.0, original=64), 128),
}


def _expected(spec, x, pos, inverse):
    f, ax, amp = O.rotary_frequencies(**{k: v for k, v in spec.items() if k != "layout"})
    halves = spec.get("layout") == "halves"
    c, s = O.rotary_tables(pos, f, ax, amp)
    ref = O.rotary_apply(x, c, s, halves, inverse)
    mag = np.zeros_like(ref)
    n = len(f)
    i = np.arange(n)
    a, b = (i, i + n) if halves else (2 * i, 2 * i + 1)
    mag[..., a] = mag[..., b] = (np.abs(x[..., a]) + np.abs(x[..., b])) * amp
    return ref, mag, 2 * n


def _check(got, ref, mag, dim, x, dtype):
    g = got.float().cpu().numpy().astype(np.float64)
    gate = 2.0 ** -21 * mag + (2.0 ** -8 * np.abs(ref) if dtype == torch.bfloat16 else 2.0 ** -24 * np.abs(ref))
    bad = np.abs(g - ref) > gate
    assert not bad[..., :dim].any(), (int(bad.sum()), float((np.abs(g - ref) / np.maximum(gate, 1e-300))[..., :dim].max()))
    assert np.array_equal(g[..., dim:], x[..., dim:])


def _positions(g, shape, far):
    p = g.integers(-far, far, shape).astype(np.int32)
    p.reshape(-1)[:2] = [0, far][:p.size]
    return p


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("name", list(SPECS))
@pytest.mark.parametrize("B,T,Hq,Hk,far", [(1, 1, 1, 1, 5), (1, 37, 3, 1, 10 ** 4), (2, 130, 5, 2, 10 ** 6)])
def test_rotary(name, dtype, B, T, Hq, Hk, far):
    spec, d = SPECS[name]
    g = np.random.default_rng(d * T + Hq)
    axes = len(spec["widths"])
    pos = _positions(g, (B, T, axes), far)
    plan = D.RotaryPlan(**spec)
    qkv = torch.from_numpy(g.standard_normal((B, T, Hq + 2 * Hk, d)).astype(np.float32)).to(dtype)
    x = qkv.float().numpy().astype(np.float64)
    dq = qkv.cuda()
    q, k = dq[:, :, :Hq], dq[:, :, Hq:Hq + Hk]
    for inverse in (False, True):
        qo = torch.empty(B, Hq, T, d, dtype=dtype, device="cuda").transpose(1, 2)
        ko = torch.empty(B, Hk, T, d, dtype=dtype, device="cuda").transpose(1, 2)
        D.dit_rotary(plan, q, k, dev(pos), qo, ko, inverse=inverse)
        ref, mag, dim = _expected(spec, x, pos, inverse)
        _check(qo, ref[:, :, :Hq], mag[:, :, :Hq], dim, x[:, :, :Hq], dtype)
        _check(ko, ref[:, :, Hq:Hq + Hk], mag[:, :, Hq:Hq + Hk], dim, x[:, :, Hq:Hq + Hk], dtype)
    assert torch.equal(dq.cpu(), qkv)  # the inputs stay
    D.dit_rotary(plan, q, k, dev(pos))   # in place, v's columns untouched
    ref, mag, dim = _expected(spec, x, pos, False)
    _check(dq[:, :, :Hq + Hk], ref[:, :, :Hq + Hk], mag[:, :, :Hq + Hk], dim, x[:, :, :Hq + Hk], dtype)
    assert torch.equal(dq[:, :, Hq + Hk:].cpu(), qkv[:, :, Hq + Hk:])
    D.dit_check()


@pytest.mark.parametrize("shift,pad", [(1, 0), (0, 1), (3, 5)])
def test_rotary_off_alignment(shift, pad):
    spec, d = SPECS["image"]
    g = np.random.default_rng(shift)
    T, H = 19, 3
    x = g.standard_normal((T, H, d)).astype(np.float32)
    mem = torch.full((T * H * (d + pad) + 8,), 5.0, device="cuda")
    v = mem[shift:shift + T * H * (d + pad)].view(T, H, d + pad)[:, :, :d]
    v.copy_(torch.from_numpy(x))
    pos = _positions(g, (T, 3), 999)
    D.dit_rotary(D.RotaryPlan(**spec), v, None, dev(pos))
    ref, mag, dim = _expected(spec, x.astype(np.float64), pos, False)
    _check(v, ref, mag, dim, x.astype(np.float64), torch.float32)
    keep = torch.ones_like(mem, dtype=torch.bool)
    keep[shift:shift + T * H * (d + pad)].view(T, H, d + pad)[:, :, :d] = False
    assert (mem[keep] == 5).all()


def test_rotary_is_its_own_gradient_and_matches_differences():
    # the transpose against the forward map: <y, R x> = <R^T y, x>, and a difference quotient of <y, R x>
    spec, d = SPECS["three-quarters"]
    g = np.random.default_rng(3)
    plan, pos = D.RotaryPlan(**spec), _positions(g, (50, 1), 10 ** 5)
    x, y = (g.standard_normal((50, 2, d)).astype(np.float32) for _ in range(2))
    fwd, bwd = torch.empty(50, 2, d, device="cuda"), torch.empty(50, 2, d, device="cuda")
    D.dit_rotary(plan, dev(x), None, dev(pos), fwd)
    D.dit_rotary(plan, dev(y), None, dev(pos), bwd, inverse=True)
    grad = bwd.cpu().numpy().astype(np.float64)
    lhs = (fwd.cpu().numpy().astype(np.float64) * y).sum()
    assert abs(lhs - (grad * x).sum()) <= 2.0 ** -20 * np.abs(x).sum() * np.abs(y).max() * plan.c.amplitude
    h = np.float32(2.0 ** -2)
    for at in ((0, 0, 0), (7, 1, 47), (49, 0, 95), (20, 1, 100)):
        xp = x.copy()
        xp[at] += h
        step = np.float64(xp[at]) - np.float64(x[at])
        out = torch.empty(50, 2, d, device="cuda")
        D.dit_rotary(plan, dev(xp), None, dev(pos), out)
        diff = ((out.double() - fwd.double()).cpu().numpy() * y).sum() / step
        # two values change; each of their four roundings is 2^-21 of values of at most 8
        assert abs(diff - grad[at]) <= 4 * 2.0 ** -21 * 8 * np.abs(y).max() * plan.c.amplitude / step + 1e-5


def test_far_positions_are_as_exact_as_near_ones():
    plan = D.RotaryPlan([128])
    pos = np.array([[-2 ** 31], [2 ** 31 - 1], [2 ** 24 + 1], [-(2 ** 30) - 7]], np.int32)
    cos, sin = torch.empty(4, 64, device="cuda"), torch.empty(4, 64, device="cuda")
    D.dit_rotary_tables(plan, dev(pos), cos, sin)
    D.dit_check()
    # whole turns off in rational arithmetic, from the plan's own fractions
    for r, p in enumerate(pos[:, 0]):
        for i in range(64):
            t = (int(p) * plan.c.turns[i]) % (1 << 64)
            a = (t if t < 1 << 63 else t - (1 << 64)) * 2.0 ** -64 * 2 * np.pi
            assert abs(cos[r, i].item() - np.cos(a)) <= 2.0 ** -22 and abs(sin[r, i].item() - np.sin(a)) <= 2.0 ** -22
    # and the fractions are those of the formula to the last place of 64-bit arithmetic
    f, _, _ = O.rotary_frequencies([128])
    want = np.cos(np.longdouble(1) * (pos.astype(np.float64) * f[None]))
    near = np.abs(pos) * f[None] < 2.0 ** 26  # where 64-bit angles still carry the cosine
    assert np.abs(cos.cpu().numpy() - want)[near].max() <= 2.0 ** -21


def test_tables_feed_the_blocks_rotary():
    # grid positions without scaling: the tables of dit_rope_tables
    L, gh, gw, d = 7, 6, 10, 128
    pos = [(i, i, i) for i in range(L)] + [(L, y - (gh - gh // 2), x - (gw - gw // 2)) for y in range(gh) for x in range(gw)]
    R = len(pos)
    a, b, c, e = (torch.empty(R, d // 2, device="cuda") for _ in range(4))
    D.dit_rope_tables(L, gh, gw, d, a, b)
    D.dit_rotary_tables(D.RotaryPlan([16, 56, 56]), torch.tensor(pos, dtype=torch.int32, device="cuda"), c, e)
    assert (a - c).abs().max() <= 2.0 ** -22 and (b - e).abs().max() <= 2.0 ** -22


@pytest.mark.parametrize("B,T,Hq,Hk,d", [(1, 3000, 3, 1, 64), (700, 1, 2, 2, 128), (4, 9, 70, 0, 32), (2, 500, 1, 1, 16)])
def test_rotary_many_rows_and_heads(B, T, Hq, Hk, d):
    # rows grouped in a CTA, batches of single rows, more units than threads, one tensor alone
    g = np.random.default_rng(B + T)
    plan, pos = D.RotaryPlan([d // 2], layout="halves"), _positions(g, (B, T, 1), 10 ** 6)
    q, k = (torch.from_numpy(g.standard_normal((B, T, h, d)).astype(np.float32)).bfloat16() for h in (Hq, Hk))
    qd, kd = q.cuda(), k.cuda()
    qo, ko = torch.empty(B, Hq, T, d, dtype=q.dtype, device="cuda"), torch.empty_like(kd)
    D.dit_rotary(plan, qd, kd if Hk else None, dev(pos), qo.transpose(1, 2), ko if Hk else None)
    for x, y in ((q, qo.transpose(1, 2)), (k, ko))[:2 if Hk else 1]:
        x64 = x.float().numpy().astype(np.float64)
        ref, mag, dim = _expected(dict(widths=[d // 2], layout="halves"), x64, pos, False)
        _check(y, ref, mag, dim, x64, torch.bfloat16)
    D.dit_check()


def test_rotary_offsets_past_32_bits():
    g = np.random.default_rng(4)
    ld = 1_200_000_008
    mem = torch.empty(2 * ld + 1024, dtype=torch.bfloat16, device="cuda")
    x = torch.from_numpy(g.standard_normal((3, 2, 64)).astype(np.float32)).bfloat16()
    v = torch.as_strided(mem, (3, 2, 64), (ld, 64, 1))
    v.copy_(x)
    out = torch.as_strided(mem, (3, 2, 64), (ld, 64, 1), 512)
    pos = _positions(g, (3, 1), 10 ** 5)
    D.dit_rotary(D.RotaryPlan([64]), v, None, dev(pos), out)
    x64 = x.float().numpy().astype(np.float64)
    ref, mag, dim = _expected(dict(widths=[64]), x64, pos, False)
    _check(out, ref, mag, dim, x64, torch.bfloat16)


def test_rotary_graph_and_empty_and_binding():
    plan = D.RotaryPlan([64], layout="halves")
    q = torch.randn(3, 4, 2, 64, device="cuda")
    pos = torch.arange(12, dtype=torch.int32, device="cuda").view(3, 4)
    out, ref = torch.empty_like(q), torch.empty_like(q)
    D.dit_rotary(plan, q, None, pos, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        D.dit_rotary(plan, q, None, pos, out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref)
    D.dit_rotary(plan, q[:0], None, pos[:0])
    D.dit_rotary(plan, q[:, :, :0], None, pos)
    for bad in (q.half(), q.cpu(), q[0, 0], q.transpose(2, 3)):
        with pytest.raises((TypeError, ValueError)):
            D.dit_rotary(plan, bad, None, pos)
    with pytest.raises(ValueError):
        D.dit_rotary(plan, q, q[:2], pos)
    with pytest.raises(ValueError):
        D.dit_rotary(plan, q, None, pos[:, :3])
    with pytest.raises(TypeError):
        D.dit_rotary(plan, q, None, pos.long())
    with pytest.raises(D.DitError):
        D.dit_rotary(D.RotaryPlan([128]), q, None, pos)
