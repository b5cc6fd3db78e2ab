"""Normed rotary heads and their gradient on the GPU against the oracle in 64 bits.

Gate. In fp32 with e = 2^-24: the mean square is off by at most (16 values of a lane + 5 steps of the butterfly +
the division + eps) e = 24 e, half of which reaches r, and rsqrtf is within 4 e: 16 e in all. x r w adds 2 e.
cos and sin are within 2^-22 = 4 e of 1, the two products and the sum of a turn add 2 e: (|a| + |b|) amp 24 e, below
2^-19 (|a| + |b|) amp, plus half a step of the output's type. In the gradient g = R^T dy is off by 8 e of its
(|a| + |b|) amp, each of the three factors r, x r and the mean by 16 e + 24 e more: 2^-18 of the sum of the terms'
magnitudes. A weight's gradient adds at most 2^9 terms one after another: 2^-14 of the sum of magnitudes."""

import numpy as np
import pytest
import torch

import diffusion_transformer_gb300 as D
import oracle as O
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu

SPECS = {
    "image": (dict(widths=[16, 56, 56]), 128),
    "image-pass": (dict(widths=[8, 28, 28]), 80),
    "halves": (dict(widths=[64], layout="halves"), 64),
    "three-quarters": (dict(widths=[96], layout="halves", scaling="yarn", factor=16.0, original=4096), 128),
    "odd-pairs": (dict(widths=[6, 4], scaling="linear", factor=4.0), 13),
    "odd-halves": (dict(widths=[14], layout="halves"), 17),
    "one-pair": (dict(widths=[2], layout="halves"), 2),
    "one-pair-wide": (dict(widths=[2]), 255),
    "wide": (dict(widths=[128, 128], theta=1e6), 256),
    "wide-halves": (dict(widths=[256], layout="halves"), 256),
}


def _tables(spec, pos):
    f, ax, amp = O.rotary_frequencies(**{k: v for k, v in spec.items() if k != "layout"})
    c, s = O.rotary_tables(pos, f, ax, amp)
    return c, s, amp, spec.get("layout") == "halves", len(f)


def _pair_sum(x, n, halves, amp):
    """|a| + |b| of each turned pair, times the amplitude; |x| behind them."""
    m = np.abs(x)
    i = np.arange(n)
    a, b = (i, i + n) if halves else (2 * i, 2 * i + 1)
    both = (m[..., a] + m[..., b]) * amp
    m[..., a] = both
    m[..., b] = both
    return m


def _half_step(dtype):
    return torch.finfo(dtype).eps / 2


def _check(got, ref, gate, dtype):
    g = got.float().cpu().numpy().astype(np.float64)
    gate = gate + _half_step(dtype) * (np.abs(ref) + gate)
    bad = np.abs(g - ref) / np.maximum(gate, 1e-300)
    assert (np.abs(g - ref) <= gate).all(), float(bad.max())


def _expect(spec, x, w, eps, pos):
    c, s, amp, halves, n = _tables(spec, pos)
    ref = O.qknorm_rotary(x, w, eps, c, s, halves)
    size = np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    return ref, 2.0 ** -19 * _pair_sum(x / size * (1 if w is None else w), n, halves, amp)


def _expect_grad(spec, x, dy, w, eps, pos):
    c, s, amp, halves, n = _tables(spec, pos)
    dx, dw = O.qknorm_rotary_gradient(x, dy, w, eps, c, s, halves)
    size = np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    xr, mg = np.abs(x) / size, _pair_sum(dy, n, halves, amp)
    mu = mg * (1 if w is None else np.abs(w))
    gate = 2.0 ** -18 * (mu + xr * np.mean(mu * xr, -1, keepdims=True)) / size
    return dx, dw, gate, 2.0 ** -14 * (mg * xr).sum(tuple(range(x.ndim - 1)))


def _inputs(name, dtype, B, T, Hq, Hk, seed):
    spec, d = SPECS[name]
    g = np.random.default_rng(seed)
    pos = g.integers(-10 ** 5, 10 ** 5, (B, T, len(spec["widths"]))).astype(np.int32)
    make = lambda: torch.from_numpy((g.standard_normal((B, T, Hq + 2 * Hk, d)) *  # noqa: E731
                                     np.exp(g.standard_normal((B, T, Hq + 2 * Hk, 1)))).astype(np.float32)).to(dtype)
    w = [(1 + 0.3 * g.standard_normal(d)).astype(np.float32) for _ in range(2)]
    return spec, d, pos, make(), make(), w


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("name", list(SPECS))
@pytest.mark.parametrize("B,T,Hq,Hk", [(1, 1, 1, 1), (1, 37, 3, 1), (2, 130, 5, 2)])
def test_forward(name, dtype, B, T, Hq, Hk):
    spec, d, pos, qkv, _, (wq, wk) = _inputs(name, dtype, B, T, Hq, Hk, T)
    x = qkv.float().numpy().astype(np.float64)
    m = qkv.cuda()
    q, k = m[:, :, :Hq], m[:, :, Hq:Hq + Hk]
    plan = D.RotaryPlan(**spec)
    qo, ko = (torch.empty(B, h, T, d, dtype=dtype, device="cuda").transpose(1, 2) for h in (Hq, Hk))
    D.dit_qknorm_rotary(plan, q, k, dev(pos), dev(wq), None, qo, ko, eps=1e-3)  # head-major outputs, one weight
    _check(qo, *_expect(spec, x[:, :, :Hq], wq, 1e-3, pos), dtype)
    _check(ko, *_expect(spec, x[:, :, Hq:Hq + Hk], None, 1e-3, pos), dtype)
    assert torch.equal(m.cpu(), qkv)
    D.dit_qknorm_rotary(plan, q, k, dev(pos), dev(wq), dev(wk))  # in place; v's columns stay
    _check(q, *_expect(spec, x[:, :, :Hq], wq, 1e-6, pos), dtype)
    _check(k, *_expect(spec, x[:, :, Hq:Hq + Hk], wk, 1e-6, pos), dtype)
    assert torch.equal(m[:, :, Hq + Hk:].cpu(), qkv[:, :, Hq + Hk:])
    D.dit_check()


def _backward(plan, q, k, dq, dk, pos, wq, wk, dqo=None, dko=None, eps=1e-6):
    d = q.shape[-1]
    ws = torch.empty(D.dit_qknorm_rotary_backward_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    gq, gk = torch.full((d,), 7.0, device="cuda"), torch.full((d,), 7.0, device="cuda")
    D.dit_qknorm_rotary_backward(plan, q, k, dq, dk, pos, wq, wk, dqo, dko, gq, gk, ws, eps=eps)
    return gq, gk


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("name", list(SPECS))
@pytest.mark.parametrize("B,T,Hq,Hk", [(1, 1, 1, 1), (1, 37, 3, 1), (2, 130, 5, 2)])
def test_backward(name, dtype, B, T, Hq, Hk):
    spec, d, pos, qkv, grad, (wq, wk) = _inputs(name, dtype, B, T, Hq, Hk, T + 1)
    x, dy = (t.float().numpy().astype(np.float64) for t in (qkv, grad))
    m, e = qkv.cuda(), grad.cuda()
    cut = (slice(0, Hq), slice(Hq, Hq + Hk))
    q, k, dq, dk = m[:, :, cut[0]], m[:, :, cut[1]], e[:, :, cut[0]], e[:, :, cut[1]]
    plan = D.RotaryPlan(**spec)
    outs = [torch.empty(B, h, T, d, dtype=dtype, device="cuda").transpose(1, 2) for h in (Hq, Hk)]
    got = _backward(plan, q, k, dq, dk, dev(pos), dev(wq), dev(wk), *outs, eps=1e-3)
    for z, w in ((0, wq), (1, wk)):
        dx, dw, gate, gate_w = _expect_grad(spec, x[:, :, cut[z]], dy[:, :, cut[z]], w, 1e-3, pos)
        _check(outs[z], dx, gate, dtype)
        _check(got[z], dw, gate_w, torch.float32)
    assert torch.equal(m.cpu(), qkv) and torch.equal(e.cpu(), grad)
    same = _backward(plan, q, k, dq, dk, dev(pos), dev(wq), dev(wk), *outs, eps=1e-3)
    assert torch.equal(got[0], same[0]) and torch.equal(got[1], same[1])  # one call's sums have one order
    again = _backward(plan, q, k, dq, dk, dev(pos), dev(wq), dev(wk), eps=1e-3)  # over the gradients; v's columns stay
    assert torch.equal(dq, outs[0]) and torch.equal(dk, outs[1]) and torch.equal(e[:, :, Hq + Hk:].cpu(), grad[:, :, Hq + Hk:])
    for z, w in ((0, wq), (1, wk)):  # (of other strides another: batches of dense rows are one)
        _, dw, _, gate_w = _expect_grad(spec, x[:, :, cut[z]], dy[:, :, cut[z]], w, 1e-3, pos)
        _check(again[z], dw, gate_w, torch.float32)
    D.dit_check()


@pytest.mark.parametrize("shift,pad,dtype", [(1, 0, torch.float32), (3, 5, torch.bfloat16), (8, 8, torch.bfloat16)])
def test_off_alignment_leaves_the_rest(shift, pad, dtype):
    spec, d = SPECS["image"]
    g = np.random.default_rng(shift)
    T, H = 19, 3
    x = torch.from_numpy(g.standard_normal((T, H, d)).astype(np.float32)).to(dtype)
    mem = torch.full((T * H * (d + pad) + 16,), 5.0, device="cuda", dtype=dtype)
    v = mem[shift:shift + T * H * (d + pad)].view(T, H, d + pad)[:, :, :d]
    v.copy_(x)
    pos = g.integers(-99, 999, (T, 3)).astype(np.int32)
    D.dit_qknorm_rotary(D.RotaryPlan(**spec), v, None, dev(pos))
    _check(v, *_expect(spec, x.double().numpy(), None, 1e-6, pos), dtype)
    keep = torch.ones_like(mem, dtype=torch.bool)
    keep[shift:shift + T * H * (d + pad)].view(T, H, d + pad)[:, :, :d] = False
    assert (mem[keep] == 5).all()


@pytest.mark.parametrize("B,T,Hq,Hk,d", [(1, 3000, 3, 1, 64), (700, 1, 2, 2, 128), (4, 9, 70, 0, 32), (2, 500, 1, 1, 16)])
def test_many_rows_and_heads(B, T, Hq, Hk, d):
    g = np.random.default_rng(B + T)
    spec = dict(widths=[d // 2], layout="halves")
    plan, pos = D.RotaryPlan(**spec), g.integers(0, 10 ** 4, (B, T, 1)).astype(np.int32)
    q, k, dq, dk = (torch.from_numpy(g.standard_normal((B, T, h, d)).astype(np.float32)).bfloat16() for h in (Hq, Hk, Hq, Hk))
    w = (1 + 0.3 * g.standard_normal(d)).astype(np.float32)
    qd, kd, dqd, dkd = q.cuda(), k.cuda(), dq.cuda(), dk.cuda()
    qo, ko = torch.empty(B, Hq, T, d, dtype=q.dtype, device="cuda").transpose(1, 2), torch.empty_like(kd)
    D.dit_qknorm_rotary(plan, qd, kd if Hk else None, dev(pos), dev(w), dev(w), qo, ko if Hk else None)
    got = _backward(plan, qd, kd if Hk else None, dqd, dkd if Hk else None, dev(pos), dev(w), dev(w))
    for z, (x, y, o, dx) in enumerate(((q, dq, qo, dqd), (k, dk, ko, dkd))):
        x64, y64 = x.double().numpy(), y.double().numpy()
        if not x64.size:
            assert (got[z] == 0).all()
            continue
        _check(o, *_expect(spec, x64, w, 1e-6, pos), torch.bfloat16)
        ref, dw, gate, gate_w = _expect_grad(spec, x64, y64, w, 1e-6, pos)
        _check(dx, ref, gate, torch.bfloat16)
        _check(got[z], dw, gate_w, torch.float32)
    D.dit_check()


def test_gradient_against_differences():
    spec, d = SPECS["three-quarters"]
    g = np.random.default_rng(3)
    plan, pos = D.RotaryPlan(**spec), g.integers(0, 10 ** 5, (50, 1)).astype(np.int32)
    x, y = (g.standard_normal((50, 2, d)).astype(np.float32) for _ in range(2))
    w = (1 + 0.3 * g.standard_normal(d)).astype(np.float32)
    grad = dev(y)
    gw, _ = _backward(plan, dev(x), None, grad, None, dev(pos), dev(w), None)

    def f(x, w):
        out = torch.empty(50, 2, d, device="cuda")
        D.dit_qknorm_rotary(plan, dev(x), None, dev(pos), dev(w), None, out)
        return out.double().cpu().numpy() * y

    # a step h: the difference's own curvature is below h^2 times a few, its roundings 128 values of 2^-19 of about 8
    h = 2.0 ** -5
    for at in ((0, 0, 0), (7, 1, 47), (49, 0, 95), (20, 1, 127)):
        lo, hi = x.copy(), x.copy()
        lo[at] -= h
        hi[at] += h
        diff = (f(hi, w) - f(lo, w))[at[0], at[1]].sum() / (np.float64(hi[at]) - np.float64(lo[at]))
        assert abs(diff - grad[at].item()) <= 8 * h * h + 128 * 2.0 ** -19 * 8 / (2 * h), at
    for j in (0, 50, 127):  # linear in the weights: no curvature
        lo, hi = w.copy(), w.copy()
        lo[j] -= 0.5
        hi[j] += 0.5
        a, b = f(x, hi), f(x, lo)
        gate = 2.0 ** -18 * (np.abs(a) + np.abs(b)).sum() + 1e-4
        assert abs((a - b).sum() / (np.float64(hi[j]) - np.float64(lo[j])) - gw[j].item()) <= gate


def test_offsets_past_32_bits():
    g = np.random.default_rng(4)
    ld = 1_200_000_008
    mem = torch.empty(2 * ld + 1024, dtype=torch.bfloat16, device="cuda")
    x = torch.from_numpy(g.standard_normal((3, 2, 64)).astype(np.float32)).bfloat16()
    v, out = (torch.as_strided(mem, (3, 2, 64), (ld, 64, 1), o) for o in (0, 512))
    v.copy_(x)
    pos = g.integers(0, 10 ** 5, (3, 1)).astype(np.int32)
    D.dit_qknorm_rotary(D.RotaryPlan([64]), v, None, dev(pos), None, None, out)
    _check(out, *_expect(dict(widths=[64]), x.double().numpy(), None, 1e-6, pos), torch.bfloat16)
    out.copy_(torch.ones_like(x))
    gq, _ = _backward(D.RotaryPlan([64]), v, None, out, None, dev(pos), None, None)
    dx, dw, gate, gate_w = _expect_grad(dict(widths=[64]), x.double().numpy(), np.ones((3, 2, 64)), None, 1e-6, pos)
    _check(out, dx, gate, torch.bfloat16)
    _check(gq, dw, gate_w, torch.float32)


def test_graph_streams_empty_and_binding():
    plan = D.RotaryPlan([64], layout="halves")
    q, y = torch.randn(3, 4, 2, 64, device="cuda"), torch.randn(3, 4, 2, 64, device="cuda")
    pos = torch.arange(12, dtype=torch.int32, device="cuda").view(3, 4)
    out, ref, dref = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    D.dit_qknorm_rotary(plan, q, None, pos, q_out=ref)
    gref, _ = _backward(plan, q, None, y, None, pos, None, None, dref)
    dout, gout = torch.empty_like(q), torch.empty_like(gref)
    ws = torch.empty(D.dit_qknorm_rotary_backward_workspace_bytes(64), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        D.dit_qknorm_rotary(plan, q, None, pos, q_out=out)
        D.dit_qknorm_rotary_backward(plan, q, None, y, None, pos, dq_out=dout, q_norm_grad=gout, ws=ws)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(dout, dref) and torch.equal(gout, gref)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out.zero_()
    s.wait_stream(torch.cuda.current_stream())
    D.dit_qknorm_rotary(plan, q, None, pos, q_out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, ref)
    D.dit_qknorm_rotary(plan, q[:0], None, pos[:0])
    gz, _ = _backward(plan, q[:0], None, y[:0], None, pos[:0], None, None)  # sums of nothing
    assert (gz == 0).all()
    w = torch.ones(64, device="cuda")
    for bad in (dict(q_norm=w.double()), dict(q_norm=w[:32]), dict(q_norm=w.cpu()), dict(q_norm=torch.ones(128, device="cuda")[::2]),
                dict(q_out=out.bfloat16()), dict(q_out=out[:2]), dict(eps=-1.0)):
        with pytest.raises((TypeError, ValueError, D.DitError)):
            D.dit_qknorm_rotary(plan, q, None, pos, **bad)
    for bad in (dict(ws=None), dict(ws=ws[:256]), dict(ws=ws, dq_out=out[:2]), dict(ws=ws, q_norm_grad=w[:8])):
        with pytest.raises((TypeError, ValueError, D.DitError)):
            D.dit_qknorm_rotary_backward(plan, q, None, y, None, pos, **bad)


def test_rows_that_are_not_finite_stay_alone():
    plan = D.RotaryPlan([64])
    x = torch.randn(40, 3, 64, device="cuda")
    y = torch.randn(40, 3, 64, device="cuda")
    pos = torch.arange(40, dtype=torch.int32, device="cuda").view(40, 1)
    ref, dref = torch.empty_like(x), torch.empty_like(x)
    D.dit_qknorm_rotary(plan, x, None, pos, q_out=ref)
    _backward(plan, x, None, y, None, pos, None, None, dref)
    bad = x.clone()
    bad[7, 1, 3], bad[9, 0, 5], bad[11] = float("nan"), float("inf"), 0
    out, dout = torch.empty_like(x), torch.empty_like(x)
    D.dit_qknorm_rotary(plan, bad, None, pos, q_out=out)
    _backward(plan, bad, None, y, None, pos, None, None, dout)
    same = torch.ones(40, 3, dtype=torch.bool, device="cuda")
    same[7, 1] = same[9, 0] = same[11] = False
    assert torch.equal(out[same], ref[same]) and torch.equal(dout[same], dref[same])
    assert (out[11] == 0).all() and torch.isfinite(dout[11]).all() and not torch.isfinite(out[7, 1]).all()
