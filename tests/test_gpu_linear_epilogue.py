"""The linear with a whole epilogue on the GPU against NumPy in 64 bits.

Gate. K exact products summed in fp32: off by K 2^-23 sum |a w| (a step per addition of the matrix unit, in parts or
not); the bias adds 2^-24. The activations' slopes stay below 1.13 and their own arithmetic within 2^-20 of the larger of
1 and |y|; gate and residual add 2^-23 of their terms. Then half a step of the output's type."""

import math

import numpy as np
import pytest
import torch

import diffusion_transformer_gb300 as D

pytestmark = pytest.mark.gpu

_erf = np.vectorize(math.erf)


def _act(y, name):
    if name == "silu":
        return y / (1 + np.exp(-y))
    if name == "gelu":
        return 0.5 * y * (1 + _erf(y / math.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * y * (1 + np.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)))
    return y


def _np(t):
    return t.double().cpu().numpy()


def _expect(a, w, bias, act, gate, gmap, res):
    A, W = _np(a), _np(w)
    y, err = A @ W.T, A.shape[1] * 2.0 ** -23 * (np.abs(A) @ np.abs(W).T)
    if bias is not None:
        y = y + _np(bias)
        err = err + 2.0 ** -23 * np.abs(y)
    out = _act(y, act)
    if act != "none":
        err = 1.13 * err + 2.0 ** -20 * np.maximum(1, np.abs(y))
    if gate is not None:
        g = _np(gate)[np.zeros(A.shape[0], int) if gmap is None else gmap.cpu().numpy()]
        out, err = out * g, err * np.abs(g) + 2.0 ** -23 * np.abs(out * g)
    if res is not None:
        out = out + _np(res)
        err = err + 2.0 ** -23 * (np.abs(out) + np.abs(_np(res)))
    return out, err


def _check(got, ref, err):
    g, half = _np(got), torch.finfo(got.dtype).eps / 2
    bad = np.abs(g - ref) - err - half * (np.abs(ref) + err)
    assert (bad <= 0).all(), (float(bad.max()), np.argwhere(bad > 0)[:5])


def _make(M, K, N, seed, dtype, rows):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    a, w = rn(M, K).bfloat16().cuda(), (rn(N, K) / math.sqrt(K)).bfloat16().cuda()
    return (a, w, rn(N).cuda(), rn(rows, N).cuda(), torch.randint(0, rows, (M,), generator=g, dtype=torch.int32).cuda(),
            rn(M, N).to(dtype).cuda())


def _ws(M, N, K):
    return torch.empty(max(16, D.dit_linear_epilogue_workspace_bytes(M, N, K)), dtype=torch.uint8, device="cuda")


SIZES = [(1, 8, 1), (1, 64, 64), (1, 4096, 384), (3, 1000, 777), (7, 72, 130), (64, 2048, 256), (128, 128, 128), (129, 136, 65),
         (200, 520, 1000), (333, 1000, 777), (513, 192, 320), (1000, 64, 2049)]


@pytest.mark.parametrize("M,K,N", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sizes_and_parts(M, K, N, dtype):
    a, w, bias, gate, gmap, res = _make(M, K, N, M + K, dtype, 3)
    for act, b, g, m, r in (("none", None, None, None, None), ("silu", bias, None, None, None), ("gelu", bias, gate, gmap, res),
                            ("gelu_tanh", None, gate[:1], None, None), ("none", None, None, None, res), ("none", bias, gate, gmap, None)):
        ref, err = _expect(a, w, b, act, g, m, r)
        for ws in (None, _ws(M, N, K)):
            out = torch.empty(M, N, dtype=dtype, device="cuda")
            D.dit_linear_epilogue(a, w, out, bias=b, activation=act, gate=g, gate_map=m, residual=r, ws=ws)
            D.dit_check()
            _check(out, ref, err)


@pytest.mark.parametrize("M,K,N", [(1, 14000, 520), (5, 8192, 100), (100, 6144, 512), (300, 4096, 250)])
def test_divided_k_is_repeatable(M, K, N):
    a, w, bias, gate, gmap, res = _make(M, K, N, 5, torch.float32, 2)
    n = D.dit_linear_epilogue_workspace_bytes(M, N, K)
    assert n > 0 or M <= 4  # up to four rows have a kernel of their own, which divides K within a CTA
    ref, err = _expect(a, w, bias, "silu", gate, gmap, res)
    outs = []
    for _ in range(3):
        out = torch.empty(M, N, device="cuda")
        D.dit_linear_epilogue(a, w, out, bias=bias, activation="silu", gate=gate, gate_map=gmap, residual=res,
                              ws=torch.full((max(n, 16),), 255, dtype=torch.uint8, device="cuda"))
        outs.append(out)
    D.dit_check()
    _check(outs[0], ref, err)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shift,pad", [(0, 0), (1, 0), (0, 3), (4, 8)])
def test_strides_alignment_and_in_place(dtype, shift, pad):
    M, K, N = 140, 128, 96
    a, w, bias, gate, gmap, res = _make(M, K, N, 9, dtype, 2)
    wide = torch.full((M * (N + pad) + 16,), 5.0, dtype=dtype, device="cuda")
    out = wide[shift:shift + M * (N + pad)].view(M, N + pad)[:, :N]
    out.copy_(res)
    aw, ww = torch.full((M, K + 8), 9.0, device="cuda").bfloat16(), torch.full((N, K + 16), 9.0, device="cuda").bfloat16()
    aw[:, :K], ww[:, :K] = a, w
    off = torch.empty(N + 1, device="cuda")[1:]
    off.copy_(bias)
    ref, err = _expect(a, w, bias, "gelu_tanh", gate, gmap, res)
    D.dit_linear_epilogue(aw[:, :K], ww[:, :K], out, bias=off, activation="gelu_tanh", gate=gate, gate_map=gmap, residual=out)
    D.dit_check()
    _check(out, ref, err)
    keep = torch.ones_like(wide, dtype=torch.bool)
    keep[shift:shift + M * (N + pad)].view(M, N + pad)[:, :N] = False
    assert (wide[keep] == 5).all()


def test_activations_over_their_range():
    # one product per output: y itself, from far negative to far positive, zeros and what is not finite
    y = torch.cat([torch.linspace(-100, 100, 4001), torch.linspace(-6, 6, 4001), torch.tensor([0.0, -0.0, 3e38, -3e38])]).bfloat16()
    N = y.numel()
    a = torch.zeros(1, 8)
    a[0, 0] = 1
    w = torch.zeros(N, 8)
    w[:, 0] = y.float()
    a, w = a.bfloat16().cuda(), w.bfloat16().cuda()
    for act in ("none", "silu", "gelu", "gelu_tanh"):
        out = torch.empty(1, N, device="cuda")
        D.dit_linear_epilogue(a, w, out, activation=act)
        with np.errstate(over="ignore"):
            ref = _act(y.double().numpy(), act)
        got = _np(out)[0]
        assert np.isfinite(got[:-2]).all()
        assert (np.abs(got - ref) <= 2.0 ** -20 * np.abs(y.double().numpy()) + 1e-30).all(), act
    bad = torch.tensor([float("inf"), float("nan")]).repeat(32)
    w[:64, 0] = bad.bfloat16().cuda()
    out = torch.empty(1, N, device="cuda")
    D.dit_linear_epilogue(a, w, out)
    assert torch.isnan(out[0, 1:64:2]).all() and torch.isinf(out[0, :64:2]).all() and torch.isfinite(out[0, 64:]).all()


def test_gate_rows_out_of_range_take_the_nearest():
    a, w, _, gate, gmap, _ = _make(40, 64, 48, 2, torch.float32, 3)
    far = torch.where(gmap == 2, 1000, torch.where(gmap == 0, -7, gmap))
    x, y = torch.empty(40, 48, device="cuda"), torch.empty(40, 48, device="cuda")
    D.dit_linear_epilogue(a, w, x, gate=gate, gate_map=gmap)
    D.dit_linear_epilogue(a, w, y, gate=gate, gate_map=far)
    assert torch.equal(x, y)


def test_offsets_past_32_bits():
    M, K, N, ld = 3, 64, 40, 1_200_000_008
    a, w, bias, _, _, res = _make(M, K, N, 3, torch.bfloat16, 1)
    mem = torch.empty(2 * ld + 4096, dtype=torch.bfloat16, device="cuda")
    view = lambda n, o: torch.as_strided(mem, (M, n), (ld, 1), o)  # noqa: E731
    A, R, O = view(K, 0), view(N, 256), view(N, 512)
    A.copy_(a)
    R.copy_(res)
    D.dit_linear_epilogue(A, w, O, bias=bias, residual=R)
    _check(O, *_expect(a, w, bias, "none", None, None, res))


def test_graphs_share_scratch_and_streams():
    M, K, N = 4, 8192, 256
    a, w, bias, gate, gmap, res = _make(M, K, N, 6, torch.float32, 2)
    ws, x, y = _ws(M, N, K), torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    D.dit_linear_epilogue(a, w, x, bias=bias, ws=ws)
    one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(one):
        D.dit_linear_epilogue(a, w, x, bias=bias, ws=ws)
    with torch.cuda.graph(two):
        D.dit_linear_epilogue(a, w, y, activation="gelu", residual=res, ws=ws)
    for _ in range(3):
        a.copy_(torch.randn(M, K, device="cuda").bfloat16())
        x.zero_()
        one.replay()
        two.replay()
        torch.cuda.synchronize()
        _check(x, *_expect(a, w, bias, "none", None, None, None))
        _check(y, *_expect(a, w, None, "gelu", None, None, res))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    z = torch.empty(M, N, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    D.dit_linear_epilogue(a, w, z, bias=bias, ws=ws, stream=s)
    s.synchronize()
    assert torch.equal(z, x)


def test_empty_and_binding_refusals():
    a, w, bias, gate, gmap, res = _make(6, 64, 32, 1, torch.float32, 2)
    out = torch.empty(6, 32, device="cuda")
    D.dit_linear_epilogue(a[:0], w, out[:0])
    D.dit_linear_epilogue(a, w[:0], out[:, :0])
    for args, kw in (((a.float(), w, out), {}), ((a, w.half(), out), {}), ((a.cpu(), w, out), {}), ((a, w[:, :32], out), {}),
                     ((a, w, out[:5]), {}), ((a, w, out.half()), {}), ((a, w, out), dict(activation="relu")),
                     ((a, w, out), dict(bias=bias[:8])), ((a, w, out), dict(bias=bias.bfloat16())), ((a, w, out), dict(gate=gate)),
                     ((a, w, out), dict(gate=gate, gate_map=gmap.long())), ((a, w, out), dict(gate_map=gmap)),
                     ((a, w, out), dict(residual=res.bfloat16())), ((a, w, out), dict(residual=res[:3])),
                     ((a[:, :60], w[:, :60], out), {}), ((a.t(), w, out), {}), ((a, w, out), dict(ws=torch.empty(16)))):
        with pytest.raises((TypeError, ValueError, D.DitError)):
            D.dit_linear_epilogue(*args, **kw)
    D.dit_check()
