"""The linear with a whole epilogue where its arguments are extreme, in every kernel that ends in it, and its scratch across
graphs and streams where K is divided.

Gate. One exact product per output, so y is exact; an activation's arithmetic is within 2^-20 |y| (fp32 steps, arguments of the
exponential up to 100 included), and results below 1e-30 may be 0. Then half a step of the output's type."""

import math

import numpy as np
import pytest
import torch

import diffusion_transformer_gb300 as D

pytestmark = pytest.mark.gpu

_erf = np.vectorize(math.erf)


def _act(y, name):
    with np.errstate(over="ignore"):
        if name == "silu":
            return y / (1 + np.exp(-y))
        if name == "gelu":
            return 0.5 * y * (1 + _erf(y / math.sqrt(2)))
        if name == "gelu_tanh":
            return 0.5 * y * (1 + np.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)))
    return y


def _np(t):
    return t.double().cpu().numpy()


def _ws(M, N, K):
    return torch.empty(max(16, D.dit_linear_epilogue_workspace_bytes(M, N, K)), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K", [(1, 8), (8, 8), (130, 8), (8, 4096), (130, 4096)])  # rows on the plain cores, tiles, divided K
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "gelu_tanh"])
def test_activations_over_their_range(dtype, M, K, act):
    y = torch.cat([torch.linspace(-100, 100, 401), torch.linspace(-6, 6, 401), torch.tensor([0.0, -0.0, 1e-30, 3e38, -3e38])]).bfloat16()
    N = y.numel()
    a, w = torch.zeros(M, K), torch.zeros(N, K)
    a[:, K // 2], w[:, K // 2] = 1, y.float()
    a, w = a.bfloat16().cuda(), w.bfloat16().cuda()
    assert K < 4096 or D.dit_linear_epilogue_workspace_bytes(M, N, K) > 0
    ref, half = _act(y.double().numpy(), act), torch.finfo(dtype).eps / 2
    gate = 2.0 ** -20 * np.abs(y.double().numpy()) * (act != "none")
    for ws in (None, _ws(M, N, K)):
        out = torch.empty(M, N, dtype=dtype, device="cuda")
        D.dit_linear_epilogue(a, w, out, activation=act, ws=ws)
        D.dit_check()
        off = np.abs(_np(out) - ref)
        bad = ~(off <= gate + half * (np.abs(ref) + gate) + 1e-30)
        assert not bad.any(), (y[np.argwhere(bad)[0][1]].item(), _np(out)[bad][0], ref[np.argwhere(bad)[0][1]])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K", [(1, 8), (130, 8), (130, 4096)])
def test_what_is_not_finite_stays_in_its_outputs(dtype, M, K):
    g = torch.Generator().manual_seed(K)
    N = 200
    a, w = torch.randn(M, K, generator=g).bfloat16().cuda(), torch.randn(N, K, generator=g).bfloat16().cuda()
    clean, out = (torch.empty(M, N, dtype=dtype, device="cuda") for _ in range(2))
    D.dit_linear_epilogue(a, w, clean, activation="silu", ws=_ws(M, N, K))
    w[7, 3], w[100, 0] = float("nan"), float("inf")
    if M > 1:
        a[129, 1] = float("nan")
    D.dit_linear_epilogue(a, w, out, activation="silu", ws=_ws(M, N, K))
    D.dit_check()
    rows, cols = torch.arange(M, device="cuda") != 129, torch.ones(N, dtype=torch.bool, device="cuda")
    cols[7], cols[100] = False, False
    assert torch.equal(out[rows][:, cols], clean[rows][:, cols])
    assert torch.isnan(out[:, 7]).all() and not torch.isfinite(out[rows][:, 100][a[rows, 0] > 0]).any()
    assert torch.isnan(out[~rows]).all()


@pytest.mark.parametrize("M", [5, 100])
def test_graphs_share_the_scratch_of_divided_k(M):
    K, N = 8192, 256
    n = D.dit_linear_epilogue_workspace_bytes(M, N, K)
    assert n > 0
    g = torch.Generator().manual_seed(M)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    a, w, bias, res = rn(M, K).bfloat16().cuda(), (rn(N, K) / math.sqrt(K)).bfloat16().cuda(), rn(N).cuda(), rn(M, N).cuda()
    b, v = rn(M, K).bfloat16().cuda(), (rn(N, K) / math.sqrt(K)).bfloat16().cuda()
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    x, y = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    D.dit_linear_epilogue(a, w, x, bias=bias, ws=ws)
    one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(one):
        D.dit_linear_epilogue(a, w, x, bias=bias, ws=ws)
        D.dit_linear_epilogue(b, v, y, residual=res, ws=ws)  # over the same parts, straight behind
    with torch.cuda.graph(two):
        D.dit_linear_epilogue(b, w, y, bias=bias, activation="gelu", ws=ws)

    def near(got, p, q, *, bias=None, res=None, act="none"):
        P, Q = _np(p), _np(q)
        ref, err = P @ Q.T, K * 2.0 ** -23 * (np.abs(P) @ np.abs(Q).T)
        ref = ref if bias is None else ref + _np(bias)
        err = 1.13 * err + 2.0 ** -20 * np.maximum(1, np.abs(ref))
        ref = _act(ref, act)
        ref = ref if res is None else ref + _np(res)
        assert (np.abs(_np(got) - ref) <= err + 2.0 ** -22 * (np.abs(ref) + err) + 2.0 ** -22 * (0 if res is None else np.abs(_np(res)))).all()

    for i in range(3):
        a.copy_(torch.randn(M, K, device="cuda").bfloat16())
        x.zero_(), y.zero_()
        one.replay()
        z = y.clone()
        two.replay()
        torch.cuda.synchronize()
        near(x, a, w, bias=bias)
        near(z, b, v, res=res)
        near(y, b, w, bias=bias, act="gelu")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = torch.empty(M, N, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    D.dit_linear_epilogue(a, w, other, bias=bias, ws=ws, stream=s)
    s.synchronize()
    assert torch.equal(other, x)
    D.dit_check()
