"""A transformer block with biases over a packed batch of sequences, out of the library's single operators: QKV with bias,
normed and turned heads where they stand, attention within each sequence, output linear onto the residual rows through
gates, a GELU MLP, and the heads' gradient. Each step against 64 bits on the values that the library's step before it
left, with that operator's own gate (see their tests); then the whole run as one captured graph."""

import math

import numpy as np
import pytest
import torch

import diffusion_transformer_gb300 as D
import oracle as O
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu

H, Hk, d, F = 4, 2, 64, 512
C = H * d
LENS = [70, 1, 133, 64]
ROWS = sum(LENS)


def _np(t):
    return t.double().cpu().numpy()


def _weights():
    g = torch.Generator().manual_seed(7)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    lin = lambda n, k: ((rn(n, k) / math.sqrt(k)).bfloat16().cuda(), (0.3 * rn(n)).cuda())  # noqa: E731
    return dict(qkv=lin((H + 2 * Hk) * d, C), out=lin(C, C), up=lin(F, C), down=lin(C, F), q_norm=(1 + 0.2 * rn(d)).cuda(),
                k_norm=(1 + 0.2 * rn(d)).cuda(), gate=rn(len(LENS), C).cuda(), x=rn(ROWS, C).bfloat16().cuda())


class Run:
    def __init__(self):
        self.w = _weights()
        self.plan = D.RotaryPlan([16, 24, 24])
        self.starts = [0] + list(np.cumsum(LENS))
        self.start = dev(np.array(self.starts, np.int32))
        self.seq = torch.repeat_interleave(torch.arange(len(LENS)), torch.tensor(LENS)).int().cuda()
        pos = np.concatenate([np.arange(n) for n in LENS])
        self.pos = np.stack([pos, pos // 8, pos % 8], 1).astype(np.int32)
        self.posd = dev(self.pos)
        # a text of nine rows in front of every sequence sees itself alone
        self.visible = np.concatenate([np.where(np.arange(n) < 9, min(9, n), n) for n in LENS]).astype(np.int32)
        self.vis = dev(self.visible)
        new = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.qkv, self.heads, self.o = new(ROWS, (H + 2 * Hk) * d), new(ROWS, H + Hk, d), new(ROWS, H, d)
        self.y, self.a, self.z = new(ROWS, C), new(ROWS, F), new(ROWS, C)
        self.ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
        assert self.ws.numel() >= max(D.dit_attention_packed_workspace_bytes(ROWS, ROWS, len(LENS), H, Hk, d),
                                      *(D.dit_linear_epilogue_workspace_bytes(ROWS, n, k) for n, k in ((512, C), (C, C), (F, C), (C, F))))

    def __call__(self):
        w = self.w
        D.dit_linear_epilogue(w["x"], w["qkv"][0], self.qkv, bias=w["qkv"][1], ws=self.ws)
        v = self.qkv.view(ROWS, H + 2 * Hk, d)
        D.dit_qknorm_rotary(self.plan, v[:, :H], v[:, H:H + Hk], self.posd, w["q_norm"], w["k_norm"], self.heads[:, :H],
                            self.heads[:, H:])
        D.dit_attention_packed(self.heads[:, :H], self.heads[:, H:], v[:, H + Hk:], self.o, self.start, self.start,
                               visible=self.vis, ws=self.ws)
        D.dit_linear_epilogue(self.o.view(ROWS, C), w["out"][0], self.y, bias=w["out"][1], gate=w["gate"], gate_map=self.seq,
                              residual=w["x"], ws=self.ws)
        D.dit_linear_epilogue(self.y, w["up"][0], self.a, bias=w["up"][1], activation="gelu_tanh", ws=self.ws)
        D.dit_linear_epilogue(self.a, w["down"][0], self.z, bias=w["down"][1], residual=self.y, ws=self.ws)


def _linear(a, wb, act=None, gate=None, res=None):
    A, W, b = _np(a), _np(wb[0]), _np(wb[1])
    y = A @ W.T + b
    err = A.shape[1] * 2.0 ** -23 * (np.abs(A) @ np.abs(W).T) + 2.0 ** -23 * np.abs(y)
    if act:
        err = 1.13 * err + 2.0 ** -20 * np.maximum(1, np.abs(y))
        y = 0.5 * y * (1 + np.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)))
    if gate is not None:
        y, err = y * gate, err * np.abs(gate) + 2.0 ** -23 * np.abs(y * gate)
    if res is not None:
        y = y + _np(res)
        err = err + 2.0 ** -23 * (np.abs(y) + np.abs(_np(res)))
    return y, err


def _near(got, ref, err):
    assert (np.abs(_np(got) - ref) <= err + 2.0 ** -8 * (np.abs(ref) + err)).all()


def test_block_over_packed_sequences():
    run = Run()
    run()
    D.dit_check()
    w, v = run.w, run.qkv.view(ROWS, H + 2 * Hk, d)
    _near(run.qkv, *_linear(w["x"], w["qkv"]))
    f, ax, amp = O.rotary_frequencies([16, 24, 24])
    c, s = O.rotary_tables(run.pos, f, ax, amp)
    for cut, n in ((slice(0, H), "q_norm"), (slice(H, H + Hk), "k_norm")):
        x, wn = _np(v[:, cut]), _np(w[n])
        ref = O.qknorm_rotary(x, wn, 1e-6, c, s, False)
        size = np.abs(x / np.sqrt(np.mean(x * x, -1, keepdims=True) + 1e-6) * wn)
        pair = np.repeat(size[..., 0::2] + size[..., 1::2], 2, -1)
        _near(run.heads[:, cut], ref, 2.0 ** -19 * pair)
    q, k, val = _np(run.heads[:, :H]), _np(run.heads[:, H:]), _np(v[:, H + Hk:])
    ref, _, mag = O.attention_packed(q, k, val, run.starts, run.starts, run.visible, d ** -0.5)
    big = np.abs(q).sum(2).max() * np.abs(k).max() * d ** -0.5
    t = d * 2.0 ** -23 * big + 2.0 ** -20 * (1 + big)
    _near(run.o, ref, (2.0 ** -8 + 3 * t + ROWS * 2.0 ** -22) * mag)
    _near(run.y, *_linear(run.o.view(ROWS, C), w["out"], gate=_np(w["gate"])[run.seq.cpu().numpy()], res=w["x"]))
    _near(run.a, *_linear(run.y, w["up"], act=True))
    _near(run.z, *_linear(run.a, w["down"], res=run.y))


def test_sequences_do_not_see_each_other():
    run = Run()
    run()
    first = run.z.clone()
    run.w["x"][LENS[0]:] = torch.randn(ROWS - LENS[0], C, device="cuda").bfloat16()
    run()
    D.dit_check()
    assert torch.equal(run.z[:LENS[0]], first[:LENS[0]]) and not torch.equal(run.z, first)


def test_block_as_one_graph():
    run = Run()
    run()
    ref = run.z.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    run.z.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(run.z, ref)
    # the gradient of the heads, captured while an earlier graph lives, over its own inputs
    v, dy = run.qkv.view(ROWS, H + 2 * Hk, d), torch.randn(ROWS, H + Hk, d, device="cuda").bfloat16()
    outs = [[torch.empty(ROWS, n, d, dtype=torch.bfloat16, device="cuda") for n in (H, Hk)] + [torch.empty(d, device="cuda") for _ in range(2)]
            for _ in range(2)]
    ws = torch.empty(D.dit_qknorm_rotary_backward_workspace_bytes(d), dtype=torch.uint8, device="cuda")

    def back(o):
        D.dit_qknorm_rotary_backward(run.plan, v[:, :H], v[:, H:H + Hk], dy[:, :H], dy[:, H:], run.posd, run.w["q_norm"],
                                     run.w["k_norm"], o[0], o[1], o[2], o[3], ws)

    back(outs[0])
    second = torch.cuda.CUDAGraph()
    with torch.cuda.graph(second):
        back(outs[1])
    graph.replay()
    second.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*outs))
