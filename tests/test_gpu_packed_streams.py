"""The packed operators at once on several streams, each with its own scratch: what a call alone gives, bit by bit."""

import pytest
import torch

import diffusion_transformer_gb300 as D

pytestmark = pytest.mark.gpu


def _ws(n):
    return torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")


def _calls(seed):
    """(call of a stream, outputs) of each operator, over inputs of this seed."""
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    out = []
    for rows, keys, heads, kv, d, cap in ((1100, 1100, 8, 8, 128, 0.0), (700, 1500, 8, 2, 64, 50.0), (6, 5000, 16, 4, 128, 0.0), (300, 300, 12, 12, 64, 30.0)):
        q, k, v = rn(rows, heads, d).bfloat16(), rn(keys, kv, d).bfloat16(), rn(keys, kv, d).bfloat16()
        o, lse = torch.empty_like(q), torch.empty(heads, rows, device="cuda")
        ws = _ws(D.dit_attention_packed_workspace_bytes(rows, keys, 1, heads, kv, d))
        out.append((lambda s, a=(q, k, v, o), c=cap, lse=lse, ws=ws: D.dit_attention_packed(*a, cap=c, lse=lse, ws=ws, stream=s), [o, lse]))
    for M, K, N in ((1, 2048, 512), (20, 8192, 256), (500, 512, 1000)):
        a, w, bias, res = rn(M, K).bfloat16(), rn(N, K).bfloat16(), rn(N), rn(M, N)
        o, ws = torch.empty(M, N, device="cuda"), _ws(D.dit_linear_epilogue_workspace_bytes(M, N, K))
        out.append((lambda s, a=(a, w, o), b=bias, r=res, ws=ws: D.dit_linear_epilogue(*a, bias=b, activation="silu", residual=r, ws=ws, stream=s), [o]))
    plan = D.RotaryPlan(widths=[16, 24, 24], layout="pairs", theta=10000.0)
    q, k, dq, dk = (rn(900, h, 64).bfloat16() for h in (6, 2, 6, 2))
    w, pos = rn(64), torch.randint(-9, 900, (900, 3), generator=g, dtype=torch.int32).cuda()
    oq, ok, xq, xk, gq, gk = *(torch.empty_like(t) for t in (q, k, q, k)), torch.empty(64, device="cuda"), torch.empty(64, device="cuda")
    ws = _ws(D.dit_qknorm_rotary_backward_workspace_bytes(64))
    out.append((lambda s: D.dit_qknorm_rotary(plan, q, k, pos, w, None, oq, ok, stream=s), [oq, ok]))
    out.append((lambda s: D.dit_qknorm_rotary_backward(plan, q, k, dq, dk, pos, w, None, xq, xk, gq, gk, ws, stream=s), [xq, xk, gq, gk]))
    return out


def test_calls_on_several_streams_at_once():
    streams = [torch.cuda.Stream() for _ in range(4)]
    sets = [_calls(i) for i in range(4)]
    want = []
    for calls in sets:
        for call, outs in calls:
            call(None)
            want.append([t.clone() for t in outs])
            [t.zero_() for t in outs]
    D.dit_check()
    torch.cuda.synchronize()
    for turn in range(6):
        for i in range(len(sets[0])):
            for j, (s, calls) in enumerate(zip(streams, sets)):  # another operator on each stream
                calls[(i + 2 * j + turn) % len(calls)][0](s)
    torch.cuda.synchronize()
    D.dit_check()
    got = [outs for calls in sets for _, outs in calls]
    for g, w in zip(got, want):
        for a, b in zip(g, w):
            assert torch.equal(a, b)
