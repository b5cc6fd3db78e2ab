"""Packed attention under a set error word: a call may stop short wherever it waits, but it returns, the word is reported, and
from then on calls are right again."""

import numpy as np
import pytest
import torch

import diffusion_transformer_gb300 as D
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu

JOBS = {  # whole tiles under a running and a fixed maximum, a part of them without keys, parts of a key range, few rows
    "plain": dict(rows=1500, keys=1500, heads=8, kv=8, d=128),
    "groups": dict(rows=700, keys=3000, heads=12, kv=3, d=64),
    "biased": dict(rows=1100, keys=1300, heads=6, kv=6, d=128, bias=True, causal=True),
    "capped": dict(rows=1100, keys=1300, heads=6, kv=2, d=64, cap=50.0, causal=True),
    "wide": dict(rows=600, keys=1300, heads=4, kv=4, d=128, cap=1000.0),
    "parts": dict(rows=300, keys=6000, heads=1, kv=1, d=64, ws=True),
    "rows": dict(rows=9, keys=9000, heads=16, kv=4, d=128, ws=True, bias=True),
    "short": dict(rows=300, keys=300, heads=8, kv=8, d=64, causal=True),
}


def _make(rows, keys, heads, kv, d, cap=0.0, bias=False, causal=False, ws=False):
    g = torch.Generator().manual_seed(rows + keys)
    rn = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    q, k, v = 2 * rn(rows, heads, d), rn(keys, kv, d), rn(keys, kv, d)
    vis = dev(np.arange(rows, dtype=np.int32) + 1 + keys - rows) if causal else None
    slope = torch.exp2(-torch.arange(1, heads + 1, device="cuda").float()) if bias else None
    n = D.dit_attention_packed_workspace_bytes(rows, keys, 1, heads, kv, d) if ws else 0
    assert n > 0 or not ws
    scratch = torch.empty(n, dtype=torch.uint8, device="cuda") if ws else None
    return lambda o: D.dit_attention_packed(q, k, v, o, visible=vis, cap=cap, slope=slope, ws=scratch), torch.empty_like(q)


def test_calls_under_a_set_error_word():
    jobs = {n: _make(**kw) for n, kw in JOBS.items()}
    want = {}
    for n, (call, o) in jobs.items():
        call(o)
        D.dit_check()
        want[n] = o.clone()
    D.dit_selftest_bounded_wait(False)  # sets the word, for all that is queued behind it
    for _ in range(4):
        for call, o in jobs.values():
            call(o)
    with pytest.raises(D.DitError) as e:
        D.dit_check()
    assert e.value.status == D.DIT_ETIMEOUT
    D.dit_check()
    for n, (call, o) in jobs.items():
        o.fill_(9)
        call(o)
        D.dit_check()
        assert torch.equal(o, want[n]), n
