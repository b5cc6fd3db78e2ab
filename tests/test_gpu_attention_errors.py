"""Joint attention under a set error word: a call may stop short wherever it waits, but what it has in flight is waited for; the
word is reported, and from then on calls are right again."""

import pytest
import torch

import diffusion_transformer_gb300 as D

pytestmark = pytest.mark.gpu


def test_calls_under_a_set_error_word():
    g = torch.Generator().manual_seed(9)
    rn = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    jobs = []
    for R, heads, d, split in ((1000, 48, 64, True), (700, 6, 128, False), (2000, 24, 128, True)):
        dims = D.DitDims(heads * d, heads, d, 256)
        x = [rn(heads, R, d) for _ in range(2)]
        q, k = (((t / t.pow(2).mean(-1, keepdim=True).sqrt()).bfloat16()) for t in x)
        vt = torch.zeros(heads, d, D.dit_vt_stride(R), dtype=torch.bfloat16, device="cuda")
        vt[:, :, :R] = rn(heads, d, R).bfloat16()
        n = D.dit_attention_workspace_bytes(dims, R) if split else 0  # the persistent schedule, where the shape takes it
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda") if n else None
        o = torch.empty(R, heads * d, dtype=torch.bfloat16, device="cuda")
        jobs.append((lambda a=(dims, R, q, k, vt), o=o, ws=ws: D.dit_attention(*a, o, ws=ws), o))  # running maximum
        o = torch.empty_like(o)
        jobs.append((lambda a=(dims, R, q, k, vt), o=o, ws=ws: D.dit_attention_qknorm(*a, None, None, o, ws=ws), o))  # fixed
    want = []
    for call, o in jobs:
        call()
        D.dit_check()
        want.append(o.clone())
    D.dit_selftest_bounded_wait(False)  # sets the word, for all that is queued behind it
    for _ in range(4):
        for call, _ in jobs:
            call()
    with pytest.raises(D.DitError) as e:
        D.dit_check()
    assert e.value.status == D.DIT_ETIMEOUT
    D.dit_check()
    for (call, o), x in zip(jobs, want):
        o.fill_(9)
        call()
        D.dit_check()
        assert torch.equal(o, x)
