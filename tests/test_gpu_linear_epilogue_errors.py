"""The linear with a whole epilogue under a set error word: a call may stop short wherever it waits, but what it has in flight is
waited for; the word is reported, and from then on calls are right again."""

import pytest
import torch

import diffusion_transformer_gb300 as D

pytestmark = pytest.mark.gpu


def test_calls_under_a_set_error_word():
    g = torch.Generator().manual_seed(4)
    rn = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    jobs = []
    for M, K, N in ((2000, 2048, 4096), (333, 1000, 777), (20, 8192, 256), (1, 4096, 512), (100, 512, 3000)):  # pairs, single CTAs, divided K, rows
        a, w, res = rn(M, K).bfloat16(), rn(N, K).bfloat16(), rn(M, N)
        n = D.dit_linear_epilogue_workspace_bytes(M, N, K)
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
        jobs.append((a, w, res, ws, torch.empty(M, N, device="cuda")))
    run = lambda a, w, res, ws, out: D.dit_linear_epilogue(a, w, out, activation="silu", residual=res, ws=ws)  # noqa: E731
    want = []
    for j in jobs:
        run(*j)
        D.dit_check()
        want.append(j[-1].clone())
    D.dit_selftest_bounded_wait(False)  # sets the word, for all that is queued behind it
    for _ in range(4):
        for j in jobs:
            run(*j)
    with pytest.raises(D.DitError) as e:
        D.dit_check()
    assert e.value.status == D.DIT_ETIMEOUT
    D.dit_check()
    for j, x in zip(jobs, want):
        j[-1].fill_(9)
        run(*j)
        D.dit_check()
        assert torch.equal(j[-1], x)
