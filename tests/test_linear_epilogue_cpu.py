"""Refusals of the linear with a whole epilogue, before any CUDA call, and its scratch sizes."""

import ctypes

import pytest

import diffusion_transformer_gb300 as D


@pytest.fixture(scope="module")
def L():
    from diffusion_transformer_gb300 import build
    build.build()
    return D.lib()


def _call(L, a=1 << 12, M=5, lda=64, K=64, w=1 << 13, N=24, ldw=64, out=1 << 14, type=0, ldo=24, ws=None, **kw):
    e = dict(bias=0, gate=0, gate_map=0, residual=0, ld_gate=24, ld_residual=24, gate_rows=1, activation=0)
    e.update(kw)
    e = D.dit_epilogue(*e.values())
    return L.dit_linear_epilogue(a, M, lda, K, w, N, ldw, ctypes.addressof(e), out, type, ldo, ws, 1 << 20 if ws else 0, None)


def test_refusals(L):
    assert L.dit_linear_epilogue(1 << 12, 5, 64, 64, 1 << 13, 24, 64, None, 1 << 14, 0, 24, None, 0, None) == -1
    for kw in (dict(a=0), dict(a=(1 << 12) + 8), dict(w=0), dict(w=(1 << 13) + 2), dict(out=0), dict(out=(1 << 14) + 1), dict(type=1, out=(1 << 14) + 2),
               dict(type=2), dict(M=-1), dict(N=-1), dict(K=0), dict(lda=56), dict(lda=68), dict(lda=1 << 39), dict(ldw=56), dict(ldw=68),
               dict(ldo=23), dict(activation=4), dict(activation=-1), dict(bias=3), dict(gate=2), dict(gate_map=1), dict(residual=1),
               dict(residual=1 << 15, ld_residual=23), dict(residual=1 << 14, ld_residual=25), dict(gate=1 << 15, gate_rows=0),
               dict(gate=1 << 15, gate_rows=2, ld_gate=23), dict(out=1 << 12), dict(out=1 << 13), dict(ws=(1 << 20) + 8)):
        assert _call(L, **kw) == -1, kw
    for kw in (dict(K=60), dict(K=65), dict(M=(1 << 30) + 1), dict(N=(1 << 30) + 1), dict(K=(1 << 30) + 8)):
        assert _call(L, **kw) == -2, kw
    assert _call(L, M=0, a=0, out=0) == 0 and _call(L, N=0, w=0, out=0) == 0


def test_scratch_sizes(L):
    f = D.dit_linear_epilogue_workspace_bytes
    assert f(0, 8, 8) == f(8, 0, 8) == f(8, 8, 0) == f(8, 8, 12) == 0
    assert f(1, 64, 64) == 0
    for far in (2 ** 31, 2 ** 32 + 8):
        with pytest.raises(ValueError):
            f(far, 8, 8)
