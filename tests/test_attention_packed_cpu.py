"""The oracle of the packed attention pinned by hand and against the joint attention's, and the library's refusals,
which come before any CUDA call."""

import ctypes
import math

import numpy as np
import pytest

import diffusion_transformer_gb300 as D
import oracle as O


def test_one_key_and_equal_scores_and_nothing():
    v = np.arange(12.0).reshape(3, 1, 4)
    q, k = np.ones((2, 1, 4)), np.zeros((3, 1, 4))
    o, lse, _ = O.attention_packed(q, k, v, [0, 2], [0, 3])
    assert np.allclose(o, v.mean(0)) and np.allclose(lse, math.log(3))
    o, lse, _ = O.attention_packed(q, k, v, [0, 2], [0, 3], visible=[1, 0])
    assert np.allclose(o[0, 0], v[0, 0]) and (o[1] == 0).all() and lse[0, 0] == 0 and lse[0, 1] == -np.inf


def test_cap_and_bias_by_hand():
    q, k, v = np.full((1, 2, 1), 2.0), np.array([3.0, -1.0]).reshape(2, 1, 1), np.array([1.0, 0.0]).reshape(2, 1, 1)
    o, lse, _ = O.attention_packed(q, k, v, [0, 1], [0, 2], scale=0.5, cap=2.0, slope=np.array([0.0, 0.25]))
    a, b = 2 * math.tanh(1.5), 2 * math.tanh(-0.5)  # keys at distance 1 and 0
    for h, s in ((0, 0.0), (1, 0.25)):
        w = np.exp([a - s, b])
        assert np.allclose(o[0, h, 0], w[0] / w.sum()) and np.allclose(lse[h, 0], math.log(w.sum()))


def test_segments_are_apart_and_rows_outside_have_no_value():
    g = np.random.default_rng(0)
    q, k, v = g.standard_normal((9, 4, 8)), g.standard_normal((11, 2, 8)), g.standard_normal((11, 2, 8))
    o, lse, mag = O.attention_packed(q, k, v, [1, 4, 4, 8], [0, 5, 6, 10])
    assert np.isnan(o[[0, 8]]).all() and np.isnan(lse[:, [0, 8]]).all() and (np.abs(o[1:8]) <= mag[1:8]).all()
    k[0:5], v[0:5], k[10], v[10] = 7, np.nan, np.nan, np.nan
    again = O.attention_packed(q, k, v, [1, 4, 4, 8], [0, 5, 6, 10])[0]
    assert np.array_equal(o[4:8], again[4:8])


@pytest.fixture(scope="module")
def L():
    from diffusion_transformer_gb300 import build
    build.build()
    return D.lib()


def _call(L, ws=None, **kw):
    base = dict(q=1 << 12, k=1 << 13, v=1 << 14, o=1 << 15, lse=0, q_start=1 << 16, k_start=1 << 17, visible=0, slope=0,
                q_row=256, q_head=64, k_row=128, k_head=64, v_row=128, v_head=64, o_row=256, o_head=64, q_rows=5, k_rows=7,
                segments=2, heads=4, kv_heads=2, head_dim=64, scale=0.125, cap=0.0)
    base.update(kw)
    a = D.dit_packed_attention(*base.values())
    return L.dit_attention_packed(ctypes.addressof(a), ws, 1 << 20 if ws else 0, None)


def test_refusals(L):
    assert L.dit_attention_packed(None, None, 0, None) == -1
    for n in ("q", "k", "v", "o"):
        for bad in (0, (1 << 12) + 8):
            assert _call(L, **{n: bad}) == -1, n
    for n in ("q_row", "q_head", "k_row", "k_head", "v_row", "v_head", "o_row", "o_head"):
        for bad in (0, -64, 60, 1 << 39):
            assert _call(L, **{n: bad}) == -1, (n, bad)
    for n in ("lse", "q_start", "k_start", "visible", "slope"):
        assert _call(L, **{n: (1 << 18) + 2}) == -1, n
    for kw in (dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(cap=-1.0),
               dict(cap=float("nan")), dict(cap=float("inf")), dict(cap=1e-39), dict(scale=3e38), dict(cap=3e38), dict(q_start=0), dict(k_start=0), dict(q_start=0, k_start=0),
               dict(segments=1, q_start=0), dict(q_rows=-1), dict(k_rows=-1), dict(segments=-1), dict(heads=0),
               dict(kv_heads=0), dict(head_dim=0), dict(o=1 << 12), dict(o=1 << 13), dict(o=1 << 14)):
        assert _call(L, **kw) == -1, kw
    for kw in (dict(head_dim=96), dict(heads=3), dict(heads=129, kv_heads=1), dict(q_rows=2 ** 31 - 1), dict(k_rows=2 ** 31 - 1),
               dict(heads=65536, kv_heads=65536)):
        assert _call(L, **kw) == -2, kw
    assert _call(L, ws=(1 << 20) + 8) == -1
    assert _call(L, q_rows=0, q=0, o=0) == 0 and _call(L, segments=0, q_start=0, k_start=0) == 0


def test_workspace_sizes(L):
    f = D.dit_attention_packed_workspace_bytes
    assert f(0, 10, 1, 4, 2, 64) == f(4, 10, 0, 4, 2, 64) == f(4, 10, 1, 4, 3, 64) == f(4, 10, 1, 4, 2, 80) == 0
    assert f(1, 100, 1, 4, 2, 64) == 0  # too few keys to part
    for far in (2 ** 31, 2 ** 32 + 5):
        with pytest.raises(ValueError):
            f(far, 10, 1, 4, 2, 64)
