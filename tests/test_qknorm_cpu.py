"""The oracle of the normed rotary heads pinned by hand and by differences, and the library's refusals, which come
before any CUDA call."""

import ctypes

import numpy as np
import pytest

import diffusion_transformer_gb300 as D
import oracle as O


def test_norm_and_turn_by_hand():
    c, s = np.array([[0.0]]), np.array([[1.0]])  # a quarter turn
    x = np.array([[[3.0, 4.0, 0.0, 0.0]]])      # root of the mean square: 2.5
    assert np.allclose(O.qknorm_rotary(x, None, 0.0, c, s, False), [[[-1.6, 1.2, 0, 0]]])
    assert np.allclose(O.qknorm_rotary(x, np.array([1.0, 2, 3, 4]), 0.0, c, s, False), [[[-3.2, 1.2, 0, 0]]])
    assert np.allclose(O.qknorm_rotary(x, None, 18.75, c, s, False), [[[-0.8, 0.6, 0, 0]]])  # 6.25 + eps = 25


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("weights", [False, True])
def test_gradient_against_differences(halves, weights):
    g = np.random.default_rng(5)
    x, dy = g.standard_normal((3, 2, 10)), g.standard_normal((3, 2, 10))
    w = g.standard_normal(10) if weights else None
    c, s = O.rotary_tables(g.integers(-50, 50, (3, 1)), np.array([1.0, 0.3, 0.02]), np.array([0, 0, 0]), 1.25)
    f = lambda x, w: (dy * O.qknorm_rotary(x, w, 0.125, c, s, halves)).sum()  # noqa: E731
    dx, dw = O.qknorm_rotary_gradient(x, dy, w, 0.125, c, s, halves)
    h = 1e-5
    for at in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[at] = h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dx[at]) < 1e-8
    one = np.ones(10) if w is None else w
    for j in range(10):
        e = np.zeros(10)
        e[j] = h
        assert abs((f(x, one + e) - f(x, one - e)) / (2 * h) - dw[j]) < 1e-8


def _rows(**kw):
    base = dict(x=256, out=1 << 20, heads=2, x_batch=0, x_row=256, x_head=128, out_batch=0, out_row=256, out_head=128)
    base.update(kw)
    return D.dit_rotary_rows(*base.values())


def _grad(**kw):
    base = dict(x=256, dy=1 << 20, dx=1 << 21, heads=2, x_batch=0, x_row=256, x_head=128, dy_batch=0, dy_row=256, dy_head=128,
                dx_batch=0, dx_row=256, dx_head=128)
    base.update(kw)
    return D.dit_rotary_grad(*base.values())


@pytest.fixture(scope="module")
def L():
    from diffusion_transformer_gb300 import build
    build.build()
    return D.lib()


def _forward(L, q, k=None, plan=None, eps=1e-6, type=0, batch=1, rows=3, dim=128, pos=4096, wq=None):
    plan = plan or D.RotaryPlan([16, 56, 56])
    r = lambda t: None if t is None else ctypes.addressof(t)  # noqa: E731
    return L.dit_qknorm_rotary(plan.ref, r(q), r(k), wq, None, eps, type, batch, rows, dim, pos, None)


def test_forward_refusals(L):
    k = _rows(x=1 << 22, out=1 << 23)
    for kw in (dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(type=2), dict(batch=-1), dict(rows=-1),
               dict(dim=126), dict(pos=None), dict(pos=4097), dict(wq=258)):
        assert _forward(L, _rows(), k, **kw) == -1, kw
    assert _forward(L, _rows(), None, dim=258) == -2
    assert _forward(L, None) == -1
    assert _forward(L, _rows(heads=-1)) == -1 and _forward(L, _rows(heads=(1 << 20) + 1)) == -2
    assert _forward(L, _rows(x=None)) == -1 and _forward(L, _rows(out=None)) == -1 and _forward(L, _rows(x=257)) == -1
    assert _forward(L, _rows(out_row=0)) == -1 and _forward(L, _rows(out_head=0)) == -1
    assert _forward(L, _rows(), _rows()) == -1                                 # one output for both
    assert _forward(L, _rows(), _rows(x=1 << 20, out=1 << 23)) == -1            # k reads what q writes
    assert _forward(L, _rows(out=256, out_row=512)) == -1                      # in place under other strides
    assert _forward(L, _rows(heads=0)) == 0 and _forward(L, _rows(), rows=0) == 0 and _forward(L, _rows(), batch=0, pos=None) == 0


def test_backward_refusals(L):
    plan = D.RotaryPlan([16, 56, 56])
    n = D.dit_qknorm_rotary_backward_workspace_bytes(128)
    assert n > 0 and D.dit_qknorm_rotary_backward_workspace_bytes(0) == 0 == D.dit_qknorm_rotary_backward_workspace_bytes(257)

    def call(q, k=None, eps=1e-6, dim=128, rows=3, ws=1 << 30, ws_bytes=n, gq=None, gk=None):
        r = lambda t: None if t is None else ctypes.addressof(t)  # noqa: E731
        return L.dit_qknorm_rotary_backward(plan.ref, r(q), r(k), None, None, eps, 0, 1, rows, dim, 4096, gq, gk, ws, ws_bytes, None)

    assert call(None) == -1 and call(_grad(), eps=-1.0) == -1 and call(_grad(), dim=100) == -1
    assert call(_grad(), ws=None) == -3 and call(_grad(), ws_bytes=n - 1) == -3 and call(_grad(), ws=(1 << 30) + 16) == -1
    assert call(_grad(), gq=4097) == -1 and call(_grad(), gq=4096, gk=4096) == -1
    assert call(_grad(dy=None)) == -1 and call(_grad(dx=3)) == -1 and call(_grad(dx_row=0)) == -1
    assert call(_grad(dx=256, dx_row=512)) == -1 and call(_grad(dx=1 << 20, dx_head=256)) == -1
    assert call(_grad(), _grad()) == -1                                        # one dx for both
    assert call(_grad(dx=1 << 25), _grad(x=1 << 23, dy=1 << 25, dx=1 << 24)) == -1  # q's dx over k's dy
    assert call(_grad(), rows=0) == 0                                          # nothing asked for, nothing launched
