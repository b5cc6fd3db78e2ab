"""The 4-bit block's binding refuses tensors smaller than the dimensions say and tensors on another device (stand-ins
for tensors and for the library: no GPU)."""

import types

import pytest
import torch

import diffusion_transformer_gb300 as D
from tests.test_binding_sizes_cpu import Rows

F32 = torch.float32
L, N, H, HEADS, DIM, FFN = 3, 5, 256, 4, 64, 128


class On(Rows):
    def __init__(self, *shape, device=0):
        super().__init__(*shape, dtype=F32)
        self.device = device

    def get_device(self):
        return self.device


def _matrices(device=0):
    return [types.SimpleNamespace(c=D.dit_fp4_matrix(0, n, k, 256, 256, 256), format=0, rows=n, cols=k, device=device)
            for n, k in ((3 * H, H), (H, H), (2 * FFN, H), (H, FFN))]


@pytest.fixture
def call(monkeypatch):
    made = []
    D._torch()
    stub = types.SimpleNamespace(dit_block_forward_fp4=lambda *a: made.append(a) or 0)
    monkeypatch.setattr(D, "lib", lambda: stub)
    monkeypatch.setattr(D, "_current", lambda stream: (0, 0))
    monkeypatch.setattr(D, "_stream", lambda stream: 0)
    monkeypatch.setattr(D, "_ptr", lambda t, *a: None if t is None else 256)

    def run(mats=None, norms=(None,) * 4, mod=(On(2, 6, H), On(L + N)), split=False, device=0, **changed):
        t = (3 * DIM // 8) if split else DIM // 2
        a = dict(txt=On(L, H), img=On(N, H), txt_cos=On(L, t), txt_sin=On(L, t), img_cos=On(N, t), img_sin=On(N, t), ws=On(1 << 20))
        a.update(changed)
        before = len(made)
        D.dit_block_forward_fp4(D.DitDims(H, HEADS, DIM, FFN, rope_split=split), D.Fp4BlockWeights(mats or _matrices(), *norms),
                                mod=D.Modulation(*mod), **a)
        assert len(made) == before + 1

    run.made = made
    return run


def test_what_fits_is_called(call):
    call()
    call(split=True)
    call(norms=(On(H), On(H), On(DIM), On(DIM)))
    call(txt=None, txt_cos=None, txt_sin=None, mod=(On(1, 6, H), None))
    call(img_cos=On(N + 4, DIM // 2))  # tables may hold more rows than are used


@pytest.mark.parametrize("bad", [
    dict(img=On(N, H - 4)), dict(txt=On(L, 2 * H)), dict(txt_cos=On(L - 1, DIM // 2)), dict(txt_sin=On(L, DIM // 4)),
    dict(img_cos=On(N, 3 * DIM // 8)), dict(img_sin=On(N - 1, DIM // 2)), dict(split=True, img_sin=On(N, DIM // 4)),
    dict(norms=(On(H - 1), None, None, None)), dict(norms=(None, On(DIM), None, None)), dict(norms=(None, None, On(DIM - 1), None)),
    dict(norms=(None, None, None, On(1))), dict(mod=(On(2, 5, H), None)), dict(mod=(On(2, 6, H), On(L + N - 1)))])
def test_too_small(call, bad):
    with pytest.raises(ValueError):
        call(**bad)
    assert not call.made


@pytest.mark.parametrize("name,shape", [("img", (N, H)), ("txt", (L, H)), ("txt_cos", (L, DIM // 2)), ("img_sin", (N, DIM // 2)),
                                        ("ws", (1 << 20,))])
def test_another_device(call, name, shape):
    with pytest.raises(ValueError):
        call(**{name: On(*shape, device=1)})
    assert not call.made


def test_weights_on_another_device(call):
    for bad in (dict(mats=_matrices(1)), dict(mats=_matrices()[:3] + _matrices(1)[3:]), dict(norms=(On(H, device=1), None, None, None)),
                dict(mod=(On(2, 6, H, device=1), None)), dict(mod=(On(2, 6, H), On(L + N, device=1))), dict(mats=_matrices()[:3])):
        with pytest.raises(ValueError):
            call(**bad)
    assert not call.made
