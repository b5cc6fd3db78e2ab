"""Sizes past 32 bits are refused by the binding: handed on, they would be cut to their low 32 bits and the call
would do the work of a smaller matrix. (Stand-ins for tensors and for the library: no GPU.)"""

import types

import pytest
import torch

import diffusion_transformer_gb300 as D

FAR = 2 ** 32 + 3


class Rows:
    """What the binding asks of a CUDA tensor."""

    def __init__(self, *shape, dtype=torch.bfloat16):
        self.shape, self.dtype = torch.Size(shape), dtype

    def stride(self):
        s, out = 1, []
        for n in reversed(self.shape):
            out.insert(0, s)
            s *= n
        return tuple(out)

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 256

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return 2


@pytest.fixture
def calls(monkeypatch):
    made = []
    D._torch()
    stub = types.SimpleNamespace(dit_linear_fp4=lambda *a: made.append(a) or 0, dit_rotary=lambda *a: made.append(a) or 0,
                                 dit_rotary_tables=lambda *a: made.append(a) or 0)
    monkeypatch.setattr(D, "lib", lambda: stub)
    monkeypatch.setattr(D, "_current", lambda stream: (0, 0))
    monkeypatch.setattr(D, "_positions", lambda *a: 256)
    monkeypatch.setattr(D, "_ptr", lambda *a: 256)
    return made


def test_linear_of_more_rows_than_32_bits(calls):
    w = types.SimpleNamespace(rows=8, cols=1, ref=None, device=0)
    D.dit_linear_fp4(Rows(3, 1), w, Rows(3, 8), Rows(256))
    assert len(calls) == 1
    with pytest.raises(ValueError):
        D.dit_linear_fp4(Rows(FAR, 1), w, Rows(FAR, 8), Rows(256))
    assert len(calls) == 1


@pytest.mark.parametrize("shape", [(FAR, 1, 2), (FAR, 1, 1, 2), (1, FAR, 1, 2), (1, 1, FAR, 2), (1, 1, 1, FAR)])
def test_rotary_of_more_than_32_bits(calls, shape):
    plan = types.SimpleNamespace(ref=None, axes=1, dim=2)
    D.dit_rotary(plan, Rows(1, 3, 1, 2), None, Rows(3))
    assert len(calls) == 1
    for q, k in ((Rows(*shape), None), (Rows(*shape), Rows(*shape)), (Rows(1, 1, 1, 2), Rows(1, 1, FAR, 2))):
        with pytest.raises(ValueError):
            D.dit_rotary(plan, q, k, Rows(FAR))
    assert len(calls) == 1


def test_tables_of_more_rows_than_32_bits(calls):
    plan = types.SimpleNamespace(ref=None, axes=1, dim=2)
    with pytest.raises(ValueError):
        D.dit_rotary_tables(plan, Rows(FAR), Rows(FAR, 1, dtype=torch.float32), Rows(FAR, 1, dtype=torch.float32))
    assert not calls


def test_sizes_of_matrices_and_plans():
    dims = D.DitDims(256, 4, 64, 128)
    for ask in (lambda n: D.dit_fp4_code_bytes(n, 32), lambda n: D.dit_fp4_code_bytes(3, n),
                lambda n: D.dit_fp4_scale_bytes(0, n, 32), lambda n: D.dit_fp4_scale_bytes(0, 3, n),
                lambda n: D.dit_linear_fp4_workspace_bytes(0, n, 4, 32), lambda n: D.dit_linear_fp4_workspace_bytes(0, 4, n, 32),
                lambda n: D.dit_linear_fp4_workspace_bytes(0, 4, 4, n), lambda n: D.dit_block_fp4_workspace_bytes(dims, 0, 0, n),
                lambda n: D.dit_block_fp4_workspace_bytes(dims, 0, n, 4)):
        assert ask(64) > 0
        for far in (FAR, 2 ** 31, -2 ** 32 + 64):
            with pytest.raises(ValueError):
                ask(far)
    few = torch.empty(D.dit_fp4_code_bytes(3, 32), dtype=torch.uint8)
    with pytest.raises(ValueError, match="32 bits"):
        D.Fp4Matrix(0, FAR, 32, few, torch.empty(512, dtype=torch.uint8), torch.empty(3))
    for bad in (dict(widths=[2 ** 32 + 4]), dict(widths=[16], scaling="yarn", factor=2.0, original=2 ** 32 + 64)):
        with pytest.raises(ValueError):
            D.RotaryPlan(**bad)
