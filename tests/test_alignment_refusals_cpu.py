"""Pointers that a kernel reads in whole words are refused off those words' boundaries, before any CUDA call."""

import ctypes

import pytest

import diffusion_transformer_gb300 as D

SHAPES = ((768, 256), (256, 256), (256, 256), (256, 128))


def _fp4_block(L=4, **at):
    """The status of a 4-bit block call whose pointers are 4096 but for those named."""
    p = dict.fromkeys("txt img txt_cos txt_sin img_cos img_sin mod map norm1 norm2 q_norm k_norm ws".split(), 4096)
    p.update(at)
    M = D.dit_fp4_matrix
    w = D.dit_block_wfp4((M * 4)(*[M(0, a, b, 4096, 4096, 4096) for a, b in SHAPES]), p["norm1"], p["norm2"], p["q_norm"],
                         p["k_norm"])
    dims, mod, r = D.dit_dims(256, 4, 64, 128, 1e-6, 1e-6, 0), D.dit_mod(p["mod"], p["map"], 1), ctypes.byref
    return D.lib().dit_block_forward_fp4(r(dims), r(w), p["txt"], L, p["img"], 5, p["txt_cos"], p["txt_sin"], p["img_cos"],
                                         p["img_sin"], r(mod), p["ws"], 1 << 30, None)


@pytest.mark.parametrize("name,offsets", [(n, (4, 8, 12)) for n in ("txt", "img", "txt_cos", "txt_sin", "img_cos", "img_sin",
                                                                     "mod", "norm1", "norm2")]
                         + [(n, (1, 2)) for n in ("map", "q_norm", "k_norm")])
def test_fp4_block_pointers(name, offsets):
    for off in offsets:
        assert _fp4_block(**{name: 4096 + off}) == D.DIT_EINVAL
    if name in ("txt_cos", "txt_sin"):  # without text rows its tables are not looked at
        import torch
        if not torch.cuda.is_available():  # past the checks there is only the missing device here
            assert _fp4_block(L=0, **{name: 4097}) == D.DIT_ECUDA


@pytest.mark.parametrize("name", ["txt_cos", "txt_sin", "img_cos", "img_sin"])
def test_bf16_block_tables(name):
    p = dict.fromkeys(("txt_cos", "txt_sin", "img_cos", "img_sin"), 4096)
    p[name] += 4
    dims, mod, r = D.dit_dims(256, 4, 64, 128, 1e-6, 1e-6, 0), D.dit_mod(4096, None, 1), ctypes.byref
    w = D.dit_block_w(4096, 4096, 4096, 4096, None, None, None, None)
    assert D.lib().dit_block_forward(r(dims), r(w), 4096, 4, 4096, 5, p["txt_cos"], p["txt_sin"], p["img_cos"], p["img_sin"],
                                     r(mod), 4096, 1 << 30, None) == D.DIT_EINVAL
    assert D.lib().dit_block_forward_noalloc(r(dims), r(w), 4096, 4, 4096, 5, p["txt_cos"], p["txt_sin"], p["img_cos"],
                                             p["img_sin"], r(mod), None) == D.DIT_EINVAL


def test_rotary_positions_and_tables():
    p, r, at = D.RotaryPlan([64], layout="halves"), ctypes.byref, ctypes.c_void_p
    q = D.dit_rotary_rows(4096, 4096, 4, 0, 256, 64, 0, 256, 64)
    for off in (1, 2, 3):
        assert D.lib().dit_rotary(r(p.c), r(q), None, 0, 1, 3, 64, at(4096 + off), 0, None) == D.DIT_EINVAL
        for bad in range(3):
            pos, cos, sin = (at(4096 + (off if i == bad else 0)) for i in range(3))
            assert D.lib().dit_rotary_tables(r(p.c), pos, 3, cos, sin, None) == D.DIT_EINVAL
