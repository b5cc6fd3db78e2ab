"""CPU pins of the 4-bit oracle: closed forms of both formats, ties, extremes and the stored layout."""

import numpy as np
import pytest

import oracle as O

NV, MX = 0, 1


def test_e4m3_values_are_the_published_ones():
    v = O.e4m3_values()
    assert len(v) == 127 and v[0] == 0 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[-1] == 448
    assert np.all(np.diff(v) > 0)


@pytest.mark.parametrize("fmt", [NV, MX])
def test_values_on_the_grid_come_back(fmt):
    # rows that hold only code values times a power of two (NV: times the largest block scale 448 too, so
    # that the row scale A / 2688 is that power of two exactly), the largest code in every block
    g = np.random.default_rng(1)
    grid = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
    n = 16 if fmt == NV else 32
    x = (grid[g.integers(0, 8, (6, 4 * n))] * g.choice([-1, 1], (6, 4 * n))).astype(np.float32)
    x[:, ::n] = 6
    x *= np.float32(448 * 2.0 ** -3 if fmt == NV else 2.0 ** -3)
    c, s, row = O.fp4_quantize(x, fmt)
    assert np.array_equal(O.fp4_values(c, s, row, fmt, 4 * n), x)


def test_ties_go_to_the_even_code():
    x = np.zeros((1, 32), np.float32)
    x[0, :8] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    c, s, _ = O.fp4_quantize(x, MX)
    assert s[0, 0] == 127 and list(c[0, :8]) == [7, 0, 2, 2, 4, 4, 6, 6]
    c, _, _ = O.fp4_quantize(-x, MX)
    assert list(c[0, :8]) == [15, 8, 10, 10, 12, 12, 14, 14]


def test_mx_scale_is_the_power_two_below_the_largest_and_saturates():
    for top in (1.0, 4.0, 7.99, 2.0 ** -126, 2.0 ** -130, 2.0 ** 127):
        x = np.zeros((1, 32), np.float32)
        x[0, 3] = top
        c, s, _ = O.fp4_quantize(x, MX)
        e = max(int(np.floor(np.log2(np.float64(top)))) - 2, -127)
        assert s[0, 0] == e + 127
        assert c[0, 3] == (7 if top == 7.99 else {1.0: 6, 4.0: 6, 2.0 ** -126: 4, 2.0 ** -130: 0, 2.0 ** 127: 6}[top])


def test_zero_tiny_and_non_finite_rows():
    x = np.ones((5, 40), np.float32)
    x[0] = 0
    x[1] = 2.0 ** -110
    x[2, 7] = np.inf
    x[3, 33] = np.nan
    c, s, row = O.fp4_quantize(x, NV)
    assert row[0] == 0 and row[1] == 0 and np.isnan(row[2]) and np.isnan(row[3]) and row[4] == np.float32(1) / np.float32(2688)
    assert not c[:4].any() and not s[:4].any()
    c, s, _ = O.fp4_quantize(x, MX)
    assert list(s[2]) == [255, 125] and list(s[3]) == [125, 255] and list(s[0]) == [0, 0]
    v = O.fp4_values(c, s, None, MX, 40)
    assert np.isnan(v[2, :32]).all() and np.array_equal(v[2, 32:], x[2, 32:])


@pytest.mark.parametrize("fmt", [NV, MX])
def test_error_is_bounded(fmt):
    # half a step of the code (at most 1 of a block scale that maps the largest magnitude to at most 8, or,
    # NV, whose e4m3 scale is off by at most 2^-4 of itself)
    g = np.random.default_rng(2)
    x = (g.standard_normal((9, 300)) * np.exp(g.standard_normal((9, 1)))).astype(np.float32)
    c, s, row = O.fp4_quantize(x, fmt)
    v = O.fp4_values(c, s, row, fmt, 300)
    n = 16 if fmt == NV else 32
    for r in range(9):
        for b in range(0, 300, n):
            top = np.abs(x[r, b:b + n]).max()
            assert np.abs(v[r, b:b + n] - x[r, b:b + n]).max() <= (1 / 6 + 1 / 16 if fmt == NV else 0.25 + 1e-6) * top


def test_layout_of_a_scale_byte():
    s = np.arange(200 * 9, dtype=np.int64).reshape(200, 9).astype(np.uint8)
    codes = np.zeros((200, 288), np.uint8)
    codes[:, 0], codes[:, 1] = 3, 12
    packed, tiles = O.fp4_pack(codes, s, MX)
    assert packed.shape == (200, 144) and packed[0, 0] == 0xC3 and len(tiles) == 2 * 3 * 512
    for r, b in ((0, 0), (31, 3), (32, 4), (127, 8), (128, 0), (199, 8)):
        assert tiles[((r // 128) * 3 + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4] == s[r, b]


@pytest.mark.parametrize("fmt", [NV, MX])
def test_block_with_exact_operands_is_the_plain_block(fmt, monkeypatch):
    # with a quantiser that loses nothing the 4-bit block is the block of the same weights
    import dit_inputs as DI
    import oracle.fp4 as F
    inp = DI.block_inputs("tiny")
    sh = inp.shape
    monkeypatch.setattr(F, "fp4_quantize", lambda x, f: (x, None, None))
    monkeypatch.setattr(F, "fp4_values", lambda x, s, r, f, K: x)
    W = [O.bf16_to_f64(w) for w in (inp.wqkv, inp.wout, inp.wup, inp.wdown)]
    x = np.concatenate([inp.txt, inp.img])
    cos, sin = O.rope_tables(O.positions(sh.L, sh.grid_h, sh.grid_w), sh.head_dim)
    got = F.block_forward_fp4_rows(x, W, fmt, inp.mod, inp.mod_map, cos, sin, sh.heads, sh.head_dim, eps=sh.eps,
                                   qk_eps=sh.qk_eps)
    ref = np.concatenate(O.block_forward(inp))
    # only the activations' rounding to bf16 (2^-8 each) is between them
    assert np.abs(got - ref).max() <= 4 * 2.0 ** -8 * np.sqrt(np.mean(ref ** 2))
