"""Packed attention where a cap is far above the scores, on the GPU against the oracle in 64 bits.

Gate. A score is d exact products summed in fp32: off by d 2^-23 sum |q k| scale; its cap, bias and maximum and the
exponential are off by at most 2^-20 (1 + |x| + bias), |x| the score under its cap. The cap itself is in no term: a score far
below it is as good as without it. Weights round to bf16 (2^-8), sums over n keys are fp32 (n 2^-23)."""

import numpy as np
import pytest
import torch

import diffusion_transformer_gb300 as D
import oracle as O
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu


def _bf16(g, *shape, gain=1.0):
    return torch.from_numpy((gain * g.standard_normal(shape)).astype(np.float32)).bfloat16()


def _np(t):
    return t.double().cpu().numpy()


def _gate(q, k, nk, mag, scale, cap, slope):
    big = max((np.abs(q[:, h]) @ np.abs(k[:, h * k.shape[1] // q.shape[1]]).T).max() for h in range(q.shape[1])) * scale
    far = (np.abs(slope).max() if slope is not None else 0.0) * max(len(q), nk)
    t = q.shape[2] * 2.0 ** -23 * big + 2.0 ** -20 * (1 + (min(big, cap) if cap else big) + far)
    return t, (2.0 ** -8 + 3 * t + nk * 2.0 ** -22) * mag


def _check(o, lse, q, k, v, vis, scale, cap, slope):
    q, k, v, got = _np(q), _np(k), _np(v), _np(o)
    ref, rlse, mag = O.attention_packed(q, k, v, [0, len(q)], [0, len(k)], vis, scale, cap, slope)
    t, gate = _gate(q, k, len(k), mag, scale, cap, slope)
    off = np.abs(got - ref)
    assert (off <= gate + 2.0 ** -8 * (np.abs(ref) + gate)).all(), float(np.nanmax(off / (gate + 1e-300)))
    if lse is not None:
        gl, none = _np(lse), np.isneginf(rlse)
        assert np.array_equal(np.isneginf(gl), none)
        gl, rl = gl[~none], rlse[~none]
        assert (np.abs(gl - rl) <= t + len(k) * 2.0 ** -23 + 2.0 ** -20 * (1 + np.abs(rl))).all(), float(np.abs(gl - rl).max())


def _ws(q, k):
    n = D.dit_attention_packed_workspace_bytes(q.shape[0], k.shape[0], 1, q.shape[1], k.shape[1], q.shape[2])
    return torch.empty(max(16, n), dtype=torch.uint8, device="cuda")


ROWS = [3, 200]  # the few-rows kernel, and whole tiles (more rows than a tile's over more than 1024 keys)
KEYS = 1100


@pytest.mark.parametrize("cap", [60.0, 177.0, 178.0, 1e3, 1e4, 1e5, 1e6, 1e7, 1e12, 1e30, 2e38])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("d", [64, 128])
def test_scores_far_below_their_cap(cap, rows, d):
    g = np.random.default_rng(rows + d)
    q, k, v = _bf16(g, rows, 2, d, gain=2.0), _bf16(g, KEYS, 2, d), _bf16(g, KEYS, 2, d)
    vis = g.integers(0, KEYS + 1, rows).astype(np.int32)
    for slope in (None, np.array([0.25, 2.0 ** -6])):
        for ws in (None, _ws(q, k)):
            o, lse = torch.empty_like(q).cuda(), torch.empty(2, rows, device="cuda")
            D.dit_attention_packed(q.cuda(), k.cuda(), v.cuda(), o, visible=dev(vis), cap=cap, lse=lse, ws=ws,
                                   slope=None if slope is None else dev(slope.astype(np.float32)))
            D.dit_check()
            _check(o, lse, q, k, v, vis, d ** -0.5, cap, slope)


@pytest.mark.parametrize("cap", [60.0, 300.0, 1e4])
@pytest.mark.parametrize("rows", ROWS)
def test_scores_around_a_large_cap(cap, rows):
    # from far below the cap to three times it on either side, half of it among them
    g = np.random.default_rng(rows)
    d = 64
    q, k, v = _bf16(g, rows, 2, d), torch.zeros(KEYS, 2, d), _bf16(g, KEYS, 2, d)
    q[:] = 0
    q[:, :, 0] = 1
    k[:, :, 0] = torch.from_numpy(cap * np.concatenate([np.linspace(-3, 3, KEYS - 200), np.linspace(-0.01, 0.01, 200)])[:, None])
    k = k.bfloat16()
    o, lse = torch.empty_like(q).cuda(), torch.empty(2, rows, device="cuda")
    D.dit_attention_packed(q.cuda(), k.cuda(), v.cuda(), o, scale=1.0, cap=cap, lse=lse)
    D.dit_check()
    _check(o, lse, q, k, v, None, 1.0, cap, None)


@pytest.mark.parametrize("rows", ROWS)
def test_what_is_masked_never_matters_under_a_large_cap(rows):
    g = np.random.default_rng(7)
    d = 128
    q, k, v = _bf16(g, rows, 2, d, gain=2.0), _bf16(g, KEYS, 2, d), _bf16(g, KEYS, 2, d)
    vis = (np.arange(rows) + 300).astype(np.int32)
    kb, vb = k.clone(), v.clone()
    kb[302:], vb[301:] = float("nan"), float("inf")  # rows 0 and 1 see neither; their neighbours in the tile do
    o = torch.empty_like(q).cuda()
    D.dit_attention_packed(q.cuda(), kb.cuda(), vb.cuda(), o, visible=dev(vis), cap=1e6)
    D.dit_check()
    _check(o[:2], None, q[:2], k, v, vis[:2], d ** -0.5, 1e6, None)
    assert not torch.isfinite(o[2:].float()).any()


@pytest.mark.parametrize("power", [100, 40, -40])
@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("rows,keys", [(200, 1100), (300, 6000), (3, 700)])
def test_values_far_from_one_under_a_cap(power, sign, rows, keys):
    # every score near its cap, above or below: weights taken against something else than the row's maximum leave V its range
    g = np.random.default_rng(rows)
    d, H = 64, 2
    q = (sign * 40.0 * (np.abs(g.standard_normal((rows, H, d))) + 0.5)).astype(np.float32)
    k = (np.abs(g.standard_normal((keys, H, d))) + 0.5).astype(np.float32)
    q, k, v = torch.from_numpy(q).bfloat16(), torch.from_numpy(k).bfloat16(), _bf16(g, keys, H, d, gain=2.0 ** power)
    vis = g.integers(1, keys + 1, rows).astype(np.int32)
    for cap in (50.0, 55.0):
        for slope in (None, np.array([0.5, 2.0 ** -8])):
            for ws in (None, _ws(q, k)):
                o, lse = torch.empty_like(q).cuda(), torch.empty(H, rows, device="cuda")
                D.dit_attention_packed(q.cuda(), k.cuda(), v.cuda(), o, visible=dev(vis), cap=cap, lse=lse, ws=ws,
                                       slope=None if slope is None else dev(slope.astype(np.float32)))
                D.dit_check()
                _check(o, lse, q, k, v, vis, d ** -0.5, cap, slope)


def test_infinities_that_a_row_does_see_under_a_cap():
    g = np.random.default_rng(3)
    d, rows, H = 64, 200, 1
    q, k, v = _bf16(g, rows, H, d, gain=40.0), _bf16(g, KEYS, H, d), _bf16(g, KEYS, H, d)
    vis = np.where(np.arange(rows) % 2, 500, 400).astype(np.int32)
    v[450, 0, 3], v[20, 0, 40], k[470] = float("inf"), float("-inf"), 0.0
    o = torch.empty_like(q).cuda()
    D.dit_attention_packed(q.cuda(), k.cuda(), v.cuda(), o, visible=dev(vis), cap=50.0)
    D.dit_check()
    got = o.float().cpu().numpy()[:, 0]
    assert np.isposinf(got[1::2, 3]).all() and np.isneginf(got[:, 40]).all() and np.isfinite(got[::2, :40]).all()
    assert np.isfinite(np.delete(got, [3, 40], 1)).all()
    keep = [c for c in range(d) if c not in (3, 40)]
    clean = v.clone()
    clean[450, 0, 3], clean[20, 0, 40] = 0.0, 0.0
    ref, _, mag = O.attention_packed(_np(q), _np(k), _np(clean), [0, rows], [0, KEYS], vis, 0.125, 50.0, None)
    _, gate = _gate(_np(q), _np(k), KEYS, mag, 0.125, 50.0, None)
    off = np.abs(got - ref[:, 0])[:, keep]
    assert (off <= (gate + 2.0 ** -8 * (np.abs(ref) + gate))[:, 0][:, keep]).all()


@pytest.mark.parametrize("slope", [1e4, 1e7, 1e12])
@pytest.mark.parametrize("cap", [0.0, 20.0, 1000.0])
@pytest.mark.parametrize("rows", ROWS)
def test_steep_biases_leave_the_nearest_key(slope, cap, rows):
    # rows past what they see: their nearest key is a hundred places away and outweighs all others
    g = np.random.default_rng(5)
    d = 64
    q, k, v = _bf16(g, rows, 2, d), _bf16(g, KEYS, 2, d), _bf16(g, KEYS, 2, d)
    vis = (np.arange(rows) + KEYS - rows - 100 + g.integers(0, 90, rows)).astype(np.int32)
    o, lse = torch.empty_like(q).cuda(), torch.empty(2, rows, device="cuda")
    D.dit_attention_packed(q.cuda(), k.cuda(), v.cuda(), o, visible=dev(vis), cap=cap, lse=lse,
                           slope=torch.full((2,), slope, device="cuda"))
    D.dit_check()
    assert torch.equal(o.cpu(), v[torch.from_numpy(vis).long() - 1])
    far = (np.arange(rows) + KEYS - rows - vis + 1)[None] * slope
    assert (np.abs(_np(lse) + far) <= 100 + 2.0 ** -20 * far).all()


@pytest.mark.parametrize("cap", [0.0, 50.0, 1000.0])
@pytest.mark.parametrize("rows", ROWS)
def test_columns_not_finite_on_either_side_of_the_mask(rows, cap):
    # by column of V, key 200 seen by all rows and key 600 by none of the first half: what is seen decides alone
    g = np.random.default_rng(11)
    d, inf, nan = 64, float("inf"), float("nan")
    q, k, v = _bf16(g, rows, 1, d), _bf16(g, KEYS, 1, d), _bf16(g, KEYS, 1, d)
    half = rows // 2
    vis = np.where(np.arange(rows) < half, 500, 900).astype(np.int32)
    clean = v.clone()
    for c, (seen, hidden) in enumerate([(0.5, nan), (0.5, inf), (nan, nan), (inf, nan), (-inf, inf), (inf, 0.5), (nan, 0.5), (inf, inf)]):
        v[200, 0, c], v[600, 0, c] = seen, hidden
    v[201, 0, 8], v[200, 0, 8], v[600, 0, 8] = inf, -inf, inf  # both infinities seen: NaN
    o = torch.empty_like(q).cuda()
    for ws in (None, _ws(q, k)):
        D.dit_attention_packed(q.cuda(), k.cuda(), v.cuda(), o.fill_(9), visible=dev(vis), cap=cap, ws=ws)
        D.dit_check()
        got = o.float().cpu().numpy()[:half, 0]
        assert np.isfinite(got[:, :2]).all() and np.isnan(got[:, [2, 6, 8]]).all()
        assert np.isposinf(got[:, [3, 5, 7]]).all() and np.isneginf(got[:, 4]).all() and np.isfinite(got[:, 9:]).all()
        clean[200, 0, :2] = 0.5
        ref, _, mag = O.attention_packed(_np(q[:half]), _np(k), _np(clean), [0, half], [0, KEYS], vis[:half], 0.125, cap, None)
        _, gate = _gate(_np(q[:half]), _np(k), KEYS, mag, 0.125, cap, None)
        off = np.abs(got - ref[:, 0])
        for c in [0, 1] + list(range(9, d)):
            assert (off[:, c] <= (gate + 2.0 ** -8 * (np.abs(ref) + gate))[:, 0, c]).all(), c


def test_rows_that_are_not_finite_cost_no_more_than_others_by_much():
    # NaN scores, and infinities that rows do see, leave nothing to sum again
    g = torch.Generator().manual_seed(2)
    rn = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    n, H, d = 4096, 8, 64
    q, k, v = rn(n, H, d), rn(n, H, d), rn(n, H, d)
    vis, o = torch.arange(1, n + 1, dtype=torch.int32, device="cuda"), torch.empty(n, H, d, dtype=torch.bfloat16, device="cuda")

    def ms(cap):
        run = lambda: D.dit_attention_packed(q, k, v, o, visible=vis, cap=cap)  # noqa: E731
        run()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        run(), run()
        b.record()
        torch.cuda.synchronize()
        return a.elapsed_time(b) / 2

    v[5, :, 7] = float("inf")
    assert ms(0.0) < 20 and ms(50.0) < 20  # 60 to 100 ms with all rows summed again
    assert torch.isposinf(o[6:, :, 7]).all() and torch.isfinite(o[:, :, 8:].float()).all()
    q[:] = float("nan")
    assert ms(0.0) < 20 and ms(50.0) < 20
    assert torch.isnan(o.float()).all()
    D.dit_check()
