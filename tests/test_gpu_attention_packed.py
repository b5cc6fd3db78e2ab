"""Packed attention on the GPU against the oracle in 64 bits.

Gate. A score is d exact products summed in fp32: off by d 2^-23 sum |q k| scale, and the steps to its weight (scale,
cap, bias, maximum, exponential) by at most 2^-20 (1 + |x| + cap): together a relative error t of every weight. A weight
rounds to bf16 (2^-8), the sums over n keys are fp32 (n 2^-23): |o - ref| <= (2^-8 + 3 t + n 2^-22) sum w |v| / sum w,
plus half a step of the output (2^-8). lse: t + n 2^-23 + 2^-20 (1 + |lse|)."""

import numpy as np
import pytest
import torch

import diffusion_transformer_gb300 as D
import oracle as O
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu


def _starts(lens, first=0):
    return [first] + list(first + np.cumsum(lens))


def _bf16(g, *shape, gain=1.0):
    return torch.from_numpy((gain * g.standard_normal(shape)).astype(np.float32)).bfloat16()


def _np(t):
    return t.double().cpu().numpy()


def _check(o, lse, q, k, v, qs, ks, vis, scale, cap, slope):
    q, k, v = _np(q), _np(k), _np(v)
    ref, rlse, mag = O.attention_packed(q, k, v, qs, ks, vis, scale, cap, slope)
    d, heads = q.shape[2], q.shape[1]
    for s in range(len(qs) - 1):
        a, b = slice(qs[s], qs[s + 1]), slice(ks[s], ks[s + 1])
        nq, nk = qs[s + 1] - qs[s], ks[s + 1] - ks[s]
        if nq == 0:
            continue
        big = 0.0
        if nk:  # the largest score of the segment, by norms
            big = np.nan_to_num(np.abs(q[a])).sum(2).max() * np.nan_to_num(np.abs(k[b])).max() * scale
        far = (np.abs(slope).max() if slope is not None else 0.0) * max(nq, nk)
        t = d * 2.0 ** -23 * big + 2.0 ** -20 * (1 + (min(big, cap) if cap else big) + far + cap)
        gate = (2.0 ** -8 + 3 * t + nk * 2.0 ** -22) * mag[a]
        got = _np(o[a])
        off = np.abs(got - ref[a])
        assert (off <= gate + 2.0 ** -8 * (np.abs(ref[a]) + gate) + 1e-30).all(), (s, float(np.nanmax(off / (gate + 1e-30))))
        if lse is not None:
            gl, rl = _np(lse[:, a]), rlse[:, a]
            none = np.isneginf(rl)
            assert np.array_equal(np.isneginf(gl), none), s
            assert (np.abs(gl - rl)[~none] <= t + nk * 2.0 ** -23 + 2.0 ** -20 * (1 + np.abs(rl[~none]))).all(), s


def _visible(kind, qlens, klens, g):
    if kind == "all":
        return None
    out = []
    for nq, nk in zip(qlens, klens):
        i = np.arange(nq) + nk - nq
        if kind == "causal":
            out.append(i + 1)
        elif kind == "any":  # any count, none and past the end among them
            out.append(g.integers(-3, nk + 9, nq))
        elif kind == "none":
            out.append(np.zeros(nq, np.int64))
        else:  # a text in front that sees itself alone
            out.append(np.where(i < 17, min(17, nk), nk))
    return np.concatenate(out).astype(np.int32)


LENS = {
    "one": ([1], [1]),
    "few": ([5], [5]),
    "tile": ([128], [128]),
    "past": ([129], [257]),
    "pair": ([300], [385]),
    "ragged": ([200, 1, 0, 64, 77, 3], [513, 77, 5, 0, 77, 128]),
    "rows": ([1, 1, 1, 1, 1], [300, 1, 0, 129, 700]),
    "drafts": ([3, 7, 2], [900, 33, 640]),
}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("heads,kv", [(2, 2), (6, 2), (5, 1)])
@pytest.mark.parametrize("mask", ["all", "causal", "any"])
def test_lengths_masks_and_heads(d, lens, heads, kv, mask):
    qlens, klens = LENS[lens]
    g = np.random.default_rng(sum(qlens) + heads)
    qs, ks = _starts(qlens, 2), _starts(klens, 3)  # rows of no segment in front and behind
    q, k, v = _bf16(g, qs[-1] + 5, heads, d, gain=2.0), _bf16(g, ks[-1] + 4, kv, d), _bf16(g, ks[-1] + 4, kv, d)
    vis = _visible(mask, qlens, klens, g)
    if vis is not None:
        vis = np.concatenate([[9, 9], vis, [9] * 5]).astype(np.int32)
    nan = float("nan")
    k[:3], k[ks[-1]:], v[:3], v[ks[-1]:] = nan, nan, nan, nan
    for cap, slope in ((0.0, None), (20.0, None), (0.0, 2.0 ** -np.arange(1, heads + 1)), (5.0, 2.0 ** -np.arange(3, heads + 3))):
        for part in (False, True):
            o, lse = torch.full_like(q, 3.0).cuda(), torch.full((heads, q.shape[0]), 3.0, device="cuda")
            n = D.dit_attention_packed_workspace_bytes(q.shape[0], k.shape[0], len(qlens), heads, kv, d)
            if part and n == 0:
                continue
            D.dit_attention_packed(q.cuda(), k.cuda(), v.cuda(), o, dev(np.array(qs, np.int32)), dev(np.array(ks, np.int32)),
                                   visible=None if vis is None else dev(vis), cap=cap,
                                   slope=None if slope is None else dev(slope.astype(np.float32)), lse=lse,
                                   ws=torch.empty(n, dtype=torch.uint8, device="cuda") if part else None)
            D.dit_check()
            _check(o, lse, q, k, v, qs, ks, vis, d ** -0.5, cap, slope)
            for out in (o[:2], o[qs[-1]:], lse[:, :2], lse[:, qs[-1]:]):
                assert (out == 3).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("mask", ["none", "text", "causal"])
def test_long_segments(d, mask):
    g = np.random.default_rng(d)
    qlens = klens = [700, 1, 300]
    qs = ks = _starts(qlens)
    q, k, v = _bf16(g, 1001, 4, d, gain=3.0), _bf16(g, 1001, 2, d), _bf16(g, 1001, 2, d)
    vis = _visible(mask, qlens, klens, g)
    o, lse = torch.empty_like(q).cuda(), torch.empty(4, 1001, device="cuda")
    at = dev(np.array(qs, np.int32))
    D.dit_attention_packed(q.cuda(), k.cuda(), v.cuda(), o, at, at, visible=dev(vis), lse=lse)
    D.dit_check()
    _check(o, lse, q, k, v, qs, ks, vis, d ** -0.5, 0.0, None)


@pytest.mark.parametrize("heads,kv", [(1, 1), (24, 8), (40, 1), (128, 1), (96, 2)])
@pytest.mark.parametrize("rows", [1, 2, 9])
def test_few_rows_over_long_keys(heads, kv, rows):
    g = np.random.default_rng(heads + rows)
    d, keys = 128, 5000
    q, k, v = _bf16(g, rows, heads, d, gain=2.0), _bf16(g, keys, kv, d), _bf16(g, keys, kv, d)
    n = D.dit_attention_packed_workspace_bytes(rows, keys, 1, heads, kv, d)
    assert n > 0
    outs = []
    for ws in (torch.empty(n, dtype=torch.uint8, device="cuda"), None):
        o, lse = torch.empty_like(q).cuda(), torch.empty(heads, rows, device="cuda")
        D.dit_attention_packed(q.cuda(), k.cuda(), v.cuda(), o, lse=lse, ws=ws, scale=0.05)
        D.dit_check()
        _check(o, lse, q, k, v, [0, rows], [0, keys], None, 0.05, 0.0, None)
        outs.append(o)
    again = torch.empty_like(outs[0])
    D.dit_attention_packed(q.cuda(), k.cuda(), v.cuda(), again, scale=0.05, ws=torch.empty(n, dtype=torch.uint8, device="cuda"))
    assert torch.equal(again, outs[0])


def test_columns_of_one_product_and_head_major():
    g = np.random.default_rng(8)
    H, Hk, d, n = 6, 3, 64, 190
    qkv = _bf16(g, n, H + 2 * Hk, d)
    m = qkv.cuda()
    q, k, v = m[:, :H], m[:, H:H + Hk], m[:, H + Hk:]
    wide = torch.full((n, H * d + 16), 3.0, dtype=torch.bfloat16, device="cuda")
    o = wide[:, :H * d].view(n, H, d)
    D.dit_attention_packed(q, k, v, o)
    _check(o, None, q, k, v, [0, n], [0, n], None, d ** -0.5, 0.0, None)
    assert (wide[:, H * d:] == 3).all()
    heads = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v, o)]  # [heads, rows, d] in memory
    D.dit_attention_packed(*heads)
    assert torch.equal(heads[3], o)
    one = [t[:, :1] for t in (q, k, v)]  # one head: its stride does not matter
    out = torch.empty(n, 1, d, dtype=torch.bfloat16, device="cuda")
    D.dit_attention_packed(*one, out)
    assert torch.equal(out, o[:, :1])


@pytest.mark.parametrize("rows", [1, 260])
def test_what_is_masked_never_matters(rows):
    # NaN and infinities in keys and values that rows do not see: alone in their rows' results
    g = np.random.default_rng(rows)
    d, nk, H = 128, 600, 2
    q, k, v = _bf16(g, 2 * rows, H, d), _bf16(g, 2 * nk, H, d), _bf16(g, 2 * nk, H, d)
    vis = np.concatenate([np.full(rows, 333), np.minimum(np.arange(rows) + 280, nk)]).astype(np.int32)
    qs, ks = [0, rows, 2 * rows], [0, nk, 2 * nk]
    at = [dev(np.array(s, np.int32)) for s in (qs, ks)]
    n = D.dit_attention_packed_workspace_bytes(2 * rows, 2 * nk, 2, H, H, d)
    for ws in (None, torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")):
        clean, out = torch.empty_like(q).cuda(), torch.empty_like(q).cuda()
        lse = torch.empty(2, H, 2 * rows, device="cuda")
        D.dit_attention_packed(q.cuda(), k.cuda(), v.cuda(), clean, *at, visible=dev(vis), lse=lse[0], ws=ws)
        kb, vb = k.clone(), v.clone()
        kb[333:nk], vb[333:nk] = float("nan"), float("inf")      # behind all rows of the first segment
        vb[nk + 300:nk + 340:7], kb[nk + 301] = float("nan"), float("-inf")  # between the rows of the second
        D.dit_attention_packed(q.cuda(), kb.cuda(), vb.cuda(), out, *at, visible=dev(vis), lse=lse[1], ws=ws)
        D.dit_check()
        sure = vis <= 300
        sure[:rows] = True
        assert torch.equal(out[:rows], clean[:rows]) and torch.equal(lse[1, :, :rows], lse[0, :, :rows])
        keep = torch.from_numpy(sure)
        _check(out[keep.cuda()], None, q[keep], k, v, [0, rows, int(sure.sum())], ks, vis[sure], d ** -0.5, 0.0, None)
        sees = torch.from_numpy(vis > 301)
        sees[:rows] = False
        assert torch.isnan(out[sees.cuda()].float()).any(-1).all()


def test_far_scores_and_one_dominant_key():
    d, n = 64, 300
    q, k, v = torch.zeros(n, 1, d), torch.zeros(n, 1, d), torch.randn(n, 1, d, generator=torch.Generator().manual_seed(1))
    q[:, 0, 0] = torch.linspace(-3000, 3000, n)
    k[:, 0, 0] = torch.linspace(-30, 30, n)
    q, k, v = q.bfloat16(), k.bfloat16(), v.bfloat16()
    o, lse = torch.empty(n, 1, d, dtype=torch.bfloat16, device="cuda"), torch.empty(1, n, device="cuda")
    D.dit_attention_packed(q.cuda(), k.cuda(), v.cuda(), o, scale=1.0, lse=lse)
    # scores in steps of 600 at the ends: the first rows take the first key, the last rows the last
    assert torch.equal(o[0].cpu(), v[0]) and torch.equal(o[-1].cpu(), v[-1]) and torch.isfinite(lse).all()
    assert abs(lse[0, 0].item() - 90000) <= 90000 * 2.0 ** -7


def test_offsets_past_32_bits():
    g = np.random.default_rng(4)
    d, step = 64, 1_200_000_008
    mem = torch.empty(2 * step + 4096, dtype=torch.bfloat16, device="cuda")
    x = _bf16(g, 3, 2, d)
    view = lambda o: torch.as_strided(mem, (3, 2, d), (step, d, 1), o)  # noqa: E731
    k, v, q, o = view(0), view(512), view(1024), view(2048)
    for t, s in ((k, 0), (v, 1), (q, 2)):
        t.copy_(x.roll(s, 0))
    D.dit_attention_packed(q, k, v, o)
    _check(o, None, x.roll(2, 0), x, x.roll(1, 0), [0, 3], [0, 3], None, d ** -0.5, 0.0, None)


def test_no_keys_and_no_rows():
    q = torch.randn(5, 2, 64, device="cuda").bfloat16()
    k = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = torch.ones_like(q), torch.ones(2, 5, device="cuda")
    D.dit_attention_packed(q, k, k, o, lse=lse)
    assert (o == 0).all() and torch.isneginf(lse).all()
    D.dit_attention_packed(q[:0], q, q, o[:0])
    at = torch.zeros(1, dtype=torch.int32, device="cuda")
    D.dit_attention_packed(q, q, q, o.fill_(2), at, at)  # no segments
    assert (o == 2).all()
    D.dit_check()


def test_many_segments_find_their_tiles():
    g = np.random.default_rng(1)
    lens = list(g.integers(0, 4, 700))
    qs = _starts(lens)
    q, k, v = _bf16(g, qs[-1], 2, 64), _bf16(g, qs[-1], 1, 64), _bf16(g, qs[-1], 1, 64)
    o, lse = torch.empty_like(q).cuda(), torch.empty(2, qs[-1], device="cuda")
    at = dev(np.array(qs, np.int32))
    D.dit_attention_packed(q.cuda(), k.cuda(), v.cuda(), o, at, at, lse=lse)
    _check(o, lse, q, k, v, qs, qs, None, 0.125, 0.0, None)


def test_graph_serves_other_lengths_and_other_streams():
    g = np.random.default_rng(2)
    q, k, v = _bf16(g, 6, 4, 128).cuda(), _bf16(g, 4096, 2, 128).cuda(), _bf16(g, 4096, 2, 128).cuda()
    qs, ks = [0, 1, 2, 3, 4, 5, 6], [[0, 700, 1400, 2000, 3000, 3500, 4096], [0, 3, 3, 2500, 2600, 2601, 4000]]
    at, kt = dev(np.array(qs, np.int32)), dev(np.array(ks[0], np.int32))
    n = D.dit_attention_packed_workspace_bytes(6, 4096, 6, 4, 2, 128)
    o, o2, ws = torch.empty_like(q), torch.empty_like(q), torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    D.dit_attention_packed(q, k, v, o, at, kt, ws=ws)
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(first):
        D.dit_attention_packed(q, k, v, o, at, kt, ws=ws)
    with torch.cuda.graph(second):  # another graph over the same scratch, replayed after the first
        D.dit_attention_packed(q, k, v, o2, at, kt, cap=3.0, ws=ws)
    for lens in ks + ks[:1]:
        kt.copy_(torch.tensor(lens, dtype=torch.int32))
        first.replay()
        second.replay()
        torch.cuda.synchronize()
        _check(o, None, q, k, v, qs, lens, None, 128 ** -0.5, 0.0, None)
        _check(o2, None, q, k, v, qs, lens, None, 128 ** -0.5, 3.0, None)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o3 = torch.empty_like(q)
    s.wait_stream(torch.cuda.current_stream())
    D.dit_attention_packed(q, k, v, o3, at, kt, ws=ws, stream=s)
    s.synchronize()
    assert torch.equal(o3, o)


def test_binding_refusals():
    q = torch.randn(5, 4, 64, device="cuda").bfloat16()
    k, o = q[:, :2], torch.empty_like(q)
    at = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    D.dit_attention_packed(q, k, k, o, at, at)
    for args, kw in (((q.float(), k, k, o), {}), ((q.cpu(), k, k, o), {}), ((q, k, k[:4], o), {}), ((q, k, k, o[:4]), {}),
                     ((q[0], k, k, o), {}), ((q.transpose(1, 2), k, k, o), {}), ((q, q[:, :, :32], q[:, :, :32], o), {}),
                     ((q, k, k, o, at), {}), ((q, k, k, o, at, at[:1]), {}), ((q, k, k, o, at.long(), at.long()), {}),
                     ((q, k, k, o, at, at), dict(visible=at)), ((q, k, k, o), dict(slope=at)), ((q, k, k, o), dict(lse=at)),
                     ((q, k, k, o), dict(cap=-1.0)), ((q, k, k, o), dict(scale=0.0)), ((q, k, k, q), {}),
                     ((q[:, :3], k, k, o[:, :3]), {}), ((q, k, k, o), dict(ws=torch.empty(64)))):
        with pytest.raises((TypeError, ValueError, D.DitError)):
            D.dit_attention_packed(*args, **kw)
    D.dit_check()


@pytest.mark.parametrize("cap", [1.0, 38.0, 39.0, 50.0, 55.0, 56.0, 90.0, 1000.0])
@pytest.mark.parametrize("sign", [-1.0, 1.0])
def test_caps_reached_on_either_side(cap, sign):
    # every score near its cap, above or below: the weights stay in range whatever maximum they are taken against
    g = np.random.default_rng(int(cap))
    d, n, H = 64, 300, 2
    k = np.abs(g.standard_normal((n, H, d))) + 0.5
    q = torch.from_numpy((sign * 40.0 * (np.abs(g.standard_normal((n, H, d))) + 0.5)).astype(np.float32)).bfloat16()
    k, v = torch.from_numpy(k.astype(np.float32)).bfloat16(), _bf16(g, n, H, d)
    scale = 0.125 * cap / 50.0
    vis = np.minimum(np.arange(n) + 1, 200).astype(np.int32)
    for slope in (None, np.array([0.5, 2.0 ** -8])):
        o, lse = torch.empty_like(q).cuda(), torch.empty(H, n, device="cuda")
        D.dit_attention_packed(q.cuda(), k.cuda(), v.cuda(), o, visible=dev(vis), scale=scale, cap=cap, lse=lse,
                               slope=None if slope is None else dev(slope.astype(np.float32)))
        D.dit_check()
        _check(o, lse, q, k, v, [0, n], [0, n], vis, scale, cap, slope)


WORK = {  # many tiles, long and short ones side by side, one tile over many keys
    "long": ([900], [900], 48, 48, 64),
    "ragged": ([500, 1, 0, 640, 129, 300], [500, 40, 9, 700, 129, 1000], 48, 48, 64),
    "groups": ([400, 700, 90], [400, 700, 2000], 64, 32, 128),
    "one-unit": ([130], [60000], 1, 1, 64),
    "many": ([130] * 40, [130] * 40, 32, 32, 64),
}


@pytest.mark.parametrize("name", list(WORK))
@pytest.mark.parametrize("mask", ["all", "causal", "any"])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (20.0, True)])
def test_many_tiles(name, mask, cap, bias):
    qlens, klens, heads, kv, d = WORK[name]
    g = np.random.default_rng(len(name))
    qs, ks = _starts(qlens, 1), _starts(klens, 2)
    n = D.dit_attention_packed_workspace_bytes(qs[-1] + 3, ks[-1] + 3, len(qlens), heads, kv, d)
    q, k, v = _bf16(g, qs[-1] + 3, heads, d, gain=2.0), _bf16(g, ks[-1] + 3, kv, d), _bf16(g, ks[-1] + 3, kv, d)
    vis = _visible(mask, qlens, klens, g)
    if vis is not None:
        vis = np.concatenate([[9], vis, [9] * 3]).astype(np.int32)
    v[ks[-1]:], v[:2] = float("nan"), float("inf")
    slope = 2.0 ** -np.linspace(1, 9, heads) if bias else None
    outs = []
    for fill in (0, 255):
        o, lse = torch.full_like(q, 3.0).cuda(), torch.full((heads, q.shape[0]), 3.0, device="cuda")
        D.dit_attention_packed(q.cuda(), k.cuda(), v.cuda(), o, dev(np.array(qs, np.int32)), dev(np.array(ks, np.int32)),
                               visible=None if vis is None else dev(vis), cap=cap, lse=lse,
                               slope=None if slope is None else dev(slope.astype(np.float32)),
                               ws=torch.full((max(n, 16),), fill, dtype=torch.uint8, device="cuda"))
        D.dit_check()
        outs.append((o, lse))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    for out in (o[:1], o[qs[-1]:], lse[:, :1], lse[:, qs[-1]:]):
        assert (out == 3).all()
    few = [0, heads // 2, heads - 1] if heads > 3 else list(range(heads))  # the oracle's time
    keys = [h * kv // heads for h in few]
    _check(o[:, few], lse[few], q[:, few], k[:, keys], v[:, keys], qs, ks, vis, d ** -0.5, cap,
           None if slope is None else slope[few])


def test_many_tiles_what_is_masked_never_matters():
    g = np.random.default_rng(3)
    H, d, n = 48, 64, 900
    q, k, v = _bf16(g, n, H, d), _bf16(g, n, H, d), _bf16(g, n, H, d)
    vis = (np.arange(n) + 1).astype(np.int32)
    ws = torch.empty(max(16, D.dit_attention_packed_workspace_bytes(n, n, 1, H, H, d)), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q).cuda()
    vb, kb = v.clone(), k.clone()
    vb[500::97], kb[501::97] = float("nan"), float("inf")
    D.dit_attention_packed(q.cuda(), kb.cuda(), vb.cuda(), out, visible=dev(vis), ws=ws)
    D.dit_check()
    few = [0, 20, 47]
    _check(out[:500, few], None, q[:500, few], k[:, few], v[:, few], [0, 500], [0, n], vis[:500], d ** -0.5, 0.0, None)
    assert torch.isnan(out[500:].float()).any(-1).all()


@pytest.mark.parametrize("rows", [1, 300])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_far_keys_preferred(rows, cap):
    # negative slopes: the bias grows with the distance, far past what a cap bounds
    g = np.random.default_rng(rows)
    d, n, H = 64, 900, 4
    q, k, v = _bf16(g, rows, H, d), _bf16(g, n, 2, d), _bf16(g, n, 2, d)
    slope = np.array([-0.5, 0.25, -0.01, 0.0])
    o, lse = torch.empty_like(q).cuda(), torch.empty(H, rows, device="cuda")
    D.dit_attention_packed(q.cuda(), k.cuda(), v.cuda(), o, cap=cap, lse=lse, slope=dev(slope.astype(np.float32)))
    D.dit_check()
    _check(o, lse, q, k, v, [0, rows], [0, n], None, 0.125, cap, slope)


@pytest.mark.parametrize("rows,n", [(700, 300), (3000, 1100), (40, 9)])
@pytest.mark.parametrize("cap", [0.0, 20.0, 50.0])
def test_more_rows_than_keys_with_a_bias(rows, n, cap):
    # the first rows' places lie before the first key: even their nearest key is far, and the row still has its weights
    g = np.random.default_rng(rows + n)
    d, H = 64, 4
    q, k, v = _bf16(g, rows, H, d), _bf16(g, n, 4, d), _bf16(g, n, 4, d)
    slope = np.array([0.5, 2.0 ** -8, 2.0, 0.0])
    vis = g.integers(0, n + 1, rows).astype(np.int32)
    for visible in (None, vis):
        o, lse = torch.empty_like(q).cuda(), torch.empty(H, rows, device="cuda")
        D.dit_attention_packed(q.cuda(), k.cuda(), v.cuda(), o, cap=cap, lse=lse, slope=dev(slope.astype(np.float32)),
                               visible=None if visible is None else dev(visible))
        D.dit_check()
        _check(o, lse, q, k, v, [0, rows], [0, n], visible, 0.125, cap, slope)


LIB = D


class _Behind:
    """The library over caches that go on behind the last sequence, with NaN there: key segments count as long ones, so
    tall segments run in whole tiles however few keys they have."""

    dit_check = staticmethod(LIB.dit_check)

    @staticmethod
    def more(segments):
        return 1025 * segments

    def dit_attention_packed_workspace_bytes(self, q_rows, k_rows, segments, *rest):
        return LIB.dit_attention_packed_workspace_bytes(q_rows, k_rows + self.more(segments), segments, *rest)

    def dit_attention_packed(self, q, k, v, o, at=None, kt=None, **kw):
        if at is None:
            at, kt = (dev(np.array([0, t.shape[0]], np.int32)) for t in (q, k))
        rows = self.more(at.numel() - 1)
        k, v = (torch.cat([t, t.new_full((rows, *t.shape[1:]), float("nan"))]) for t in (k, v))
        LIB.dit_attention_packed(q, k, v, o, at, kt, **kw)


@pytest.fixture
def behind(monkeypatch):
    monkeypatch.setitem(globals(), "D", _Behind())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", ["past", "pair", "ragged"])
@pytest.mark.parametrize("heads,kv", [(2, 2), (6, 2), (5, 1)])
@pytest.mark.parametrize("mask", ["all", "causal", "any"])
def test_whole_tiles_lengths_masks_and_heads(behind, d, lens, heads, kv, mask):
    test_lengths_masks_and_heads(d, lens, heads, kv, mask)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("mask", ["none", "text", "causal"])
def test_whole_tiles_long_segments(behind, d, mask):
    test_long_segments(d, mask)


def test_whole_tiles_what_is_masked_never_matters(behind):
    test_what_is_masked_never_matters(260)
    test_many_tiles_what_is_masked_never_matters()


@pytest.mark.parametrize("cap", [1.0, 38.0, 39.0, 50.0, 55.0, 56.0, 90.0, 1000.0])
@pytest.mark.parametrize("sign", [-1.0, 1.0])
def test_whole_tiles_caps_reached_on_either_side(behind, cap, sign):
    test_caps_reached_on_either_side(cap, sign)


@pytest.mark.parametrize("name", list(WORK))
@pytest.mark.parametrize("mask", ["all", "causal", "any"])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (20.0, True)])
def test_whole_tiles_many(behind, name, mask, cap, bias):
    test_many_tiles(name, mask, cap, bias)


@pytest.mark.parametrize("cap", [0.0, 20.0, 50.0])
def test_whole_tiles_biases(behind, cap):
    test_far_keys_preferred(300, cap)
    test_more_rows_than_keys_with_a_bias(700, 300, cap)


def test_whole_tiles_far_scores(behind):
    test_far_scores_and_one_dominant_key()


def test_whole_tiles_of_columns_and_head_major():
    g = np.random.default_rng(9)
    H, Hk, d, n = 6, 3, 64, 190
    m = _bf16(g, n + 1025, H + 2 * Hk, d)
    m[n:] = float("nan")
    m = m.cuda()
    q, k, v, o = m[:n, :H], m[:, H:H + Hk], m[:, H + Hk:], torch.empty(n, H, d, dtype=torch.bfloat16, device="cuda")
    at = dev(np.array([0, n], np.int32))
    D.dit_attention_packed(q, k, v, o, at, at)
    _check(o, None, q, k[:n], v[:n], [0, n], [0, n], None, d ** -0.5, 0.0, None)
    heads = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v, o)]
    D.dit_attention_packed(*heads, at, at)
    assert torch.equal(heads[3], o)
    D.dit_check()
