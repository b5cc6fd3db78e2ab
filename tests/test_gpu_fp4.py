"""Microscaled 4-bit matrices on the GPU against the oracle (oracle/fp4.py): codes, scales and row scales
bit for bit, the values bit for bit, and products against 64 bits.

Product gate. The values are exact in fp32 and every product of two code-times-scale values is exact;
what is rounded is the fp32 accumulation. A tensor-core step sums 64 columns and the accumulator with
the terms aligned to the largest: allow one unit (2^-23) of the magnitude of everything summed so far
per step, in either direction, so |error| <= (K / 64 + 2) 2^-23 S with S = sum |a||b| (one extra step for
split sums joined at the end, one for the two row-scale products' half units). A store as bf16 adds half
a step, 2^-8 of the value. A fp32 FMA loop stays within the same bound only for short K; the largest here
through such a loop would err randomly, far below K 2^-24 S."""

import numpy as np
import pytest
import torch

import diffusion_transformer_gb300 as D
import oracle as O
from tests.gpu_util import bf16_bits, dev, workspace

pytestmark = pytest.mark.gpu

NV, MX = D.DIT_FP4_NV, D.DIT_FP4_MX
FMT = pytest.mark.parametrize("fmt", [NV, MX], ids=["nv", "mx"])


def _rows(g, R, K, bf16=True):
    """Activations with rows of unlike size and a few wide columns, as float32 (bf16 values if asked)."""
    x = g.standard_normal((R, K)) * np.exp(g.standard_normal((R, 1))) * np.where(g.random(K) < 0.02, 20, 1)
    return _as_bf16(x) if bf16 else x.astype(np.float32)


def _as_bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).bfloat16().float().numpy()


def _on_gpu(x, dtype, pad=0, shift=0):
    """x on the GPU with `pad` values between rows and its first value `shift` values into its memory."""
    R, K = x.shape
    mem = torch.full((R * (K + pad) + shift + 64,), 77.0, dtype=dtype, device="cuda")
    v = mem[shift:shift + R * (K + pad)].view(R, K + pad)[:, :K]
    v.copy_(torch.from_numpy(x))
    return v


def _stored(codes, scale, fmt, R, K):
    return O.fp4_pack(codes, scale, fmt)


def _check_quantised(m, x, fmt):
    codes, scale, row = O.fp4_quantize(x, fmt)
    packed, tiles = O.fp4_pack(codes, scale, fmt)
    R = x.shape[0]
    assert np.array_equal(m.codes.cpu().numpy().reshape(R, -1), packed)
    got = m.scales.cpu().numpy().reshape(-1, tiles.size // 512 // max(1, -(-R // 128)), 32, 4, 4)
    want = tiles.reshape(got.shape)
    r = np.arange(R)
    at = (r // 128, slice(None), r % 32, (r % 128) // 32)
    assert np.array_equal(got[at], want[at])
    if fmt == NV:
        assert np.array_equal(m.row_scale.cpu().numpy(), row, equal_nan=True)
    return codes, scale, row


@FMT
@pytest.mark.parametrize("R,K,dtype,pad,shift", [
    (1, 1, torch.bfloat16, 0, 0), (1, 16, torch.float32, 0, 0), (3, 31, torch.bfloat16, 0, 0),
    (5, 64, torch.bfloat16, 0, 0), (130, 100, torch.float32, 28, 0), (33, 1000, torch.bfloat16, 3, 5),
    (7, 1003, torch.float32, 0, 1), (2, 4096, torch.bfloat16, 0, 0), (9, 5000, torch.bfloat16, 8, 8),
    (300, 48, torch.float32, 0, 0), (1001, 17, torch.float32, 0, 0), (613, 128, torch.bfloat16, 0, 0),
    (2045, 192, torch.bfloat16, 8, 0), (4, 12288, torch.bfloat16, 0, 0), (3, 20011, torch.float32, 0, 0)])
def test_quantize_is_bit_exact(fmt, R, K, dtype, pad, shift):
    g = np.random.default_rng(R * 7919 + K)
    x = _rows(g, R, K, dtype == torch.bfloat16)
    if R > 2:
        x[1] = 0
        x[2] *= _as_bf16(np.full(1, 1e-30))[0]
        x = _as_bf16(x) if dtype == torch.bfloat16 else x
    xd = _on_gpu(x, dtype, pad, shift)
    m = D.Fp4Matrix.empty(fmt, R, K)
    m.codes.fill_(255)
    m.scales.fill_(255)
    D.dit_fp4_quantize(xd, m)
    codes, scale, row = _check_quantised(m, x, fmt)
    want = O.fp4_values(codes, scale, row, fmt, K)
    for odt in (torch.float32, torch.bfloat16):
        out = _on_gpu(np.zeros((R, K), np.float32), odt, pad, shift)
        D.dit_fp4_dequantize(m, out)
        w = torch.from_numpy(want).to(odt).float().numpy()
        assert np.array_equal(out.float().cpu().numpy(), w)
        if pad:  # what lies between the rows stays
            whole = torch.as_strided(out, (R, K + pad), (K + pad, 1))
            assert (whole[:-1, K:] == 77).all()
    D.dit_check()


@FMT
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("R,K", [(3, 15), (5, 65), (5003, 65), (5003, 229), (700, 533), (640, 4009), (4, 9001)])
def test_rows_at_every_alignment(fmt, dtype, R, K):
    """Rows that start at every offset from 16 bytes, and what lies around them left as it was."""
    per = 16 // torch.empty(0, dtype=dtype).element_size()
    x = _rows(np.random.default_rng(R + K), R, K)
    m, back = D.Fp4Matrix.empty(fmt, R, K), None
    for shift in range(per):
        for pad in (0, 1) if R < 10 else (1,):
            xd = _on_gpu(x, dtype, pad, shift)
            m.codes.fill_(255)
            m.scales.fill_(255)
            D.dit_fp4_quantize(xd, m)
            if back is None:
                codes, scale, row = _check_quantised(m, x, fmt)
                want = torch.from_numpy(O.fp4_values(codes, scale, row, fmt, K)).to(dtype).cuda()
                back = m.codes.clone(), m.scales.clone()
            else:
                assert torch.equal(m.codes, back[0])
                r = torch.arange(R, device="cuda")
                got, ref = (t.view(-(-R // 128), -1, 32, 4, 4)[r // 128, :, r % 32, r % 128 // 32]
                            for t in (m.scales, back[1]))
                assert torch.equal(got, ref)
            mem = torch.full((shift + R * (K + pad) + 64,), 77.0, dtype=dtype, device="cuda")
            D.dit_fp4_dequantize(m, mem[shift:shift + R * (K + pad)].view(R, K + pad)[:, :K])
            body = mem[shift:shift + R * (K + pad)].view(R, K + pad)
            assert torch.equal(body[:, :K], want)
            assert (body[:, K:] == 77).all() and (mem[:shift] == 77).all() and (mem[shift + R * (K + pad):] == 77).all()
    D.dit_check()


@FMT
def test_quantize_extremes(fmt):
    K = 96
    x = np.ones((14, K), np.float32)
    x[0, 5] = np.inf
    x[1, 40] = -np.inf
    x[2, 95] = np.nan
    x[3] = 2.0 ** -99
    x[4] = 2.0 ** -100
    x[5] = np.nextafter(np.float32(2.0 ** -100), np.float32(0))
    x[6] = 2.0 ** -140
    x[7] = 3.3e38
    x[8, ::2] = -3.4e38
    x[9] = -0.0
    x[10, :] = np.float32(2.0 ** -126)
    x[11, :16] = 1e-30
    x[12] = np.linspace(-6, 6, K)
    x[13] = np.repeat([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], 12) * np.float32(1.5)
    m = D.Fp4Matrix.empty(fmt, *x.shape)
    D.dit_fp4_quantize(dev(x), m)
    codes, scale, row = _check_quantised(m, x, fmt)
    out = torch.empty(x.shape, device="cuda")
    D.dit_fp4_dequantize(m, out)
    assert np.array_equal(out.cpu().numpy(), O.fp4_values(codes, scale, row, fmt, K), equal_nan=True)


def _product_gate(a, b, K):
    S = np.abs(a) @ np.abs(b).T
    return (K / 64 + 2) * 2.0 ** -23 * S


def _quantised(x, fmt):
    codes, scale, row = O.fp4_quantize(x, fmt)
    packed, tiles = O.fp4_pack(codes, scale, fmt)
    m = D.Fp4Matrix(fmt, *x.shape, dev(packed), dev(tiles), None if row is None else dev(row))
    return m, O.fp4_values(codes, scale, row, fmt, x.shape[1]).astype(np.float64)


def _check_product(out, a, b, K, what=""):
    ref = a @ b.T
    got = out.float().cpu().numpy().astype(np.float64)
    gate = _product_gate(a, b, K) + (2.0 ** -8 * np.abs(ref) if out.dtype == torch.bfloat16 else 0) + 1e-37
    bad = np.abs(got - ref) > gate
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4], float((np.abs(got - ref) / gate).max()))


SIZES = [(1, 16, 16), (1, 1, 1), (1, 1000, 256), (2, 130, 100), (8, 128, 4096), (16, 77, 333), (17, 256, 1000),
         (64, 1000, 512), (65, 384, 64), (127, 129, 31), (128, 128, 128), (129, 257, 257), (200, 1024, 1056),
         (256, 256, 4096), (333, 777, 1000), (513, 640, 2048), (1088, 512, 3104), (40, 4096, 8000), (1, 9000, 2000),
         (1100, 1500, 777), (1537, 1025, 2000), (2304, 768, 96), (300, 5200, 520)]
# one or more for every kernel and tile: pairs with 128, 192 and 256 rows (several rounds, so that accumulators
# and their overlap are reused), either operand first; clusters of two, four and eight
SIZES += [(4911, 784, 96), (1044, 3856, 2100), (1030, 7712, 96), (1037, 8720, 520), (1030, 8672, 96), (1155, 8194, 96),
          (250, 3000, 5000), (60, 3000, 5000), (100, 300, 5003), (40, 777, 9001)]


@FMT
@pytest.mark.parametrize("M,N,K", SIZES)
def test_matmul(fmt, M, N, K):
    g = np.random.default_rng(M + 31 * N + 1009 * K)
    a, av = _quantised(_rows(g, M, K), fmt)
    b, bv = _quantised(_rows(g, N, K) * np.float32(0.02), fmt)
    for dt, pad, shift in ((torch.float32, 0, 0), (torch.bfloat16, 0, 0), (torch.bfloat16, 3, 1)):
        out = _on_gpu(np.full((M, N), 9.0, np.float32), dt, pad, shift)
        D.dit_fp4_matmul(a, b, out)
        D.dit_check()
        _check_product(out, av, bv, K, (dt, pad))
        if pad:
            assert (torch.as_strided(out, (M, N + pad), (N + pad, 1))[:-1, N:] == 77).all()


@FMT
@pytest.mark.parametrize("M,N,K,dtype", [(1, 300, 1000, torch.bfloat16), (70, 130, 96, torch.float32),
                                         (300, 512, 768, torch.bfloat16)])
def test_linear_equals_quantise_and_product(fmt, M, N, K, dtype):
    g = np.random.default_rng(M * N)
    x = _rows(g, M, K, dtype == torch.bfloat16)
    w, wv = _quantised(_rows(g, N, K) * np.float32(0.02), fmt)
    xd = _on_gpu(x, dtype, 5, 0)
    out, two = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    D.dit_linear_fp4(xd, w, out, workspace(D.dit_linear_fp4_workspace_bytes(fmt, M, N, K)))
    a = D.Fp4Matrix.empty(fmt, M, K)
    D.dit_fp4_quantize(xd, a)
    D.dit_fp4_matmul(a, w, two)
    D.dit_check()
    assert torch.equal(out, two)
    codes, scale, row = O.fp4_quantize(x, fmt)
    _check_product(out, O.fp4_values(codes, scale, row, fmt, K).astype(np.float64), wv, K)
    assert np.array_equal(xd.float().cpu().numpy(), x)


@FMT
def test_non_finite_rows_stay_in_their_row(fmt):
    g = np.random.default_rng(5)
    M, N, K = 140, 150, 320
    x, w = _rows(g, M, K, False), _rows(g, N, K, False)
    x[3, 17], x[130, 300], x[60] = np.inf, np.nan, 0
    w[149, 5] = np.nan
    w[10] = 0
    a, b = D.Fp4Matrix.empty(fmt, M, K), D.Fp4Matrix.empty(fmt, N, K)
    D.dit_fp4_quantize(dev(x), a)
    D.dit_fp4_quantize(dev(w), b)
    out = torch.empty(M, N, device="cuda")
    D.dit_fp4_matmul(a, b, out)
    D.dit_check()
    o = out.cpu().numpy()
    nan = np.zeros((M, N), bool)
    nan[[3, 130]] = True
    nan[:, 149] = True
    assert np.array_equal(np.isnan(o), nan)
    assert (o[60, :149] == 0).all() and (o[np.delete(np.arange(M), [3, 130]), 10] == 0).all()


@FMT
@pytest.mark.parametrize("M,N,K", [(1, 97, 40), (130, 300, 328), (700, 1500, 1000)])
def test_what_lies_past_the_rows_never_matters(fmt, M, N, K):
    """Scale bytes of rows past the last, and the workspace, may hold anything (255 is NaN in both formats)."""
    g = np.random.default_rng(M + N)
    x, w = dev(_rows(g, M, K, False)), dev(_rows(g, N, K, False))
    outs = []
    for fill in (0, 255):
        b = D.Fp4Matrix.empty(fmt, N, K)
        b.codes.fill_(fill)
        b.scales.fill_(fill)
        D.dit_fp4_quantize(w, b)
        ws = workspace(D.dit_linear_fp4_workspace_bytes(fmt, M, N, K))
        ws.view(torch.uint8).fill_(fill)
        outs.append(torch.full((M, N), 77.0, device="cuda"))
        D.dit_linear_fp4(x, b, outs[-1], ws)
    D.dit_check()
    assert torch.isfinite(outs[0]).all() and torch.equal(outs[0], outs[1])


def test_empty_and_streams_and_graph():
    g = np.random.default_rng(6)
    w, wv = _quantised(_rows(g, 96, 256), NV)
    ws = workspace(D.dit_linear_fp4_workspace_bytes(NV, 50, 96, 256))
    D.dit_linear_fp4(torch.empty(0, 256, device="cuda"), w, torch.empty(0, 96, device="cuda"), ws)
    xs = [_rows(g, 50, 256) for _ in range(2)]
    x, out = dev(xs[0]), torch.empty(50, 96, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        D.dit_linear_fp4(x, w, out, ws)
    side.synchronize()
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        D.dit_linear_fp4(x, w, out, ws)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    x.copy_(dev(xs[1]))
    graph.replay()
    torch.cuda.synchronize()
    codes, scale, row = O.fp4_quantize(xs[1], NV)
    _check_product(out, O.fp4_values(codes, scale, row, NV, 256).astype(np.float64), wv, 256)


def test_offsets_past_32_bits():
    g = np.random.default_rng(7)
    ld, R, K, N = 1_100_000_016, 3, 96, 64
    x = _rows(g, R, K)
    mem = torch.empty(2 * ld + 4096, dtype=torch.bfloat16, device="cuda")
    xd = torch.as_strided(mem, (R, K), (ld, 1))
    xd.copy_(torch.from_numpy(x))
    m = D.Fp4Matrix.empty(NV, R, K)
    D.dit_fp4_quantize(xd, m)
    codes, scale, row = _check_quantised(m, x, NV)
    back = torch.as_strided(mem, (R, K), (ld, 1), 2048)
    D.dit_fp4_dequantize(m, back)
    v = O.fp4_values(codes, scale, row, NV, K)
    assert np.array_equal(back.float().cpu().numpy(), torch.from_numpy(v).bfloat16().float().numpy())
    w, wv = _quantised(_rows(g, N, K), NV)
    out = torch.as_strided(mem, (R, N), (ld, 1), 1024)
    D.dit_fp4_matmul(m, w, out)
    _check_product(out, v.astype(np.float64), wv, K)
    # many rows, so that the pair kernel stores them: 1300 rows of 2^21 values
    a, av = _quantised(_rows(g, 1300, K), MX)
    b, bv = _quantised(_rows(g, 1100, K), MX)
    out = torch.as_strided(mem, (1300, 1100), (1 << 20, 1))
    D.dit_fp4_matmul(a, b, out)
    D.dit_check()
    _check_product(out, av, bv, K)


def test_two_streams_at_once():
    # two streams with products of both kernels, each with its own workspace, give what one alone gives
    g = np.random.default_rng(11)
    jobs = []
    for M, N, K in ((1300, 1536, 512), (20, 512, 4096), (900, 2048, 768), (64, 3000, 2000)):
        w, _ = _quantised(_rows(g, N, K), NV)
        x = dev(_rows(g, M, K)).bfloat16()
        jobs.append((x, w, workspace(D.dit_linear_fp4_workspace_bytes(NV, M, N, K)), torch.empty(M, N, device="cuda")))
    want = []
    for x, w, ws, out in jobs:
        D.dit_linear_fp4(x, w, out, ws)
        want.append(out.clone())
        out.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for i, (x, w, ws, out) in enumerate(jobs):
            D.dit_linear_fp4(x, w, out, ws, stream=streams[i % 2])
    torch.cuda.synchronize()
    D.dit_check()
    for (x, w, ws, out), ref in zip(jobs, want):
        assert torch.equal(out, ref)


def test_quantise_then_use_at_once():
    # a weight quantised by the call just before the linear is complete when the linear reads it
    g = np.random.default_rng(12)
    M, N, K = 48, 4096, 2048
    x, w = dev(_rows(g, M, K)).bfloat16(), dev(_rows(g, N, K)).bfloat16()
    m, ws = D.Fp4Matrix.empty(NV, N, K), workspace(D.dit_linear_fp4_workspace_bytes(NV, M, N, K))
    ref, out = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    D.dit_fp4_quantize(w, m)
    torch.cuda.synchronize()
    D.dit_linear_fp4(x, m, ref, ws)
    torch.cuda.synchronize()
    for _ in range(10):
        m.codes.fill_(0x77)
        m.row_scale.fill_(float("nan"))
        D.dit_fp4_quantize(w, m)
        D.dit_linear_fp4(x, m, out, ws)
        torch.cuda.synchronize()
        assert torch.equal(out, ref)


def test_binding_refusals():
    w = D.Fp4Matrix.empty(NV, 8, 64)
    x, out, ws = torch.zeros(4, 64, device="cuda"), torch.zeros(4, 8, device="cuda"), workspace(1 << 16)
    for bad in (x.half(), x.cpu(), x.t().contiguous().t(), x[:, :63], x[0]):
        with pytest.raises((TypeError, ValueError)):
            D.dit_linear_fp4(bad if bad.dim() == 2 else bad, w, out, ws)
    with pytest.raises(ValueError):
        D.dit_linear_fp4(x, w, out[:, :7], ws)
    with pytest.raises(D.DitError):
        D.dit_linear_fp4(x, w, out, ws[:64])
    with pytest.raises(ValueError):
        D.Fp4Matrix(NV, 9, 64, w.codes, w.scales, w.row_scale)
    with pytest.raises(D.DitError):
        D.dit_fp4_matmul(D.Fp4Matrix.empty(MX, 8, 64), w, torch.zeros(8, 8, device="cuda"))


@FMT
def test_columns_past_2_to_24_blocks(fmt):
    # one row so long that its scale bytes reach past 2 GB: a short row's values at its two ends and in front of that
    # border, zeros between; codes and scales are the short row's, the rest zero, and the product is the short rows'
    g = np.random.default_rng(21)
    block, n = (16, 32)[fmt], 256
    K = (1 << 24) * block + 1024 + 16
    starts = [0, (1 << 24) * block - n, K - 16 - n]  # multiples of a group of four blocks
    short = [_rows(g, 1, 3 * n) for _ in range(2)]
    ms = []
    for x in short:
        xd = torch.zeros(1, K, dtype=torch.bfloat16, device="cuda")
        for i, s in enumerate(starts):
            xd[0, s:s + n] = torch.from_numpy(x[0, i * n:(i + 1) * n])
        m, few = D.Fp4Matrix.empty(fmt, 1, K), D.Fp4Matrix.empty(fmt, 1, 3 * n)
        D.dit_fp4_quantize(xd, m)
        D.dit_fp4_quantize(dev(x).bfloat16(), few)
        scales, tiles = m.scales.view(-1, 512)[:, :4], few.scales.view(-1, 512)[:, :4]  # row 0 of each tile
        per = n // (4 * block)
        for i, s in enumerate(starts):
            assert torch.equal(m.codes[s // 2:(s + n) // 2], few.codes[i * n // 2:(i + 1) * n // 2])
            assert torch.equal(scales[s // (4 * block):][:per], tiles[i * per:(i + 1) * per])
        assert int(scales.count_nonzero()) == int(tiles.count_nonzero())
        xd.fill_(77)
        D.dit_fp4_dequantize(m, xd)
        back = torch.empty(1, 3 * n, dtype=torch.bfloat16, device="cuda")
        D.dit_fp4_dequantize(few, back)
        for i, s in enumerate(starts):
            assert torch.equal(xd[0, s:s + n], back[0, i * n:(i + 1) * n])
        assert int(xd.count_nonzero()) == int(back.count_nonzero())
        del xd, scales
        ms.append((m, few))
    D.dit_check()
    out, ref = torch.empty(1, 1, device="cuda"), torch.empty(1, 1, device="cuda")
    D.dit_fp4_matmul(ms[0][0], ms[1][0], out)
    D.dit_fp4_matmul(ms[0][1], ms[1][1], ref)
    D.dit_check()
    codes = [O.fp4_quantize(x, fmt) for x in short]
    a, b = (O.fp4_values(*c, fmt, 3 * n).astype(np.float64) for c in codes)
    for o in (out, ref):  # zeros add no rounding of their own: both as the short product
        _check_product(o, a, b, 3 * n)


@pytest.mark.parametrize("out,pad,shift", [(torch.float32, 0, 0), (torch.float32, 3, 1), (torch.bfloat16, 0, 0)],
                         ids=["fp32", "fp32-off", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 1000, 256), (17, 256, 1000), (100, 300, 5003), (129, 257, 257), (1100, 1500, 777)])
def test_rows_of_any_size_multiply_without_overflow(M, N, K, out, pad, shift):
    # rows from 2^-98 to 2^126 against one another, huge ones against tiny ones among them: wherever the value is finite
    # the product is, and as exact as the gate says; wherever it is past fp32 it is infinite. Every kernel: pairs
    # of CTAs with either operand first (off 32 bytes the second), one CTA and a cluster of them. A store below 2^-126
    # is off by half of 2^-149 (a bf16 one, which the 2^-126 steps of its type, by half of 2^-133).
    g = np.random.default_rng(M + N + K)
    x, w = (_as_bf16(g.standard_normal((n, K)).clip(-3, 3)) for n in (M, N))
    ex, ew = (g.integers(-98, 126, (n, 1)) for n in (M, N))
    ex[:1], ew[:3] = 120, [[-20], [-90], [-110 + 14]]
    if M > 8:
        ex[1:4], ew[3:5] = [[-97], [70], [0]], [[96], [64]]
    x, w = ((v * 2.0 ** (e - 2.0)).astype(np.float32) for v, e in ((x, ex), (w, ew)))
    a, av = _quantised(x, NV)
    b, bv = _quantised(w, NV)
    o = _on_gpu(np.full((M, N), 9.0, np.float32), out, pad, shift)
    D.dit_fp4_matmul(a, b, o)
    D.dit_check()
    ref, S = av @ bv.T, np.abs(av) @ np.abs(bv).T
    got = o.float().cpu().numpy().astype(np.float64)
    half = 2.0 ** -8 if out == torch.bfloat16 else 0.0
    gate = (K / 64 + 2) * 2.0 ** -23 * S + half * np.abs(ref) + 2.0 ** (-134 if half else -149)
    top = 2.0 ** 128 * (1 - (2.0 ** -9 if half else 2.0 ** -25))  # what rounds to infinity from here on
    finite, past = np.abs(ref) + gate < top, np.abs(ref) - gate > top
    assert finite.sum() > 0.2 * M * N and (M * N < 20000 or past.any())
    with np.errstate(invalid="ignore"):
        bad = finite & ~(np.abs(got - ref) <= gate)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4])
    assert np.array_equal(got[past], np.sign(ref[past]) * np.inf)


# clusters of two, four and eight CTAs for each height of the split kernel's tiles, from a single row on
CLUSTER_SIZES = [(1, 77, 6659), (16, 1024, 14000), (1, 1000, 14000), (3, 2048, 13315), (17, 77, 5123), (32, 2048, 9000),
                 (23, 3000, 12035), (65, 3000, 3331), (100, 4000, 3400)]


@FMT
@pytest.mark.parametrize("M,N,K", CLUSTER_SIZES)
def test_matmul_of_few_rows_on_clusters(fmt, M, N, K):
    test_matmul(fmt, M, N, K)


@pytest.mark.parametrize("M,N,K", [(1, 1000, 256), (100, 300, 5003), (1100, 1500, 777)])
def test_power_of_two_blocks_of_any_size_multiply(M, N, K):
    # blocks of 2^90 against blocks of 2^-110: scales meet inside the product, as exact as any others. (Sums below 2^-90
    # are left out: terms there may be subnormal.)
    g = np.random.default_rng(M + K)
    x, w = (_as_bf16(g.standard_normal((n, K))) for n in (M, N))
    x, w = ((v * 2.0 ** g.integers(lo, hi, (v.shape[0], 1))).astype(np.float32) for v, lo, hi in ((x, 0, 90), (w, -110, 0)))
    a, av = _quantised(x, MX)
    b, bv = _quantised(w, MX)
    o = torch.empty(M, N, device="cuda")
    D.dit_fp4_matmul(a, b, o)
    D.dit_check()
    ref, S = av @ bv.T, np.abs(av) @ np.abs(bv).T
    seen = S > 2.0 ** -90
    assert seen.mean() > 0.7
    assert (np.abs(o.cpu().numpy() - ref) <= (K / 64 + 2) * 2.0 ** -23 * S)[seen].all()


@FMT
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("R,K,pad", [(40, 64, 0), (40, 5003, 1), (700, 40, 0), (700, 64, 1), (700, 200, 0), (700, 250, 1),
                                     (700, 900, 0), (700, 1999, 1), (700, 2900, 0), (613, 4000, 0), (613, 4096, 1)])
def test_quantize_of_non_finite_rows_by_every_kernel(fmt, dtype, R, K, pad):
    # infinities and NaN of either sign and of both kinds, the largest and the smallest values, zeros of either sign: in the
    # kernel with a CTA per row (40 rows) and those with 8, 16 or 32 lanes per row and 1 to 8 units per lane
    g = np.random.default_rng(R + K + pad)
    x = _rows(g, R, K).astype(np.float32)
    odd = np.array([0x7f800000, 0xff800000, 0x7fc00000, 0xffc00000, 0x7f810000, 0xff810000, 0x7fff0000], np.uint32)
    odd = np.concatenate([odd, np.array([0x7f7f0000, 0xff7f0000, 0x00010000, 0x80000000, 0x00800000], np.uint32)])
    at = g.permutation(R)[:3 * len(odd)]
    for i, r in enumerate(at):
        x.view(np.uint32)[r, (0, K - 1, int(g.integers(K)))[i // len(odd)]] = odd[i % len(odd)]
    x[g.permutation(R)[:3]] = np.array([0.0, -0.0, 2.0 ** -126], np.float32)[:, None]
    mem = torch.full((R, K + pad), 77.0, dtype=dtype, device="cuda")
    bits = np.ascontiguousarray(x).view(np.uint32)
    mem[:, :K] = dev((bits >> 16).astype(np.uint16).view(np.int16)).view(torch.bfloat16) if dtype == torch.bfloat16 \
        else dev(bits.view(np.int32)).view(torch.float32)
    m, out = D.Fp4Matrix.empty(fmt, R, K), torch.empty(R, K, device="cuda")
    m.codes.fill_(255)
    m.scales.fill_(254)
    D.dit_fp4_quantize(mem[:, :K], m)
    codes, scale, row = _check_quantised(m, x, fmt)
    assert (~np.isfinite(row)).sum() >= 15 if fmt == NV else (scale == 255).sum() >= 15
    D.dit_fp4_dequantize(m, out)
    D.dit_check()
    assert np.array_equal(out.cpu().numpy(), O.fp4_values(codes, scale, row, fmt, K), equal_nan=True)


def test_products_under_a_set_error_word():
    # after a wait that gave up (the library's own diagnostic sets the word) a product may stop short, but what it has in
    # flight is waited for; the word is reported, and from then on products are right again
    g = np.random.default_rng(31)
    jobs = []
    for fmt, M, N, K in ((NV, 1300, 1536, 3000), (MX, 1037, 1500, 777), (NV, 3, 2048, 9000), (MX, 100, 3000, 3331), (NV, 333, 777, 1000)):
        a, av = _quantised(_rows(g, M, K), fmt)
        b, bv = _quantised(_rows(g, N, K), fmt)
        jobs.append((a, b, torch.empty(M, N, device="cuda"), av, bv, K))
    D.dit_check()
    D.dit_selftest_bounded_wait(False)
    for _ in range(4):
        for a, b, out, *_ in jobs:
            D.dit_fp4_matmul(a, b, out)
    with pytest.raises(D.DitError) as e:
        D.dit_check()
    assert e.value.status == D.DIT_ETIMEOUT
    D.dit_check()
    for a, b, out, av, bv, K in jobs:
        out.fill_(9)
        D.dit_fp4_matmul(a, b, out)
        D.dit_check()
        _check_product(out, av, bv, K)
