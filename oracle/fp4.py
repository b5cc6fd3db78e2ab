"""Microscaled 4-bit matrices in NumPy: quantisation (float32 decisions, as the library documents
them), the values that codes and scales stand for, and the stored layout.

Codes are kept as an index 0..7 into VALUES plus 8 for a minus sign. Rounding to a code is done by
comparing with the midpoints of neighbouring values, rounding to an e4m3 scale by the nearest of its
127 finite non-negative values: no conversion instruction or table of the CUDA side is used."""

import numpy as np

from .dit import (attention, bf16_rne_bits, bf16_to_f64, modulated_rmsnorm, qk_rmsnorm, rotate, swiglu_interleaved,
                  _mod_rows)

NV, MX = 0, 1
BLOCK = {NV: 16, MX: 32}
VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
F32 = np.float32


def e4m3_values():
    """The finite non-negative e4m3 values by their byte: 3 fraction bits, exponent bias 7, subnormals
    of 2^-9, the last byte (0x7f) a NaN and left out."""
    b = np.arange(127)
    e, f = b >> 3, b & 7
    return np.where(e == 0, f * 2.0 ** -9, (1 + f / 8.0) * 2.0 ** (e - 7.0))


def _nearest_even(v, table):
    """Index of the entry of the ascending `table` nearest to v >= 0, ties to the even index."""
    hi = np.clip(np.searchsorted(table, v, side="left"), 1, len(table) - 1)
    lo = hi - 1
    mid = (table[lo] + table[hi]) / 2  # exact: the entries have few bits
    up = (v > mid) | ((v == mid) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def _blocks(x, n):
    R, K = x.shape
    nb = -(-K // n)
    out = np.zeros((R, nb * n), dtype=F32)
    out[:, :K] = x
    return out.reshape(R, nb, n)


def fp4_quantize(x, fmt):
    """x [R, K] float32 -> (codes [R, K rounded up to 32] uint8, one per value, scale bytes [R, nb] uint8,
    row scales [R] float32 or None)."""
    x = np.asarray(x, F32)
    R, K = x.shape
    b = _blocks(x, BLOCK[fmt])
    mag = np.abs(b)
    fine = np.isfinite(b)
    with np.errstate(all="ignore"):
        if fmt == NV:
            ok = fine.all(axis=(1, 2))
            top = np.where(ok, np.where(fine, mag, 0).max(axis=(1, 2)), 0).astype(F32)
            live = ok & (top >= F32(2.0) ** -100)
            safe = np.where(live, top, F32(1)).astype(F32)
            blk = np.where(live[:, None, None], mag, 0).max(axis=2).astype(F32)
            s_in = np.minimum(blk * (F32(448) / safe)[:, None], F32(448))
            scale = _nearest_even(s_in.astype(np.float64), e4m3_values()).astype(np.uint8)
            s = e4m3_values()[scale].astype(F32)
            inv = np.where(s > 0, (F32(2688) / safe)[:, None] / np.where(s > 0, s, F32(1)), F32(0)).astype(F32)
            inv = np.where(live[:, None], inv, F32(0))
            row = np.where(ok, np.where(live, top / F32(2688), F32(0)), F32(np.nan)).astype(F32)
        else:
            ok = fine.all(axis=2)
            blk = np.where(ok, np.where(fine, mag, 0).max(axis=2), 0).astype(np.float64)
            e = np.where(blk > 0, np.floor(np.log2(np.where(blk > 0, blk, 1))) - 2, -127)
            # log2 may round up just below a power of two
            e = np.where((blk > 0) & (2.0 ** (e + 2) > blk), e - 1, e)
            e = np.clip(e, -127, 127)
            scale = np.where(ok, e + 127, 255).astype(np.uint8)
            inv = np.where(ok & (blk > 0), 2.0 ** -e, 0).astype(F32)
            row = None
        y = (np.where(np.isfinite(b), b, 0) * inv[:, :, None]).astype(F32)
    idx = _nearest_even(np.minimum(np.abs(y), 6).astype(np.float64), VALUES).astype(np.uint8)
    idx |= (np.signbit(y) & (inv[:, :, None] != 0)).astype(np.uint8) << 3
    wide = -(-K // 32) * 32
    codes = np.zeros((R, wide), np.uint8)
    flat = idx.reshape(R, -1)
    codes[:, :min(wide, flat.shape[1])] = flat[:, :wide]
    codes[:, K:] = 0
    return codes, scale, row


def fp4_values(codes, scale, row, fmt, K):
    """The float32 values: (code * s) * g, each product rounded once (the first is exact)."""
    n = BLOCK[fmt]
    v = np.where(codes & 8, -VALUES[codes & 7], VALUES[codes & 7])
    nb = scale.shape[1]
    full = np.zeros((codes.shape[0], nb * n))
    w = min(nb * n, v.shape[1])
    full[:, :w] = v[:, :w]
    full = full.reshape(codes.shape[0], nb, n)
    with np.errstate(invalid="ignore", over="ignore", under="ignore"):
        if fmt == NV:
            out = (full * e4m3_values()[scale][:, :, None]).astype(F32) * row[:, None, None]
        else:
            s = np.where(scale == 255, np.nan, 2.0 ** (scale.astype(np.float64) - 127))
            out = (full * s[:, :, None]).astype(F32)
    return out.astype(F32).reshape(codes.shape[0], -1)[:, :K]


def fp4_pack(codes, scale, fmt):
    """The stored layout: code bytes [R, wide / 2] and the scale bytes of the tiles (zero where no row is)."""
    packed = (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)
    R, nb = scale.shape
    groups = -(-nb // 4)
    tiles = np.zeros((-(-R // 128), groups, 32, 4, 4), np.uint8)  # band, group, row % 32, row / 32, block
    for r in range(R):
        padded = np.zeros(groups * 4, np.uint8)
        padded[:nb] = scale[r]
        tiles[r // 128, :, r % 32, (r % 128) // 32, :] = padded.reshape(groups, 4)
    return packed, tiles.reshape(-1)


def fp4_linear_f(x, wvalues, fmt):
    """The 4-bit linear of an activation x (taken at its bfloat16 value, quantised per row) with the
    values wvalues [out, in] that the quantised weight stands for; the product in float64."""
    xb = bf16_to_f64(bf16_rne_bits(np.asarray(x, np.float64).astype(F32))).astype(F32)
    v = fp4_values(*fp4_quantize(xb, fmt), fmt, xb.shape[1]).astype(np.float64)
    return v @ np.asarray(wvalues, np.float64).T


def block_forward_fp4_rows(x, wvalues, fmt, mod, mod_map, cos, sin, heads, head_dim, rows=None, norm1=None,
                           norm2=None, q_norm=None, k_norm=None, eps=1e-6, qk_eps=1e-6):
    """The AdaLN block (see oracle.dit.block_forward_rows for its nine steps) whose four linears (qkv, out,
    up, down) are 4-bit ones: each activation (h, o, h2, a) enters at its bfloat16 value and is quantised
    per row. wvalues: the four weights' values. Float64 otherwise; rows as in block_forward_rows."""
    x = np.asarray(x, dtype=np.float64)
    R, H = x.shape
    nh, d = heads, head_dim
    rows = np.arange(R) if rows is None else np.asarray(rows)
    sa, ca, _, _, _, _ = _mod_rows(mod, mod_map, np.arange(R))
    qkv = fp4_linear_f(modulated_rmsnorm(x, norm1, sa, ca, eps), wvalues[0], fmt)
    q = rotate(qk_rmsnorm(qkv[:, :H].reshape(R, nh, d), q_norm, qk_eps), cos, sin)
    k = rotate(qk_rmsnorm(qkv[:, H:2 * H].reshape(R, nh, d), k_norm, qk_eps), cos, sin)
    o = attention(q, k, qkv[:, 2 * H:].reshape(R, nh, d), rows)
    _, _, ga, sm, cm, gm = _mod_rows(mod, mod_map, rows)
    xr = x[rows] + ga * fp4_linear_f(o, wvalues[1], fmt)
    a = swiglu_interleaved(fp4_linear_f(modulated_rmsnorm(xr, norm2, sm, cm, eps), wvalues[2], fmt))
    return xr + gm * fp4_linear_f(a, wvalues[3], fmt)
