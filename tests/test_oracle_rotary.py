"""CPU pins of the rotary oracle, and the library's host plan against it."""

import math

import numpy as np
import pytest

import diffusion_transformer_gb300 as D
import oracle as O

SPECS = [dict(widths=[16, 56, 56]), dict(widths=[96], layout="halves", scaling="linear", factor=3.0),
         dict(widths=[2], theta=100.0), dict(widths=[64, 64], scaling="ntk", factor=4.0),
         dict(widths=[128], scaling="yarn", factor=16.0, original=4096),
         dict(widths=[16, 56, 56], scaling="yarn", factor=2.0, original=64), dict(widths=[256], theta=1e6)]


def _oracle(spec):
    return O.rotary_frequencies(**{k: v for k, v in spec.items() if k != "layout"})


def test_zero_position_is_the_identity_and_inverse_undoes():
    g = np.random.default_rng(0)
    f, ax, amp = O.rotary_frequencies([16, 56, 56])
    x = g.standard_normal((5, 3, 160))
    for halves in (False, True):
        c, s = O.rotary_tables(np.zeros((5, 3)), f, ax)
        assert np.array_equal(O.rotary_apply(x, c, s, halves), x)
        c, s = O.rotary_tables(g.integers(-99, 9999, (5, 3)), f, ax)
        y = O.rotary_apply(x, c, s, halves)
        assert np.allclose(O.rotary_apply(y, c, s, halves, inverse=True), x, atol=1e-12)
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))


def test_pair_layouts_by_hand():
    c, s = np.array([[0.0, 1.0]]), np.array([[1.0, 0.0]])  # quarter turn of pair 0, none of pair 1
    x = np.arange(5.0).reshape(1, 1, 5)
    assert list(O.rotary_apply(x, c, s, False)[0, 0]) == [-1, 0, 2, 3, 4]
    assert list(O.rotary_apply(x, c, s, True)[0, 0]) == [-2, 1, 0, 3, 4]


@pytest.mark.parametrize("spec", SPECS)
def test_host_plan_matches_the_formula(spec):
    plan = D.RotaryPlan(**spec)
    f, ax, amp = _oracle(spec)
    n = sum(spec["widths"]) // 2
    assert plan.c.pairs == n == len(f) and list(plan.c.axis[:n]) == list(ax)
    got = np.array([float(plan.c.turns[i]) for i in range(n)]) * 2.0 ** -64 * 2 * math.pi
    # both sides take a power and a logarithm in 64 bits: a few last places
    assert np.allclose(got, f, rtol=1e-13, atol=2 * math.pi * 2.0 ** -63)
    assert plan.c.amplitude == np.float32(amp)


@pytest.mark.parametrize("bad", [dict(widths=[3]), dict(widths=[0]), dict(widths=[16], theta=1.0),
                                 dict(widths=[16], theta=float("nan")), dict(widths=[16], scaling="linear", factor=0.5),
                                 dict(widths=[16], scaling="ntk", factor=float("inf")),
                                 dict(widths=[16], scaling="yarn", factor=2.0),
                                 dict(widths=[16], scaling="yarn", factor=2.0, original=64, beta_fast=0.5),
                                 dict(widths=[256, 2])])
def test_plan_refusals(bad):
    with pytest.raises(D.DitError):
        D.RotaryPlan(**bad)


def test_plan_takes_only_known_words():
    for bad in (dict(widths=[16], layout="other"), dict(widths=[16], scaling="other")):
        with pytest.raises(KeyError):
            D.RotaryPlan(**bad)
    with pytest.raises(ValueError):
        D.RotaryPlan([2] * 5)


def test_rotary_refusals_before_any_cuda_call():
    import ctypes
    L, p = D.lib(), D.RotaryPlan([64], layout="halves")
    q = D.dit_rotary_rows(256, 256, 4, 0, 256, 64, 0, 256, 64)
    pos = ctypes.c_void_p(256)

    def call(plan=p.c, q=q, k=None, type=0, batch=1, rows=3, d=64, pos=pos):
        return L.dit_rotary(ctypes.byref(plan) if plan is not None else None, ctypes.byref(q) if q else None,
                            ctypes.byref(k) if k else None, type, batch, rows, d, pos, 0, None)

    assert call(plan=None) == -1 and call(q=None) == -1 and call(type=2) == -1 and call(batch=-1) == -1
    assert call(rows=-1) == -1 and call(d=62) == -1 and call(d=512) == -2 and call(pos=None) == -1
    assert call(batch=0) == 0 and call(rows=0) == 0
    assert call(q=D.dit_rotary_rows(256, 256, 0, 0, 256, 64, 0, 256, 64)) == 0           # no heads
    assert call(q=D.dit_rotary_rows(256, 256, -1, 0, 256, 64, 0, 256, 64)) == -1
    assert call(q=D.dit_rotary_rows(None, 256, 4, 0, 256, 64, 0, 256, 64)) == -1
    assert call(q=D.dit_rotary_rows(257, 256, 4, 0, 256, 64, 0, 256, 64)) == -1          # off its type's boundary
    assert call(q=D.dit_rotary_rows(256, 256, 4, 0, 256, 64, 0, 0, 64)) == -1            # output rows on one place
    assert call(q=D.dit_rotary_rows(256, 256, 4, 0, 256, 64, 0, 256, 0)) == -1
    assert call(batch=2, q=D.dit_rotary_rows(256, 256, 4, 0, 256, 64, 0, 256, 64)) == -1
    # in place under other strides
    assert call(q=D.dit_rotary_rows(256, 256, 4, 0, 256, 64, 0, 64, 192)) == -1
    assert call(rows=1, d=64, q=D.dit_rotary_rows(256, 256, 4, 0, 256, 64, 0, 256, 128)) == -1
    # one tensor as q and as k, with an output on it
    assert call(q=q, k=q) == -1
    k = D.dit_rotary_rows(512, 256, 4, 0, 256, 64, 0, 256, 64)
    assert call(q=q, k=k) == -1 and call(q=D.dit_rotary_rows(256, 1024, 4, 0, 256, 64, 0, 256, 64), k=k) == -1
    bad = D.dit_rotary_plan()
    ctypes.memmove(ctypes.byref(bad), ctypes.byref(p.c), ctypes.sizeof(bad))
    bad.axis[5] = 7
    assert call(plan=bad) == -1
    assert L.dit_rotary_tables(ctypes.byref(p.c), pos, -1, pos, pos, None) == -1
    assert L.dit_rotary_tables(ctypes.byref(p.c), None, 4, pos, pos, None) == -1
    assert L.dit_rotary_tables(ctypes.byref(p.c), pos, 0, None, None, None) == 0


def test_fp4_refusals_before_any_cuda_call():
    import ctypes
    L = D.lib()
    M = D.dit_fp4_matrix
    x, r = ctypes.c_void_p(256), ctypes.byref
    good = M(0, 4, 40, 256, 512, 1024)
    assert L.dit_fp4_quantize(x, 0, 40, None, None) == -1
    for m in (M(2, 4, 40, 256, 512, 1024), M(0, -1, 40, 256, 512, 1024), M(0, 4, 0, 256, 512, 1024),
              M(0, 4, 40, None, 512, 1024), M(0, 4, 40, 256, 520, 1024), M(0, 4, 40, 264, 512, 1024),
              M(0, 4, 40, 256, 512, None), M(0, 4, 40, 256, 512, 1026)):
        assert L.dit_fp4_quantize(x, 0, 40, r(m), None) == -1
        assert L.dit_fp4_dequantize(r(m), x, 0, 40, None) == -1
        assert L.dit_fp4_matmul(r(good), r(m), x, 0, 400, None) == -1
        assert L.dit_linear_fp4(x, 0, 4, 40, r(m), x, 0, 400, x, 1 << 20, None) == -1
    for bad in ((None, 0, 40), (x, 2, 40), (x, 0, 39), (ctypes.c_void_p(257), 0, 40), (ctypes.c_void_p(258), 1, 40)):
        assert L.dit_fp4_quantize(*bad, r(good), None) == -1
    empty = M(0, 0, 40, None, None, None)
    assert L.dit_fp4_quantize(None, 0, 40, r(empty), None) == 0
    assert L.dit_fp4_matmul(r(empty), r(good), None, 0, 4, None) == 0
    assert L.dit_fp4_matmul(r(good), r(empty), None, 0, 4, None) == 0
    assert L.dit_fp4_matmul(r(good), r(M(0, 4, 48, 256, 512, 1024)), x, 0, 4, None) == -1   # other inner size
    assert L.dit_fp4_matmul(r(good), r(M(1, 4, 40, 256, 512, None)), x, 0, 4, None) == -1   # other format
    assert L.dit_fp4_matmul(r(good), r(good), x, 0, 3, None) == -1                          # rows overlap
    n = L.dit_linear_fp4_workspace_bytes(0, 4, 4, 40)
    assert n > 0 and L.dit_linear_fp4(x, 0, 4, 40, r(good), x, 0, 4, x, n - 1, None) == -3
    assert L.dit_linear_fp4(x, 0, 4, 40, r(good), x, 0, 4, ctypes.c_void_p(128), n, None) == -1
    assert L.dit_linear_fp4(x, 0, -1, 40, r(good), x, 0, 4, x, n, None) == -1
    assert L.dit_linear_fp4(None, 0, 0, 40, r(good), None, 0, 4, None, 0, None) == 0
    assert L.dit_fp4_code_bytes(3, 33) == 96 and L.dit_fp4_code_bytes(-1, 3) == 0
    assert L.dit_fp4_scale_bytes(0, 129, 65) == 2 * 2 * 512 and L.dit_fp4_scale_bytes(1, 129, 65) == 2 * 512
    assert L.dit_fp4_quantize(x, 0, 1 << 30, r(M(0, 4, (1 << 30) + 1, 256, 512, 1024)), None) == -2
    assert L.dit_fp4_matmul(r(good), r(M(0, (1 << 30) + 1, 40, 256, 512, 1024)), x, 0, 1 << 31, None) == -2
    assert L.dit_linear_fp4(x, 0, (1 << 30) + 1, 40, r(good), x, 0, 4, x, n, None) == -2
    dims, mod = D.dit_dims(256, 4, 64, 128, 1e-6, 1e-6, 0), D.dit_mod(256, None, 1)
    ok = D.dit_block_wfp4((M * 4)(*[M(0, a, b, 256, 512, 1024) for a, b in ((768, 256), (256, 256), (256, 256), (256, 128))]))
    need = L.dit_block_fp4_workspace_bytes(r(dims), 0, 0, 5)

    def block(w, nbytes=need, ws=x, img=x, N=5):
        return L.dit_block_forward_fp4(r(dims), r(w) if w is not None else None, None, 0, img, N, None, None, x, x,
                                       r(mod), ws, nbytes, None)

    assert need > 0 and block(None) == -1 and block(ok, need - 1) == -3 and block(ok, ws=None) == -3
    assert block(ok, img=None) == -1 and block(ok, N=0) == -1 and block(ok, ws=ctypes.c_void_p(128)) == -1
    mixed = D.dit_block_wfp4((M * 4)(*[M(i == 3, a, b, 256, 512, 1024) for i, (a, b) in
                                       enumerate(((768, 256), (256, 256), (256, 256), (256, 128)))]))
    assert block(mixed) == -1
    assert L.dit_fp4_scale_bytes(2, 1, 1) == 0 and L.dit_linear_fp4_workspace_bytes(0, 1, 1, 0) == 0


@pytest.mark.parametrize("w,theta,factor,original,fast,slow", [
    (4, 1e4, 16.0, 4096, 32.0, 1.0), (6, 1e4, 4.0, 4096, 32.0, 1.0), (32, 256.0, 2.0, 1536, 32.0, 1.0),
    (48, 256.0, 4.0, 1536, 32.0, 1.0), (64, 1e4, 4.0, 131072, 32.0, 1.0), (128, 1e4, 4.0, 65536, 32.0, 1.0),
    (128, 1e4, 16.0, 4096, 32.0, 1.0), (96, 5e5, 8.0, 8192, 16.0, 2.0)])
def test_by_parts_is_the_published_range(w, theta, factor, original, fast, slow):
    # the published range of pairs ends at the rotated width less one, not at the last pair, so that a narrow axis (or a
    # long trained length) stops inside the ramp: pairs up to floor(at(fast)) as they are, from ceil(at(slow)) on divided
    def at(turns):
        return w * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(theta))

    lo, hi = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), w - 1)
    want = []
    for k in range(w // 2):
        f = theta ** (-2.0 * k / w)
        keep = 1.0 - min(1.0, max(0.0, (k - lo) / (hi - lo)))
        want.append(f / factor * (1.0 - keep) + f * keep)
    spec = dict(widths=[w], theta=theta, scaling="yarn", factor=factor, original=original, beta_fast=fast, beta_slow=slow)
    f, _, amp = O.rotary_frequencies(**spec)
    assert np.allclose(f, want, rtol=1e-13) and amp == 0.1 * math.log(factor) + 1.0
    got = [D.RotaryPlan(**spec).c.turns[i] * 2.0 ** -64 * 2 * math.pi for i in range(w // 2)]
    assert np.allclose(got, want, rtol=1e-13, atol=2 * math.pi * 2.0 ** -63)


def test_by_parts_of_two_pairs_by_hand():
    # width 4: at(1) = 4 ln(4096 / 2 pi) / (2 ln 10^4) = 1.41, so the ramp runs from pair 0 to 2 and pair 1 is half way
    f, _, _ = O.rotary_frequencies([4], scaling="yarn", factor=16.0, original=4096)
    assert np.allclose(f, [1.0, 0.01 * (0.5 + 0.5 / 16)], rtol=1e-15)


def test_rotary_without_heads_looks_at_nothing():
    import ctypes
    p, r = D.RotaryPlan([64], layout="halves"), ctypes.byref
    none = D.dit_rotary_rows(None, None, 0, 0, 0, 0, 0, 0, 0)
    assert D.lib().dit_rotary(r(p.c), r(none), None, 0, 2, 3, 64, None, 0, None) == D.DIT_OK
    assert D.lib().dit_rotary(r(p.c), r(none), r(none), 0, 2, 3, 64, None, 0, None) == D.DIT_OK
    some = D.dit_rotary_rows(256, 256, 4, 0, 256, 64, 0, 256, 64)
    assert D.lib().dit_rotary(r(p.c), r(none), r(some), 0, 1, 3, 64, None, 0, None) == D.DIT_EINVAL


@pytest.mark.parametrize("spec", SPECS + [
    dict(widths=[4], theta=100.0), dict(widths=[256], theta=100.0), dict(widths=[64], theta=2.5e8, scaling="ntk", factor=2.0),
    dict(widths=[256], theta=100.0, scaling="yarn", factor=40.0, original=64),
    dict(widths=[256], theta=100.0, scaling="linear", factor=1.5)])
def test_fractions_against_sixty_digits(spec):
    # the plan's turns per position are off by less than 2^-54: the stated bound (64-bit floating point takes them, so
    # 2^-65, the last bit of the fraction, is out of reach)
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
    theta, scaling = Decimal(spec.get("theta", 10000.0)), spec.get("scaling", "none")
    factor, turns = Decimal(spec.get("factor", 1.0)), []
    for w in spec["widths"]:
        base = theta * (factor.ln() * w / (w - 2)).exp() if scaling == "ntk" else theta
        lo, hi = (w * (spec["original"] / (n * two_pi)).ln() / (2 * theta.ln()) if scaling == "yarn" else Decimal(0)
                  for n in (32, 1))
        lo, hi = max(0, math.floor(lo)), min(w - 1, math.ceil(hi))
        for k in range(w // 2):
            f = (base.ln() * -2 * k / w).exp()
            if scaling == "linear":
                f /= factor
            elif scaling == "yarn":
                r = min(Decimal(1), max(Decimal(0), Decimal(k - lo) / max(Decimal(hi - lo), Decimal("0.001"))))
                f = f * (1 - r) + f / factor * r
            turns.append(f / two_pi)
    plan = D.RotaryPlan(**spec)
    assert plan.c.pairs == len(turns)
    off = max(abs(Decimal(plan.c.turns[i]) / 2 ** 64 - t) for i, t in enumerate(turns))
    assert off < Decimal(2) ** -54, float(off)
