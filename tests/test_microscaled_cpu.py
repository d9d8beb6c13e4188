"""CPU checks of the microscaled operators: the plain reference of the tests
against brute force, the library's sizes and its refusals (no kernel is
launched; every bad call returns before it touches the GPU)."""

import ctypes
import itertools

import numpy as np
import pytest

import mx_reference as R
from quantized_linear_token_b200 import binding as B
from quantized_linear_token_b200 import build as Bld


@pytest.fixture(scope="module")
def lib():
    Bld.build()
    return B.load_library()


@pytest.mark.parametrize("bits", [4, 8])
def test_reference_rounding_is_nearest_even(bits):
    t = R.table(bits)
    pts = np.concatenate([t, (t[1:] + t[:-1]) / 2, t[:-1] + 0.3 * np.diff(t), [t[-1] * 1.5]])
    for v in np.concatenate([pts, -pts]):
        d = np.abs(np.abs(v) - t)
        near = np.flatnonzero(d == d.min())
        want = near[0] if len(near) == 1 else [i for i in near if i % 2 == 0][0]
        got = R.round_codes(np.array([v]), bits)[0]
        assert (got & ((1 << (bits - 1)) - 1), got >> (bits - 1)) == (want, int(np.signbit(v)))


@pytest.mark.parametrize("bits", [4, 8])
def test_reference_scale_is_the_definition(bits):
    top = R.table(bits)[-1]
    for e in (-100, -3, 0, 7, 100):
        for m in (1.0, 1.25, 1.999):
            x = np.zeros((1, 32))
            x[0, 5] = -m * 2.0 ** e
            codes, sc = R.quantize(x, bits)
            s = 2.0 ** (int(sc[0, 0]) - 127)
            assert s == 2.0 ** (e - (2 if bits == 4 else 8))
            assert abs(R.dequantize(codes, sc, bits)[0, 5] - np.clip(x[0, 5], -top * s, top * s)) <= abs(x[0, 5]) / 4


def test_reference_layout_round_trip():
    rng = np.random.default_rng(0)
    for rows, d, bits in itertools.product((1, 33, 130), (32, 160), (4, 8)):
        codes = rng.integers(0, 1 << bits, (rows, d)).astype(np.uint8)
        sc = rng.integers(0, 255, (rows, d // 32)).astype(np.uint8)
        c, t = R.pack(codes, sc, bits)
        a, b = R.unpack(c, t, d, bits)
        assert np.array_equal(a, codes) and np.array_equal(b, sc)


@pytest.mark.parametrize("rows,d,bits", [(1, 32, 4), (128, 128, 8), (129, 160, 4), (32760, 13824, 8)])
def test_sizes(lib, rows, d, bits):
    ct, rt = -(-d // 128), -(-rows // 128)
    assert B.oq_mx_codes_size(rows, d, bits) == rows * ct * 16 * bits
    assert B.oq_mx_scales_size(rows, d) == rt * ct * 512


def test_sizes_of_bad_arguments_are_zero(lib):
    for rows, d, bits in ((0, 32, 4), (-1, 32, 4), (1, 0, 4), (1, 31, 4), (1, 65536, 4), (1, 32, 5)):
        assert B.oq_mx_codes_size(rows, d, bits) == 0
    for rows, d in ((0, 32), (-1, 32), (1, 48), (1, 65536)):
        assert B.oq_mx_scales_size(rows, d) == 0


def test_layer_refusals(lib):
    h = ctypes.c_void_p()
    F = B.OQ_FLAG_MICROSCALED

    def create(d_in=256, d_out=256, a=4, w=4, flags=F):
        return lib.oq_layer_create(d_in, d_out, 0, a, w, flags, ctypes.byref(h))

    assert create(flags=F | B.OQ_FLAG_SIGNS) == 1
    assert create(d_in=0) == 1 and create(d_out=-16) == 1
    assert create(a=3) == 2 and create(a=16) == 2 and create(w=2) == 2 and create(w=8) == 2
    assert create(d_in=48) == 2 and create(d_in=65536) == 2 and create(d_out=24) == 2
    assert not h.value


# pointers that are never followed: every call below returns on its checks
P, ODD = 1 << 20, (1 << 20) + 8


def test_quantize_refusals(lib):
    q = lib.oq_mx_quantize
    assert q(P, 1, -1, 32, 4, P, P, None) == 1
    assert q(P, 1, 4, 0, 4, P, P, None) == 1
    assert q(P, 1, 4, 48, 4, P, P, None) == 2
    assert q(P, 1, 4, 65536, 4, P, P, None) == 2
    assert q(P, 1, 4, 32, 6, P, P, None) == 2
    assert q(P, 1, 1 << 31, 32, 4, P, P, None) == 2
    assert q(P, 7, 4, 32, 4, P, P, None) == 1
    assert q(None, 1, 4, 32, 4, P, P, None) == 1
    assert q(ODD, 1, 4, 32, 4, P, P, None) == 1
    assert q(P, 1, 4, 32, 4, None, P, None) == 1
    assert q(P, 1, 4, 32, 4, P + 16, P, None) == 1
    assert q(P, 1, 4, 32, 4, P, ODD, None) == 1
    assert q(None, 1, 0, 32, 4, None, None, None) == 0      # no rows: nothing to do
    assert b"oq_mx_quantize" in lib.oq_last_error()


def test_dequantize_refusals(lib):
    q = lib.oq_mx_dequantize
    assert q(P, P, -1, 32, 4, P, 1, None) == 1
    assert q(P, P, 4, 40, 4, P, 1, None) == 2
    assert q(P, P, 4, 32, 3, P, 1, None) == 2
    assert q(P, P, 4, 32, 4, P, 9, None) == 1
    assert q(P, P, 4, 32, 4, None, 1, None) == 1
    assert q(P, P, 4, 32, 4, ODD, 1, None) == 1
    assert q(None, P, 4, 32, 4, P, 1, None) == 1
    assert q(P, None, 4, 32, 4, P, 1, None) == 1
    assert q(None, None, 0, 32, 4, None, 1, None) == 0


def test_norm_refusals(lib):
    def f(x=P, r=P, dt=1, g=P, gdt=0, eps=1e-6, rows=4, d=32, bits=8, ro=P, c=P, s=P):
        return lib.oq_rms_norm_mx(x, r, dt, g, gdt, eps, rows, d, bits, ro, c, s, None)

    assert f(rows=-1) == 1 and f(d=0) == 1 and f(d=33) == 2 and f(d=65536) == 2 and f(bits=5) == 2
    assert f(dt=2) == 1 and f(gdt=3) == 1
    assert f(eps=-1e-6) == 1 and f(eps=float("nan")) == 1 and f(eps=float("inf")) == 1
    assert f(x=None) == 1 and f(x=ODD) == 1 and f(r=ODD) == 1 and f(g=ODD) == 1 and f(ro=ODD) == 1
    assert f(r=None) == 1                                    # residual_out without a residual
    assert f(c=None) == 1 and f(s=None) == 1 and f(c=P + 16) == 1 and f(s=ODD) == 1
    assert f(rows=0, x=None, r=None, ro=None, c=None, s=None) == 0


def test_overlapping_outputs_are_refused(lib):
    # 256 rows of 128 bf16 (64 KB): codes 16 KB (4 bits), scales 1 KB; nothing is launched
    X, C, S, K = 1 << 30, 2 << 30, 3 << 30, 4 << 30

    def norm(**k):
        a = {"x": X, "r": K, "g": 5 << 30, "ro": 6 << 30, "c": C, "s": S, **k}
        return lib.oq_rms_norm_mx(a["x"], a["r"], 1, a["g"], 0, 1e-6, 256, 128, 8, a["ro"], a["c"], a["s"], None)

    assert lib.oq_mx_quantize(X, 1, 256, 128, 4, X + 65504, S, None) == 1      # codes begin in x's last row
    assert lib.oq_mx_quantize(X, 1, 256, 128, 4, C, X - 16, None) == 1         # scales end in x's first
    assert lib.oq_mx_quantize(X, 1, 256, 128, 4, C, C + 16368, None) == 1      # scales in the codes
    assert lib.oq_mx_dequantize(C, S, 256, 128, 4, C + 16368, 1, None) == 1
    assert lib.oq_mx_dequantize(C, S, 256, 128, 4, S + 1008, 1, None) == 1
    assert norm(ro=X + 256) == 1 and norm(ro=K - 65520) == 1                   # a row off, not in place
    assert norm(c=X + 32) == 1 and norm(s=K + 16) == 1 and norm(g=(6 << 30) + 16) == 1
    assert b"overlaps" in lib.oq_last_error()


def test_linear_refuses_a_null_layer(lib):
    assert lib.oq_linear_mx(None, P, P, 4, P, P, P, 0, None) == 1


def test_binding_refuses_host_tensors_and_bad_shapes(lib):
    import torch
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        B.oq_mx_quantize(x, 4)
    with pytest.raises(ValueError):
        B.oq_mx_quantize(x[0], 4)
    with pytest.raises(ValueError):
        B.oq_mx_quantize(x, 5)
    with pytest.raises(ValueError):
        B.oq_mx_quantize(torch.zeros(4, 40), 4)
    with pytest.raises(ValueError):
        B.oq_rms_norm_mx(x)
    with pytest.raises(ValueError):
        B.oq_mx_dequantize(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(1, 1, 32, 4, 4, dtype=torch.uint8), 48, 4)


def test_read_back_refuses_missing_scales():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError, match="scales"):
        B.oq_mx_dequantize(torch.zeros(3, 128, dtype=torch.uint8), None, 128, 8)


def test_layer_refuses_widths_past_32_bit_tiles(lib):
    # tile origins are 32-bit: the last tile of such a width would pass them
    h = ctypes.c_void_p()
    for d_out in ((1 << 31) - 16, (1 << 31) - 1008):
        assert lib.oq_layer_create(32, d_out, 0, 4, 4, B.OQ_FLAG_MICROSCALED, ctypes.byref(h)) == 2
        assert not h.value
