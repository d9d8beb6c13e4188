"""Plain fp64 numpy statement of the microscaled operators, for the tests: the
formats (OCP Microscaling Formats v1.0), the layouts of include/orbitquant.h,
quantisation, the residual norm and the product.  No code of the library."""

import numpy as np

BLOCK = 32
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(m / 8.0 if e == 0 else 1 + m / 8.0) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)][:127])


def table(bits):
    """Magnitudes of an element type by code, ascending."""
    return E2M1 if bits == 4 else E4M3


def round_codes(w, bits):
    """Codes (sign bit on top) of fp64 values: nearest, ties to the even code, saturating."""
    t = table(bits)
    mid = (t[1:] + t[:-1]) / 2
    a = np.abs(w)
    lo, hi = np.searchsorted(mid, a, side="left"), np.searchsorted(mid, a, side="right")
    mag = np.where(hi % 2 == 0, hi, lo)
    return (mag + (np.signbit(w).astype(np.int64) << (bits - 1))).astype(np.uint8)


def code_values(codes, bits):
    c = codes.astype(np.int64)
    mag = c & ((1 << (bits - 1)) - 1)
    t = np.append(E4M3, np.nan) if bits == 8 else E2M1
    return np.where(c >> (bits - 1), -1.0, 1.0) * t[mag]


def scale_codes(x, bits):
    """Scale codes [rows, d / 32] of fp64 rows (exactly representable in fp32)."""
    a = np.abs(x.reshape(x.shape[0], -1, BLOCK))
    bad = ~np.isfinite(a).all(-1)
    amax = np.where(bad, 1.0, np.where(np.isfinite(a), a, 0).max(-1))
    e = np.frexp(np.where(amax > 0, amax, 1.0))[1] - 1 - (2 if bits == 4 else 8)
    code = np.where(amax > 0, np.maximum(e, -127), -127) + 127
    return np.where(bad, 255, code).astype(np.uint8)


def scale_values(sc):
    return np.where(sc == 255, np.nan, np.ldexp(1.0, sc.astype(np.int64) - 127))


def quantize(x, bits):
    """fp64 rows -> (element codes [rows, d], scale codes [rows, d / 32])."""
    sc = scale_codes(x, bits)
    s = np.ldexp(1.0, sc.astype(np.int64) - 127)[..., None]
    b = x.reshape(x.shape[0], -1, BLOCK)
    with np.errstate(invalid="ignore"):
        w = np.where((sc == 255)[..., None], 0.0, b / s)
    return round_codes(w, bits).reshape(x.shape), sc


def dequantize(codes, sc, bits):
    v = code_values(codes, bits).reshape(codes.shape[0], -1, BLOCK) * scale_values(sc)[..., None]
    return v.reshape(codes.shape)


def pack(codes, sc, bits):
    """The arrays of the C ABI: codes [rows, row bytes], scale tiles."""
    rows, d = codes.shape
    ct, rt = -(-d // 128), -(-rows // 128)
    c = np.zeros((rows, ct * 128), dtype=np.uint8)
    c[:, :d] = codes
    if bits == 4:
        c = c[:, 0::2] | (c[:, 1::2] << 4)
    t = np.zeros((rt, ct, 32, 4, 4), dtype=np.uint8)
    for r in range(rows):
        for k in range(d // BLOCK):
            t[r // 128, k // 4, r % 32, r // 32 % 4, k % 4] = sc[r, k]
    return c, t


def unpack(c, t, d, bits):
    rows = c.shape[0]
    if bits == 4:
        e = np.empty((rows, c.shape[1] * 2), dtype=np.uint8)
        e[:, 0::2], e[:, 1::2] = c & 15, c >> 4
    else:
        e = c
    r, k = np.arange(rows)[:, None], np.arange(d // BLOCK)[None, :]
    return e[:, :d], t[r // 128, k // 4, r % 32, r // 32 % 4, k % 4]


def bf16(x):
    """fp32 values rounded to bf16 (nearest even), as fp32."""
    b = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    b = np.where(np.isnan(x), 0x7FC00000, b + 0x7FFF + ((b >> 16) & 1)) >> 16 << 16
    return b.astype(np.uint32).view(np.float32)


def norm(x, residual, gain, eps):
    """fp64: (h, n)."""
    h = x if residual is None else x + residual
    n = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    return h, n if gain is None else n * gain


def check_quantized(n, codes, sc, bits, delta):
    """Codes of values that may be off by delta relative to the fp64 n: every
    element's code lies between those of n (1 - delta) and n (1 + delta) under
    a scale that one of the two gives its block.  Returns how many codes
    differ from those of n itself."""
    lo_s, hi_s = scale_codes(n * (1 - delta), bits), scale_codes(n * (1 + delta), bits)
    assert np.all((sc == lo_s) | (sc == hi_s)), "scales"
    s = np.repeat(np.ldexp(1.0, sc.astype(np.int64) - 127), BLOCK, axis=1)
    half = 1 << (bits - 1)
    mag = codes.astype(np.int64) & (half - 1)
    lo, hi = round_codes(np.abs(n) * (1 - delta) / s, bits), round_codes(np.abs(n) * (1 + delta) / s, bits)
    assert np.all((lo <= mag) & (mag <= hi)), "codes"
    assert np.all((mag == 0) | ((codes >= half) == (n < 0))), "signs"
    return int((codes != quantize(n, bits)[0]).sum())
