"""GPU tests of the microscaled operators through the Python binding, against
the plain fp64 reference (mx_reference.py).  Needs a B200.

Bounds.  Quantisation and read-back have one rounding, to the element type,
and are compared bit for bit.  The norm's fp32 values are off the fp64 ones by
at most DELTA relative: the sum of squares rounds in fp32 at most 75 times
(2^-24 each, all terms positive, halved by the square root), and the mean, the
root, the quotient and the two products add at most 7 half-ulps: below
48 * 2^-24, taken as 64 * 2^-24.  The product's fp32 sums add one value a 32-element block and
split; a tensor core may truncate instead of rounding, so each addition is off
by at most 2^-23 of the magnitudes summed: (K / 32 + 8) 2^-23 sum |a w|, and
bf16 y adds 2^-8 |y|."""

import ctypes

import numpy as np
import pytest

import mx_reference as R

pytestmark = pytest.mark.gpu

DELTA = 64 * 2.0 ** -24


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_linear_token_b200 import build
    build.build()
    from quantized_linear_token_b200 import binding as B
    B.load_library()
    return torch, B


def _dtype(torch, name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _rows(rng, rows, d, dtype):
    """fp32 rows (rounded to bf16 where the input is) with a scale per row, an outlier channel and a zero block."""
    x = rng.standard_normal((rows, d)) * np.exp(rng.standard_normal((rows, 1)))
    x[:, rng.integers(d)] *= 30
    x[rows // 2, :32] = 0
    x = x.astype(np.float32)
    return R.bf16(x) if dtype == "bf16" else x


def _cuda(torch, x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda().to(_dtype(torch, dtype))


def _np(t):
    return t.float().cpu().numpy() if t.dtype.is_floating_point else t.cpu().numpy()


# ------------------------------------------------------------------ quantise, read back
SHAPES = [(1, 32), (3, 160), (64, 256), (127, 128), (128, 96), (129, 288), (300, 2016), (257, 5120)]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,d", SHAPES)
def test_quantize_and_read_back(env, rows, d, dtype, bits):
    torch, B = env
    x = _rows(np.random.default_rng(rows * d + bits), rows, d, dtype)
    codes, scales = B.oq_mx_quantize(_cuda(torch, x, dtype), bits)
    want, sc = R.quantize(x.astype(np.float64), bits)
    c, t = R.pack(want, sc, bits)
    assert np.array_equal(_np(scales), t)
    assert np.array_equal(_np(codes), c)
    v = R.dequantize(want, sc, bits)
    assert np.array_equal(_np(B.oq_mx_dequantize(codes, scales, d, bits)).astype(np.float64), v)
    assert np.array_equal(_np(B.oq_mx_dequantize(codes, scales, d, bits, torch.bfloat16)).astype(np.float64), v)


@pytest.mark.parametrize("bits", [4, 8])
def test_quantize_ties_extremes_and_non_finite(env, bits):
    torch, B = env
    t = R.table(bits)
    grid = np.concatenate([t, (t[1:] + t[:-1]) / 2])
    grid = np.concatenate([grid, -grid])
    rng = np.random.default_rng(5)
    rows = []
    for e in (-140, -126, -60, 0, 60, 118):        # blocks on the element grid and on its ties, far scales
        b = rng.choice(grid, (8, 32)) * 2.0 ** e
        b[:, 0] = t[-1] * 2.0 ** e
        rows.append(b.reshape(1, -1))
    tiny = np.zeros((1, 256))
    tiny[0, 3], tiny[0, 40], tiny[0, 70] = 2.0 ** -149, -(2.0 ** -126), 3.0e38
    rows.append(tiny)
    bad = rng.standard_normal((1, 256))
    bad[0, 1], bad[0, 45], bad[0, 200] = np.inf, np.nan, -np.inf
    rows.append(bad)
    x = np.concatenate(rows).astype(np.float32)
    codes, scales = B.oq_mx_quantize(_cuda(torch, x, "fp32"), bits)
    want, sc = R.quantize(x.astype(np.float64), bits)
    c, tt = R.pack(want, sc, bits)
    assert np.array_equal(_np(scales), tt)
    assert np.array_equal(_np(codes), c)
    v = _np(B.oq_mx_dequantize(codes, scales, 256, bits))
    np.testing.assert_array_equal(v.astype(np.float64), R.dequantize(want, sc, bits).astype(np.float32))
    assert np.isnan(v[-1, :64]).all() and np.isnan(v[-1, 192:224]).all() and np.isfinite(v[-1, 64:192]).all()


def test_read_back_of_every_code(env):
    torch, B = env
    for bits in (4, 8):
        e = np.tile(np.arange(1 << bits, dtype=np.uint8), 256 >> bits).reshape(1, 256)
        for s in (0, 1, 100, 127, 200, 246, 255):
            sc = np.full((1, 8), s, dtype=np.uint8)
            c, t = R.pack(e, sc, bits)
            tc, tt = torch.from_numpy(c).cuda(), torch.from_numpy(t).cuda()
            want = R.dequantize(e, sc, bits).astype(np.float32)
            np.testing.assert_array_equal(_np(B.oq_mx_dequantize(tc, tt, 256, bits)), want)
            np.testing.assert_array_equal(_np(B.oq_mx_dequantize(tc, tt, 256, bits, torch.bfloat16)), R.bf16(want))


# ------------------------------------------------------------------ norm
@pytest.mark.parametrize("rows,d,dtype,bits,residual,gain", [
    (1, 32, "bf16", 8, True, "fp32"), (5, 96, "fp32", 4, False, None), (130, 160, "bf16", 8, True, "bf16"),
    (64, 256, "fp32", 8, True, "fp32"), (333, 2016, "bf16", 4, True, "bf16"), (1, 5120, "bf16", 8, True, "fp32"),
    (100, 5120, "fp32", 8, False, "fp32"), (17, 12288, "bf16", 8, True, None), (9, 13824, "fp32", 8, True, "bf16"),
    (3, 20032, "bf16", 8, True, "fp32"), (2, 28000, "fp32", 8, True, "fp32"), (2, 40992, "bf16", 8, True, "bf16"),
    (3, 65504, "fp32", 4, False, "fp32"),
    # rows enough for CTAs that walk over them, several rows each in the first two
    (3000, 2080, "bf16", 8, True, "fp32"), (2500, 2016, "fp32", 4, True, "bf16"), (400, 5152, "fp32", 8, False, "bf16"),
    (310, 2464, "bf16", 4, False, None), (300, 20032, "bf16", 8, True, "fp32"), (297, 13824, "fp32", 8, True, None)])
def test_norm(env, rows, d, dtype, bits, residual, gain):
    torch, B = env
    rng = np.random.default_rng(d + rows)
    x = _rows(rng, rows, d, dtype)
    r = _rows(rng, rows, d, dtype) if residual else None
    g = (1 + 0.2 * rng.standard_normal(d)).astype(np.float32) if gain else None
    if gain == "bf16":
        g = R.bf16(g)
    tx = _cuda(torch, x, dtype)
    tr = _cuda(torch, r, dtype) if residual else None
    tg = _cuda(torch, g, gain) if gain else None
    codes, scales, kept = B.oq_rms_norm_mx(tx, tg, tr, eps=1e-6, bits=bits)
    h, n = R.norm(x.astype(np.float64), None if r is None else r.astype(np.float64),
                  None if g is None else g.astype(np.float64), 1e-6)
    e, s = R.unpack(_np(codes), _np(scales), d, bits)
    off = R.check_quantized(n, e, s, bits, DELTA)
    assert off <= 10 + 1e-4 * n.size
    if residual:
        sums = x + r                       # fp32, as the kernel adds
        assert np.array_equal(_np(kept), R.bf16(sums) if dtype == "bf16" else sums)
    else:
        assert kept is None
    # what belongs to no row or block holds zeros
    ref_c, ref_t = R.pack(e, s, bits)
    assert np.array_equal(_np(codes), ref_c) and np.array_equal(_np(scales), ref_t)


def test_norm_degenerate_rows(env):
    torch, B = env
    x = np.zeros((4, 160), dtype=np.float32)
    x[1] = 1e-30
    x[2, 7] = np.nan
    x[3, 9] = 5.0
    codes, scales, _ = B.oq_rms_norm_mx(_cuda(torch, x, "fp32"))
    v = _np(B.oq_mx_dequantize(codes, scales, 160, 8))
    assert np.all(v[0] == 0) and np.isfinite(v[1]).all() and np.isnan(v[2]).all()
    want = 5.0 / np.sqrt(25 / 160 + 1e-6)
    assert abs(v[3, 9] - want) <= want / 16 and np.all(np.delete(v[3], 9) == 0)


@pytest.mark.parametrize("rows,d", [(6, 160), (6, 5120), (6, 40992), (1500, 2080)])
def test_norm_writes_the_residual_in_place(env, rows, d):
    torch, B = env
    rng = np.random.default_rng(d)
    x, r = (_cuda(torch, _rows(rng, rows, d, "bf16"), "bf16") for _ in range(2))
    want = B.oq_rms_norm_mx(x, residual=r)
    for which in ("x", "residual"):
        tx, tr = x.clone(), r.clone()
        got = B.oq_rms_norm_mx(tx, residual=tr, residual_out=tx if which == "x" else tr)
        for a, b in zip(want, got):
            assert torch.equal(a, b)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_norm_codes_are_those_of_the_exact_values(env, dtype, bits):
    # Elements next to a border between two codes are formed in fp64, so what
    # is left is the sum of squares: eight are added four fp32 roundings deep,
    # the rest in fp64, and the root halves that: 2 * 2^-24, taken as 2.5.  A
    # code may differ from the fp64 value's only that close to a border.
    # (e4m3's subnormals, below 2^-14 of a block's largest, are formed in fp32.)
    torch, B = env
    rng = np.random.default_rng(3)
    rows, d, delta = 1000, 2048, 2.5 * 2.0 ** -24
    x, r = _rows(rng, rows, d, dtype), _rows(rng, rows, d, dtype)
    g = (1 + 0.2 * rng.standard_normal(d)).astype(np.float32)
    codes, scales, _ = B.oq_rms_norm_mx(_cuda(torch, x, dtype), _cuda(torch, g, "fp32"), _cuda(torch, r, dtype), bits=bits)
    n = R.norm(x.astype(np.float64), r.astype(np.float64), g.astype(np.float64), 1e-6)[1]
    e, s = R.unpack(_np(codes), _np(scales), d, bits)
    want, sc = R.quantize(n, bits)
    normal = (want & 0x7F) >= 8 if bits == 8 else np.ones_like(want, dtype=bool)
    R.check_quantized(n, np.where(normal, e, want), s, bits, delta)
    R.check_quantized(n, e, s, bits, DELTA)


FAR = 2.0 ** -40


@pytest.mark.parametrize("rows,d,dtype,bits,residual,eps", [
    # a CTA a row, or several narrow rows a CTA, whose sums take different ways
    (26, 160, "fp32", 8, True, 0.0), (27, 512, "fp32", 4, False, 0.0), (26, 768, "bf16", 8, True, 0.0),
    (30, 2080, "bf16", 8, True, 2.0 ** -140), (14, 12288, "fp32", 8, False, 0.0), (13, 20032, "bf16", 4, True, 0.0),
    (13, 40992, "fp32", 8, True, 0.0),
    # rows that CTAs walk over, one or several each
    (320, 2080, "bf16", 8, True, 0.0), (1300, 2016, "fp32", 4, True, 2.0 ** -117), (310, 17312, "bf16", 8, True, 0.0),
    (1300, 2016, "bf16", 4, False, 0.0), (1501, 1568, "fp32", 8, False, 0.0), (450, 17312, "fp32", 8, False, 0.0),
    (900, 5120, "fp32", 8, True, 1e-36),
    # an eps beside which such rows do not count
    (320, 2080, "bf16", 8, True, 2.0 ** -116), (1300, 2016, "fp32", 4, True, 2.0 ** -116),
    (303, 17312, "fp32", 8, False, 1e-30)])
def test_norm_of_rows_whose_squares_leave_fp32(env, rows, d, dtype, bits, residual, eps):
    # Rows of every magnitude that the type holds, beside one another, with an
    # eps that hides none of them.  Where the mean square is no ordinary fp32
    # number (below 2^-121 or above 2^121 here) all is formed in fp64: at most
    # 65504 additions, the root and two products, each 2^-53, are below 2^-40.
    # (Squares that overflow are in range for no larger eps.)
    torch, B = env
    rng = np.random.default_rng(rows + d)
    e = np.array([-130, -120, -100, -76, -73, -66, -61, -59, -40, 0, 40, 61, 64, 80, 126])
    hidden = eps > 1e-35
    if hidden:
        e = np.minimum(e, 50)
    mag = 2.0 ** np.roll(e, int(rng.integers(15)))[np.arange(rows) % 15]

    def operand():
        v = (rng.uniform(0.5, 1, (rows, d)) * rng.choice([-1.0, 1.0], (rows, d)) * mag[:, None]).astype(np.float32)
        v[5::15, :] *= np.float32(2.0 ** -20)
        v[5::15, d // 2] = 2.0 ** 30           # one large element, the others far below it
        return R.bf16(v) if dtype == "bf16" else v

    x, r = operand(), operand() if residual else None
    g = (1 + 0.2 * rng.standard_normal(d)).astype(np.float32)
    codes, scales, kept = B.oq_rms_norm_mx(_cuda(torch, x, dtype), _cuda(torch, g, "fp32"),
                                           _cuda(torch, r, dtype) if residual else None, eps=eps, bits=bits)
    h, n = R.norm(x.astype(np.float64), None if r is None else r.astype(np.float64), g.astype(np.float64),
                  float(np.float32(eps)))
    v = (h * h).mean(-1) + float(np.float32(eps))
    far = (v < 2.0 ** -121) | (v > 2.0 ** 121)
    assert hidden or far.sum() >= 3 and (~far).sum() >= 3
    c, s = R.unpack(_np(codes), _np(scales), d, bits)
    R.check_quantized(n, c, s, bits, DELTA)
    if far.any():
        R.check_quantized(n[far], c[far], s[far], bits, FAR)
    if residual:
        with np.errstate(over="ignore"):
            sums = x + r
        assert np.array_equal(_np(kept), R.bf16(sums) if dtype == "bf16" else sums)


@pytest.mark.parametrize("rows", [6, 400, 1500])
def test_norm_of_far_rows_in_place(env, rows):
    torch, B = env
    rng = np.random.default_rng(rows)
    mag = 2.0 ** rng.choice([-120, -70, 0, 90], (rows, 1))
    x, r = (_cuda(torch, rng.standard_normal((rows, 2080)) * mag, "bf16") for _ in range(2))
    want = B.oq_rms_norm_mx(x, residual=r, eps=0.0)
    for which in ("x", "residual"):
        tx, tr = x.clone(), r.clone()
        got = B.oq_rms_norm_mx(tx, residual=tr, eps=0.0, residual_out=tx if which == "x" else tr)
        assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("rows,d", [(5, 160), (9, 512), (300, 2080)])
def test_norm_of_tiny_and_infinite_rows(env, rows, d):
    # a row far below eps is scaled by 1 / sqrt(eps); an infinity makes its
    # block NaN and, by 1 / sqrt(inf) = 0, the rest of its row zeros
    torch, B = env
    rng = np.random.default_rng(1)
    x = rng.standard_normal((rows, d)).astype(np.float32)
    x[1] = 1e-30
    x[3, 40], x[4, 33], x[4, 70] = np.inf, -np.inf, np.nan
    codes, scales, _ = B.oq_rms_norm_mx(_cuda(torch, x, "fp32"), eps=1e-6)
    c, s = R.unpack(_np(codes), _np(scales), d, 8)
    fine = np.ones(rows, dtype=bool)
    fine[3:5] = False
    n = R.norm(x[fine].astype(np.float64), None, None, float(np.float32(1e-6)))[1]
    R.check_quantized(n, c[fine], s[fine], 8, DELTA)
    v = _np(B.oq_mx_dequantize(codes, scales, d, 8))
    assert np.isnan(v[3, 32:64]).all() and np.all(np.delete(v[3], np.s_[32:64]) == 0)
    assert np.isnan(v[4]).all()



# ------------------------------------------------------------------ product
def _operand(rng, rows, d, bits):
    x = rng.standard_normal((rows, d)) * np.exp(rng.standard_normal((rows, 1)))
    e, s = R.quantize(R.bf16(x.astype(np.float32)).astype(np.float64), bits)
    return R.dequantize(e, s, bits), R.pack(e, s, bits)


def _product(env, T, d, n, bits, y_dtype, seed=0):
    torch, B = env
    rng = np.random.default_rng(seed + T + d + n)
    a, (ac, at) = _operand(rng, T, d, bits)
    w, (wc, wt) = _operand(rng, n, d, 4)
    layer = B.oq_layer_create(d, n, 0, bits, 4, B.OQ_FLAG_MICROSCALED)
    args = [torch.from_numpy(v).cuda() for v in (ac, at, wc, wt)]
    y = B.oq_linear_mx(layer, *args, y_dtype=_dtype(torch, y_dtype))
    torch.cuda.synchronize()
    B.oq_poll_error(layer)
    exact = a @ w.T
    tol = (d / 32 + 8) * 2.0 ** -23 * (np.abs(a) @ np.abs(w).T) + (2.0 ** -8 * np.abs(exact) if y_dtype == "bf16" else 0)
    err = np.abs(_np(y).astype(np.float64) - exact)
    assert np.all(err <= tol), f"worst {np.max(err / np.maximum(tol, 1e-300)):.3g} of the bound"
    # the same call again gives the same bits
    again = B.oq_linear_mx(layer, *args, y_dtype=_dtype(torch, y_dtype))
    assert torch.equal(y, again)
    return layer, args, y


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,d,n,y", [
    (1, 32, 16, "fp32"), (1, 256, 128, "fp32"), (1, 2016, 1040, "bf16"), (2, 5120, 272, "fp32"), (16, 128, 144, "bf16"),
    (17, 288, 256, "fp32"), (33, 1024, 96, "bf16"), (64, 640, 400, "fp32"), (65, 160, 128, "fp32"),
    (128, 2048, 512, "bf16"), (129, 96, 48, "fp32"), (256, 1056, 640, "bf16"), (200, 6720, 272, "fp32"),
    (256, 13824, 144, "bf16")])
def test_product_small_batches(env, T, d, n, y, bits):
    _product(env, T, d, n, bits, y)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,d,n,y", [
    (257, 32, 16, "fp32"), (257, 256, 192, "fp32"), (300, 160, 208, "bf16"), (384, 2016, 1040, "fp32"),
    (512, 640, 384, "bf16"), (1001, 1056, 592, "bf16"), (2600, 288, 4624, "fp32")])
def test_product_large_batches(env, T, d, n, y, bits):
    _product(env, T, d, n, bits, y)


def _tile_width(T, n, sms):
    """The large product's rule: the tile width whose waves over the CTA pairs cost least; and its waves."""
    best = None
    for w in (448, 320, 256, 192, 128):
        waves = -(-(-(-T // 256) * -(-n // w)) // (sms // 2))
        cost = waves * (16384 + 1024 + 72 * w)
        if best is None or cost < best[0]:
            best = (cost, w, waves)
    return best[1:]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("y_dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T,n,width,waves", [
    (333, 1040, 128, 1), (500, 5104, 192, 1), (760, 5104, 256, 1), (1000, 5104, 320, 1), (5000, 1232, 448, 1),
    # several tiles a pair: the accumulator is handed back, and the ring of stages goes on
    (19001, 112, 128, 2), (19001, 368, 192, 3), (3000, 2864, 256, 2), (5000, 2000, 320, 2), (5000, 2480, 448, 2)])
def test_product_of_every_tile_width(env, T, n, width, waves, y_dtype, bits):
    # K of 17 column tiles: more stages than the ring holds at either width of
    # codes, the last one of 4-bit codes half empty.  All of y against fp64
    # products of the values that the codes stand for, in the module's bound.
    torch, B = env
    if torch.cuda.get_device_properties(0).multi_processor_count == 148:
        assert _tile_width(T, n, 148) == (width, waves)
    d = 2144
    gen = torch.Generator(device="cuda").manual_seed(T + n)
    x = torch.randn(T, d, generator=gen, device="cuda") * torch.exp(torch.randn(T, 1, generator=gen, device="cuda"))
    x[:, 5] *= 30
    w = torch.randn(n, d, generator=gen, device="cuda") * torch.exp(torch.randn(n, 1, generator=gen, device="cuda"))
    args = (*B.oq_mx_quantize(x, bits), *B.oq_mx_quantize(w, 4))
    layer = B.oq_layer_create(d, n, 0, bits, 4, B.OQ_FLAG_MICROSCALED)
    y = torch.full((T, n), float("nan"), dtype=_dtype(torch, y_dtype), device="cuda")
    assert B.oq_linear_mx(layer, *args, y=y) is y
    a = B.oq_mx_dequantize(*args[:2], d, bits).double()
    v = B.oq_mx_dequantize(*args[2:], d, 4).double()
    exact = a @ v.T
    tol = (d / 32 + 8) * 2.0 ** -23 * (a.abs() @ v.abs().T)
    if y_dtype == "bf16":
        tol += 2.0 ** -8 * exact.abs()
    err = (y.double() - exact).abs()
    assert bool((err <= tol).all()), f"worst {float((err / tol).max()):.3g} of the bound"
    assert torch.equal(B.oq_linear_mx(layer, *args, y_dtype=_dtype(torch, y_dtype)), y)
    B.oq_poll_error(layer)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T", [1, 40, 200, 600])
def test_product_is_exact_where_fp32_is(env, T, bits):
    # values in halves, at most 6 (e2m1's grid, which e4m3 holds too), scales 1
    # and 2: every partial sum is a multiple of 1/4 below 2^22, exact in fp32
    torch, B = env
    rng = np.random.default_rng(T)
    d, n = 1504, 336
    ops = []
    for rows, b in ((T, bits), (n, 4)):
        v = rng.choice(R.E2M1, (rows, d)) * rng.choice([-1.0, 1.0], (rows, d))
        e = R.round_codes(v, b)
        s = rng.integers(127, 129, (rows, d // 32)).astype(np.uint8)
        ops.append((R.dequantize(e, s, b), R.pack(e, s, b)))
    layer = B.oq_layer_create(d, n, 0, bits, 4, B.OQ_FLAG_MICROSCALED)
    (a, (ac, at)), (w, (wc, wt)) = ops
    y = B.oq_linear_mx(layer, *[torch.from_numpy(v).cuda() for v in (ac, at, wc, wt)])
    assert np.array_equal(_np(y).astype(np.float64), a @ w.T)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T", [40, 300])
def test_product_of_nan_blocks(env, T, bits):
    torch, B = env
    layer, (ac, at, wc, wt), y = _product(env, T, 416, 160, bits, "fp32")
    at, wt = at.clone(), wt.clone()
    at[0, 1, 7, 0, 2] = 255          # row 7, block 6
    wt[0, 0, 3, 1, 0] = 255          # weight row 35, block 0
    z = _np(B.oq_linear_mx(layer, ac, at, wc, wt))
    want = _np(y).copy()
    want[7, :] = np.nan
    want[:, 35] = np.nan
    np.testing.assert_array_equal(z, want)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T", [9, 280])
def test_product_over_the_range_of_scales(env, T, bits):
    # a scale code per row from 2^-110 to 2^110, against weight rows from 2^-60
    # to 2^60 (products stay normal in fp32 where both ends do not meet)
    torch, B = env
    rng = np.random.default_rng(bits)
    d, n = 288, 80
    ops = []
    for rows, b, far in ((T, bits, 110), (n, 4, 60)):
        v = rng.choice(R.E2M1[1:], (rows, d)) * rng.choice([-1.0, 1.0], (rows, d))
        s = np.repeat(127 + rng.integers(-far, far + 1, (rows, 1)), d // 32, axis=1).astype(np.uint8)
        e = R.round_codes(v, b)
        ops.append((R.dequantize(e, s, b), R.pack(e, s, b)))
    layer = B.oq_layer_create(d, n, 0, bits, 4, B.OQ_FLAG_MICROSCALED)
    (a, (ac, at)), (w, (wc, wt)) = ops
    y = _np(B.oq_linear_mx(layer, *[torch.from_numpy(v).cuda() for v in (ac, at, wc, wt)])).astype(np.float64)
    # Every partial sum is a multiple of a quarter of the two rows' scales, and
    # at most 288 * 36 of them, so fp32 holds it exactly: as long as it is normal
    # (first condition), and as no partial sum can overflow, which the sum of
    # magnitudes bounds (the result alone does not: terms of both signs).
    exact = a @ w.T
    fine = (np.abs(a).max(1)[:, None] * np.abs(w).max(1)[None, :] > 2.0 ** -100) & (np.abs(a) @ np.abs(w).T < 2.0 ** 127)
    assert fine.mean() > 0.5 and np.array_equal(y[fine], exact[fine])


def test_offsets_past_32_bits(env):
    # 4.6e9 elements of x, 2.3 GB of codes; and y of 4.4e9 elements: the last
    # rows are those of a call on them alone
    torch, B = env
    rows, d = 70016, 65504                # the last 128-row tile begins at a multiple of 128
    x = torch.empty(rows, d, dtype=torch.bfloat16, device="cuda")
    x[:-300].zero_()
    gen = torch.Generator(device="cuda").manual_seed(4)
    x[-300:] = torch.randn(300, d, generator=gen, device="cuda").bfloat16()
    start = (rows - 300) // 128 * 128
    codes, scales = B.oq_mx_quantize(x, 4)
    c, s = B.oq_mx_quantize(x[start:], 4)
    assert torch.equal(codes[start:], c) and torch.equal(scales[start // 128:], s)
    v = B.oq_mx_dequantize(codes, scales, d, 4, torch.bfloat16)
    assert torch.equal(v[start:], B.oq_mx_dequantize(c, s, d, 4, torch.bfloat16))
    del v, codes, scales, c, s
    codes, scales, kept = B.oq_rms_norm_mx(x, residual=x, residual_out=x)
    assert kept is x
    codes1, scales1, _ = B.oq_rms_norm_mx(x[start:])      # h = 2x doubled x in place; the norm of 2x is the same
    assert torch.equal(codes[start:], codes1) and torch.equal(scales[start // 128:], scales1)
    del x, kept, codes, scales, codes1, scales1
    T, k, n = 1 << 19, 64, 8448
    layer = B.oq_layer_create(k, n, 0, 4, 4, B.OQ_FLAG_MICROSCALED)
    ac, at = B.oq_mx_quantize(torch.randn(T, k, generator=gen, device="cuda"), 4)
    wc, wt = B.oq_mx_quantize(torch.randn(n, k, generator=gen, device="cuda"), 4)
    y = B.oq_linear_mx(layer, ac, at, wc, wt, y_dtype=torch.bfloat16)
    last = B.oq_linear_mx(layer, ac[-384:], at[-3:], wc, wt, y_dtype=torch.bfloat16)
    assert torch.equal(y[-384:], last)
    torch.cuda.synchronize()
    B.oq_poll_error(layer)
    del y
    torch.cuda.empty_cache()


def test_product_leaves_what_is_not_its_own(env):
    torch, B = env
    for T in (5, 300):
        layer, args, y = _product(env, T, 288, 144, 8, "bf16")
        buf = torch.full((T + 4, 144), 7.0, dtype=torch.bfloat16, device="cuda")
        B.oq_linear_mx(layer, *args, y=buf[2:T + 2])
        assert torch.equal(buf[2:T + 2], y)
        assert (buf[:2] == 7).all() and (buf[T + 2:] == 7).all()


# ------------------------------------------------------------------ together, streams, graphs, refusals
@pytest.mark.parametrize("T,d,n", [(1, 2016, 1040), (333, 2016, 1040), (70, 5120, 256)])
def test_block_input_chain(env, T, d, n):
    # residual, norm, 8-bit codes, projection: as a block's input runs
    torch, B = env
    rng = np.random.default_rng(T)
    x, r = _rows(rng, T, d, "bf16"), _rows(rng, T, d, "bf16")
    g = (1 + 0.1 * rng.standard_normal(d)).astype(np.float32)
    w = (0.02 * rng.standard_normal((n, d))).astype(np.float32)
    layer = B.oq_layer_create(d, n, 0, 8, 4, B.OQ_FLAG_MICROSCALED)
    wc, wt = B.oq_mx_quantize(_cuda(torch, w, "fp32"), 4)
    codes, scales, kept = B.oq_rms_norm_mx(_cuda(torch, x, "bf16"), _cuda(torch, g, "fp32"), _cuda(torch, r, "bf16"))
    y = _np(B.oq_linear_mx(layer, codes, scales, wc, wt))
    B.oq_poll_error(layer)
    a = R.dequantize(*R.unpack(_np(codes), _np(scales), d, 8), 8)
    wq = R.dequantize(*R.quantize(w.astype(np.float64), 4), 4)
    R.check_quantized(R.norm(x.astype(np.float64), r.astype(np.float64), g.astype(np.float64), 1e-6)[1],
                      *R.unpack(_np(codes), _np(scales), d, 8), 8, DELTA)
    assert np.all(np.abs(y - a @ wq.T) <= (d / 32 + 8) * 2.0 ** -23 * (np.abs(a) @ np.abs(wq).T))
    assert np.array_equal(_np(kept), R.bf16(x + r))


@pytest.mark.parametrize("T", [3, 300])
def test_graph_replay_and_other_stream(env, T):
    torch, B = env
    d, n = 672, 208
    layer = B.oq_layer_create(d, n, 0, 8, 4, B.OQ_FLAG_MICROSCALED)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, r = (torch.randn(T, d, generator=gen, device="cuda").bfloat16() for _ in range(2))
    wc, wt = B.oq_mx_quantize(torch.randn(n, d, generator=gen, device="cuda"), 4)

    def step():
        codes, scales, kept = B.oq_rms_norm_mx(x, residual=r)
        return B.oq_linear_mx(layer, codes, scales, wc, wt), kept

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    x.mul_(2)
    graph.replay()
    want = step()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    torch.cuda.synchronize()
    B.oq_poll_error(layer)


@pytest.mark.parametrize("T", [30, 300])
def test_two_calls_at_once_on_one_layer(env, T):
    torch, B = env
    layer, args, y = _product(env, T, 2016, 400, 4, "fp32")
    streams = [torch.cuda.Stream() for _ in range(4)]
    outs = []
    for k in range(12):
        with torch.cuda.stream(streams[k % 4]):
            outs.append(B.oq_linear_mx(layer, *args))
    torch.cuda.synchronize()
    assert all(torch.equal(o, y) for o in outs)


def test_empty_batch(env):
    torch, B = env
    x = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16)
    codes, scales = B.oq_mx_quantize(x, 4)
    assert tuple(codes.shape) == (0, 64) and tuple(scales.shape) == (0, 1, 32, 4, 4)
    assert tuple(B.oq_mx_dequantize(codes, scales, 64, 4).shape) == (0, 64)
    layer = B.oq_layer_create(64, 32, 0, 4, 4, B.OQ_FLAG_MICROSCALED)
    wc, wt = B.oq_mx_quantize(torch.zeros(32, 64, device="cuda"), 4)
    assert tuple(B.oq_linear_mx(layer, codes, scales, wc, wt).shape) == (0, 32)
    assert B.oq_rms_norm_mx(x, residual=x)[2].shape == x.shape


def test_refusals_on_a_microscaled_layer(env):
    torch, B = env
    layer = B.oq_layer_create(256, 256, 0, 4, 4, B.OQ_FLAG_MICROSCALED)
    x = torch.zeros(4, 256, device="cuda")
    for call in (lambda: B.oq_rotate_quantize(layer, x), lambda: B.oq_weight_prepare(layer, torch.zeros(256, 256, device="cuda")),
                 lambda: B.oq_rotate_quantize_levels(layer, x.bfloat16()), lambda: layer.perm(),
                 lambda: B.oq_linear_fused(layer, x, torch.zeros(256, 32, dtype=torch.int32, device="cuda"), x[0])):
        with pytest.raises(B.OrbitQuantError) as e:
            call()
        assert e.value.status == 2
    assert B.oq_linear_fused_workspace_size(layer, 10) == 0
    assert B.oq_linear_fused_decoded_workspace_size(layer, 10) == 0
    assert B.oq_linear_fused_host_workspace_size(layer, 1, 10) == 0
    # and the microscaled product on another kind of layer
    plain = B.oq_layer_create(256, 256, 0, 4, 4)
    codes, scales = B.oq_mx_quantize(x, 4)
    wc, wt = B.oq_mx_quantize(torch.zeros(256, 256, device="cuda"), 4)
    with pytest.raises(ValueError):
        B.oq_linear_mx(plain, codes, scales, wc, wt)
    L = B.load_library()
    p = [ctypes.c_void_p(t.data_ptr()) for t in (codes, scales, wc, wt, x)]
    assert L.oq_linear_mx(plain.handle, p[0], p[1], 4, p[2], p[3], p[4], 0, None) == 2
    assert L.oq_linear_mx(layer.handle, p[0], p[1], 4, p[2], p[3], None, 0, None) == 1
    assert L.oq_linear_mx(layer.handle, p[0], None, 4, p[2], p[3], p[4], 0, None) == 1
    assert L.oq_linear_mx(layer.handle, p[0], p[1], 4, p[2], p[3], p[4], 5, None) == 1
    # wrong shapes and types
    for bad in ((codes[:, :64], scales, wc, wt), (codes, scales[:, :1], wc, wt), (codes, scales, wc[:128], wt),
                (codes.int(), scales, wc, wt)):
        with pytest.raises(ValueError):
            B.oq_linear_mx(layer, *bad)
    with pytest.raises(ValueError):
        B.oq_mx_quantize(x.t(), 4)
    with pytest.raises(ValueError):
        B.oq_rms_norm_mx(x, residual=x.bfloat16())
    with pytest.raises(ValueError):
        B.oq_rms_norm_mx(x, torch.ones(128, device="cuda"))
    with pytest.raises(TypeError):
        B.oq_mx_quantize(x.half(), 4)


def test_overlapping_outputs_are_refused(env):
    """Every call is refused before a launch; the arrays keep what they held."""
    torch, B = env
    layer = B.oq_layer_create(256, 256, 0, 8, 4, B.OQ_FLAG_MICROSCALED)
    x = torch.randn(64, 256, device="cuda")
    codes, scales = B.oq_mx_quantize(x, 8)
    wc, wt = B.oq_mx_quantize(torch.randn(256, 256, device="cuda"), 4)
    raw = torch.cat([codes.flatten(), torch.zeros(256 * 256 * 4, dtype=torch.uint8, device="cuda")])
    held = raw[:64 * 256].view(64, 256)
    inside = raw[64 * 256 - 16:][:64 * 256 * 4].view(torch.float32).view(64, 256)
    before = raw.clone()
    calls = (lambda: B.oq_linear_mx(layer, held, scales, wc, wt, y=inside),
             lambda: B.oq_mx_dequantize(held, scales, 256, 8, x=inside),
             lambda: B.oq_mx_quantize(inside, 8, codes=held),
             lambda: B.oq_rms_norm_mx(inside, codes=held),
             lambda: B.oq_rms_norm_mx(inside[:32], residual=x[:32], residual_out=inside[16:48]))
    for call in calls:
        with pytest.raises(B.OrbitQuantError) as e:
            call()
        assert e.value.status == 1
    with pytest.raises(ValueError):
        B.oq_linear_mx(layer, codes, scales, wc, wt, y=torch.empty(64, 256, device="cuda"), y_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    assert torch.equal(raw, before)
    # side by side is no overlap
    beside = raw[64 * 256:][:64 * 256 * 4].view(torch.float32).view(64, 256)
    assert torch.equal(B.oq_linear_mx(layer, held, scales, wc, wt, y=beside),
                       B.oq_linear_mx(layer, codes, scales, wc, wt))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("d", [32, 160, 2016, 5120])
def test_layer_words_are_those_of_its_codes(env, d, bits):
    # rows of codes are padded to 128 elements, and the layer says so
    _, B = env
    layer = B.oq_layer_create(d, 32, 0, bits, 4, B.OQ_FLAG_MICROSCALED)
    assert 4 * layer.a_words_per_row * 7 == B.oq_mx_codes_size(7, d, bits)
    assert 4 * layer.w_words_per_row * 32 == B.oq_mx_codes_size(32, d, 4)
