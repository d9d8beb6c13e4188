"""CPU checks of the operators around attention: argument checks through the C
ABI (nothing is launched) and the reference's own consistency."""

import ctypes

import numpy as np
import pytest

import attention_reference as A
import mx_reference as R
from quantized_linear_token_b200 import binding as B
from quantized_linear_token_b200 import build as Bld

# pointers that are never followed: every call below returns on its checks
P, ODD = 1 << 20, (1 << 20) + 8


@pytest.fixture(scope="module")
def lib():
    Bld.build()
    return B.load_library()


class _Handle(ctypes.Structure):
    """An oq_kv4 as the library lays it out, of the device that a machine without GPUs has (none)."""
    _fields_ = [("heads", ctypes.c_int), ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("groups", ctypes.c_int),
                ("device", ctypes.c_int), ("d_error", ctypes.c_void_p)]


@pytest.fixture(scope="module")
def kv():
    import torch
    return _Handle(8, 2, 128, 2, torch.cuda.current_device() if torch.cuda.is_available() else -1, None)


def test_create_refusals(lib):
    h = ctypes.c_void_p()
    f = lambda *a: lib.oq_kv4_create(*a, ctypes.byref(h))
    assert f(0, 1, 128) == 1 and f(4, 0, 128) == 1 and f(4, -1, 64) == 1
    assert f(4, 3, 128) == 2 and f(4, 2, 96) == 2 and f(4, 2, 256) == 2 and f(1 << 17, 1, 64) == 2
    assert lib.oq_kv4_create(4, 2, 128, None) == 1
    assert not h.value
    lib.oq_kv4_destroy(None)


def test_cache_size(lib, kv):
    assert lib.oq_kv4_cache_size(ctypes.byref(kv), 3) == 3 * 2 * 272 * 64
    for pages in (0, -1, 1 << 40, (1 << 31) // 272):
        assert lib.oq_kv4_cache_size(ctypes.byref(kv), pages) == 0
    assert lib.oq_kv4_cache_size(None, 3) == 0


@pytest.mark.parametrize("n", [1 << 60, 1 << 61, 1 << 62, (1 << 62) + 3])
def test_counts_whose_products_leave_64_bits(lib, kv, n):
    h = ctypes.byref(kv)
    assert lib.oq_kv4_cache_size(h, n) == 0
    assert lib.oq_kv4_read(h, 64 * P, n, 5 * P, 4, 6 * P, 7 * P, 2, 3, P, 2 * P, 0, None) == 2
    assert lib.oq_kv4_attention(h, P, 1024, n, 64 * P, 8, 5 * P, 4, 6 * P, 7 * P, 2, 2, 300, 0.1, 1, 0, 2 * P, None, 0, None) == 2


def test_norm_rope_refusals(lib):
    def f(q=P, qs=512, qh=4, k=2 * P, ks=256, kh=2, dt=1, T=3, D=128, gq=4 * P, gk=4 * P, gdt=0, eps=1e-6, table=5 * P, rows=9,
          rot=128, pos=6 * P, flags=0, qo=7 * P, qos=512, ko=8 * P, kos=256):
        return lib.oq_qk_norm_rope(q, qs, qh, k, ks, kh, dt, T, D, gq, gk, gdt, eps, table, rows, rot, pos, flags, qo, qos, ko, kos, None)

    assert f(T=-1) == 1 and f(D=0) == 1 and f(qh=-1) == 1 and f(qh=0, kh=0) == 1
    assert f(D=12) == 2 and f(D=264) == 2 and f(qh=1 << 17) == 2 and f(T=1 << 31) == 2
    assert f(dt=2) == 1 and f(gdt=-1) == 1 and f(flags=4) == 1 and f(flags=2) == 1
    assert f(eps=-1e-9) == 1 and f(eps=float("nan")) == 1 and f(eps=float("inf")) == 1
    assert f(gq=ODD) == 1 and f(table=ODD) == 1 and f(pos=ODD + 2) == 1 and f(rows=0) == 1
    assert f(rot=0) == 2 and f(rot=136) == 2 and f(rot=24) == 2 and f(rot=12, flags=1) == 2
    assert f(q=None) == 1 and f(q=ODD) == 1 and f(k=None) == 1 and f(qo=None) == 1 and f(ko=ODD) == 1
    assert f(qs=504) == 1 and f(qs=513) == 1 and f(kos=255) == 1 and f(qos=1 << 50) == 1
    assert b"oq_qk_norm_rope" in lib.oq_last_error()
    assert f(T=0, q=None, k=None, qo=None, ko=None) == 0


def test_norm_rope_overlaps(lib):
    """Rows may lie in each other's gaps; an output may be its own input, and nothing else."""
    def f(q=P, k=2 * P, qo=3 * P, ko=4 * P, s=(1024, 1024, 512, 256)):
        return lib.oq_qk_norm_rope(q, s[0], 4, k, s[1], 2, 1, 100, 128, None, None, 0, 1e-6, None, 0, 0, None, 0, qo, s[2], ko, s[3], None)

    ok = 3 if _no_gpu() else 0
    if _no_gpu():   # past the checks a launch is refused by the runtime
        assert f(k=P + 1024, s=(1024, 1024, 512, 256)) == ok
        assert f(k=P + 1024, qo=P, ko=P + 1024, s=(1024,) * 4) == ok
    assert f(qo=P) == 1                                      # q's place, another stride
    assert f(k=P + 1024, qo=P + 512, s=(1024,) * 3 + (256,)) == 1
    assert f(k=P + 1024, qo=P + 1024, s=(1024,) * 3 + (256,)) == 1
    assert f(ko=3 * P + 512) == 1 and f(qo=4 * P - 16) == 1
    assert b"overlap" in lib.oq_last_error()


def _no_gpu():
    import torch
    return not torch.cuda.is_available()


def test_append_refusals(lib, kv):
    def f(h=ctypes.byref(kv), q=P, qs=1024, k=2 * P, ks=256, v=3 * P, vs=256, dt=1, T=3, gq=None, gk=None, gdt=0, eps=1e-6,
          table=None, rows=0, rot=0, pos=None, flags=0, qo=4 * P, cache=64 * P, pages=8, pt=5 * P, w=4, cu=6 * P, lens=7 * P, b=2):
        return lib.oq_kv4_append(h, q, qs, k, ks, v, vs, dt, T, gq, gk, gdt, eps, table, rows, rot, pos, flags, qo, cache, pages,
                                 pt, w, cu, lens, b, None)

    assert f(h=None) == 1 and f(pages=-1) == 1 and f(w=-1) == 1 and f(b=-1) == 1 and f(T=-1) == 1
    assert f(cache=None) == 1 and f(cache=64 * P + 16) == 1 and f(pt=None) == 1 and f(cu=None) == 1 and f(lens=5 * P + 2) == 1
    assert f(pages=0) == 2 and f(pages=1 << 23) == 2 and f(w=1 << 24) == 2 and f(b=65536) == 2
    assert f(dt=3) == 1 and f(flags=8) == 1 and f(eps=-1.0) == 1 and f(flags=2, gk=P) == 1
    assert f(q=None) == 1 and f(qo=None) == 1 and f(k=None) == 1 and f(v=ODD) == 1 and f(vs=248) == 1
    assert f(table=9 * P, rows=4, rot=8) == 2
    assert f(qo=2 * P) == 1 and f(cache=3 * P) == 1 and f(cache=P - 64) == 1 and f(qo=P, qs=1032) == 1
    assert f(T=0) == 0 and f(b=0) == 0


def test_read_refusals(lib, kv):
    def f(h=ctypes.byref(kv), cache=64 * P, pages=8, pt=5 * P, w=4, cu=6 * P, lens=7 * P, b=2, T=3, k=P, v=2 * P, dt=0):
        return lib.oq_kv4_read(h, cache, pages, pt, w, cu, lens, b, T, k, v, dt, None)

    assert f(h=None) == 1 and f(T=-1) == 1 and f(dt=2) == 1 and f(k=None) == 1 and f(v=ODD) == 1
    assert f(v=P + 16) == 1 and f(k=64 * P) == 1 and f(v=5 * P - 32) == 1 and f(T=1 << 31) == 2 and f(T=0) == 0


def test_attention_refusals(lib, kv):
    def f(h=ctypes.byref(kv), q=P, qs=1024, T=3, cache=64 * P, pages=8, pt=5 * P, w=4, cu=6 * P, lens=7 * P, b=2, mq=2, ml=300,
          scale=0.1, flags=1, win=0, y=2 * P, ws=None, n=0):
        return lib.oq_kv4_attention(h, q, qs, T, cache, pages, pt, w, cu, lens, b, mq, ml, scale, flags, win, y, ws, n, None)

    assert f(h=None) == 1 and f(T=-1) == 1 and f(mq=-1) == 1 and f(ml=-1) == 1 and f(win=-1) == 1
    assert f(scale=0.0) == 1 and f(scale=-0.5) == 1 and f(scale=float("nan")) == 1 and f(scale=float("inf")) == 1
    assert f(flags=2) == 1 and f(q=None) == 1 and f(q=ODD) == 1 and f(qs=1016) == 1 and f(y=None) == 1 and f(y=ODD) == 1
    assert f(ws=None, n=4096) == 1 and f(ws=8 * P + 64, n=4096) == 1
    assert f(T=1 << 29) == 2 and f(mq=1 << 30) == 2
    assert f(y=P) == 1 and f(y=64 * P + 32) == 1 and f(ws=2 * P, n=4096) == 1 and f(ws=64 * P, n=4096) == 1
    assert f(T=0) == 0 and f(b=0) == 0 and f(mq=0) == 0
    assert lib.oq_kv4_attention_workspace_size(None, 1, 1, 1, 1) == 0
    assert lib.oq_kv4_poll_error(None) == 1


def test_w4g_refusals(lib):
    def prep(W=P, dt=0, n=16, d=256, g=64, c=2 * P, s=3 * P, z=4 * P):
        return lib.oq_w4g_prepare(W, dt, n, d, g, c, s, z, None)

    def lin(x=P, xd=1, T=3, d=256, n=16, g=64, c=2 * P, s=3 * P, z=4 * P, y=5 * P, yd=0):
        return lib.oq_linear_w4g(x, xd, T, d, n, g, c, s, z, y, yd, None)

    for f in (prep, lin):
        assert f(n=0) == 1 and f(d=-64) == 1 and f(g=16) == 2 and f(g=96) == 2 and f(d=32) == 2 and f(d=1 << 25) == 2
        assert f(c=None) == 1 and f(c=ODD) == 1 and f(s=None) == 1 and f(s=ODD) == 1
    assert prep(W=None) == 1 and prep(dt=5) == 1 and prep(W=2 * P - 16) == 1 and prep(s=2 * P + 16) == 1 and prep(z=3 * P) == 1
    assert lin(x=ODD) == 1 and lin(y=None) == 1 and lin(xd=2) == 1 and lin(yd=2) == 1 and lin(T=-1) == 1 and lin(T=655351) == 2
    assert lin(y=P) == 1 and lin(y=4 * P) == 1 and lin(T=0, x=None, y=None) == 0


def test_binding_refuses_host_tensors_and_bad_shapes(lib):
    import torch
    x = torch.zeros(2, 4, 64)
    for f in (lambda: B.oq_qk_norm_rope(x), lambda: B.oq_qk_norm_rope(x[0]), lambda: B.oq_w4g_prepare(x[0], 32),
              lambda: B.oq_linear_w4g(x[0], torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2).bfloat16(), group=32)):
        with pytest.raises(ValueError):
            f()


def test_units_cover_every_window():
    """The launches' bound on aligned windows of 32 and 16 holds for every place and count."""
    for size in (32, 16):
        for n in range(1, 200):
            for p0 in range(size):
                w = (p0 + n - 1) // size - p0 // size + 1
                assert w <= n and w <= n // size + 2


def test_query_terms_are_exact():
    """A bf16 element is the sum of two e4m3 terms at the scales the kernel takes, down to 2^-14 of its block's largest."""
    m = np.arange(128, 256) / 128.0
    for e in range(7, -8, -1):              # y in [2^e, 2^(e + 1)), the largest of the block in [128, 256)
        y = m * 2.0 ** e
        hi = R.code_values(R.round_codes(y, 8), 8)
        lo = R.code_values(R.round_codes((y - hi) * 32, 8), 8) / 32
        assert np.array_equal(hi + lo, y), e


def test_written_tokens_read_back():
    rng = np.random.default_rng(0)
    cache = rng.integers(0, 256, (3, 2, 272, 64)).astype(np.uint8)
    cache[:, :, 256:] = 127
    before = cache.copy()
    x = rng.standard_normal((2, 192))
    A.write_token(cache, 1, 77, x[0], x[1])
    k, v = A.cache_values(cache)
    for got, w in ((k, x[0]), (v, x[1])):
        want = R.dequantize(*R.quantize(np.pad(w, (0, 64)).reshape(1, -1), 4), 4)[0]
        assert np.array_equal(got[1, :, 77].ravel(), want)
    k0, v0 = A.cache_values(before)
    k0[1, :, 77], v0[1, :, 77] = k[1, :, 77], v[1, :, 77]
    assert np.array_equal(k, k0) and np.array_equal(v, v0)


def test_attention_reference_of_one_token():
    rng = np.random.default_rng(1)
    K, V = rng.standard_normal((2, 5, 1, 32))
    q = rng.standard_normal((1, 2, 32))
    y, tol = A.attention(q, K, V, np.array([True, False, True, True, True]), 0.3, True, 3)
    p = np.exp(0.3 * q[0, 1] @ K[[2, 3, 4], 0].T)
    assert np.allclose(y[0, 1], p @ V[[2, 3, 4], 0] / p.sum()) and (tol > 0).all()


@pytest.mark.parametrize("stride", [0, -512, 8, 512, 1 << 40])
def test_overlaps_of_one_token(lib, kv, stride):
    """The stride of one token says nothing: any is taken, and overlaps are found."""
    def rope(q=P, k=2 * P, qo=3 * P, ko=4 * P):
        return lib.oq_qk_norm_rope(q, stride, 4, k, stride, 2, 1, 1, 128, None, None, 0, 1e-6, None, 0, 0, None, 0, qo, stride, ko,
                                   stride, None)

    def append(q=P, k=2 * P, v=3 * P, qo=4 * P, cache=64 * P):
        return lib.oq_kv4_append(ctypes.byref(kv), q, stride, k, stride, v, stride, 1, 1, None, None, 0, 1e-6, None, 0, 0, None, 0,
                                 qo, cache, 8, 5 * P, 4, 6 * P, 7 * P, 2, None)

    def attend(q=P, y=2 * P):
        return lib.oq_kv4_attention(ctypes.byref(kv), q, stride, 1, 64 * P, 8, 5 * P, 4, 6 * P, 7 * P, 2, 1, 300, 0.1, 1, 0, y, None,
                                    0, None)

    for f in (lambda: rope(qo=4 * P), lambda: rope(qo=2 * P + 256), lambda: rope(ko=P + 512), lambda: rope(ko=P),
              lambda: append(qo=2 * P), lambda: append(qo=3 * P - 32), lambda: append(cache=P), lambda: attend(y=P),
              lambda: attend(y=P + 1024)):
        assert f() == 1
        assert b"overlap" in lib.oq_last_error()
    if _no_gpu():   # side by side, or in place: past the checks, where the runtime refuses the launch
        assert rope(qo=4 * P - 1024) == 3 and rope(qo=P, ko=2 * P) == 3 and append(qo=P) == 3


def test_arrays_beyond_64_bits_are_refused(lib, kv):
    """Strides and tables whose extents would wrap around: an overlap could go unnoticed."""
    T, stride = (1 << 31) - 1, 1 << 40
    assert lib.oq_qk_norm_rope(P, stride, 4, None, 0, 0, 1, T, 128, None, None, 0, 1e-6, None, 0, 0, None, 0, 2 * P, stride, None, 0,
                               None) == 1
    assert lib.oq_qk_norm_rope(P, 512, 4, None, 0, 0, 1, 3, 128, None, None, 0, 1e-6, 5 * P, 1 << 61, 128, None, 0, 2 * P, 512, None,
                               0, None) == 2
    # 2^22 tokens 2^40 fp32 elements apart: the last one's offset is a multiple of 2^64
    assert lib.oq_kv4_append(ctypes.byref(kv), None, 0, P, stride, 3 * P, stride, 0, (1 << 22) + 1, None, None, 0, 1e-6, None, 0, 0,
                             None, 0, None, 64 * P, 8, 5 * P, 4, 6 * P, 7 * P, 2, None) == 1
    assert b"stride" in lib.oq_last_error()
    size = lambda T: lib.oq_kv4_attention_workspace_size(ctypes.byref(kv), T, 2, 1, 100000)
    assert size(1 << 62) == size(1 << 58) == size((1 << 31) // 8) == 0


def test_calls_from_another_device_are_refused(lib, kv):
    other = _Handle(8, 2, 128, 2, kv.device + 1, None)
    h = ctypes.byref(other)
    for call in (lambda: lib.oq_kv4_poll_error(h),
                 lambda: lib.oq_kv4_read(h, 64 * P, 8, 5 * P, 4, 6 * P, 7 * P, 2, 3, P, 2 * P, 0, None),
                 lambda: lib.oq_kv4_attention(h, P, 1024, 3, 64 * P, 8, 5 * P, 4, 6 * P, 7 * P, 2, 2, 300, 0.1, 1, 0, 2 * P, None, 0,
                                              None)):
        assert call() == 1
        assert b"device" in lib.oq_last_error()


def test_a_scale_whose_product_is_infinite_is_refused(lib, kv):
    """The softmax works in powers of two: an infinite factor would make a score of 0 a NaN."""
    f = lambda scale: lib.oq_kv4_attention(ctypes.byref(kv), P, 1024, 3, 64 * P, 8, 5 * P, 4, 6 * P, 7 * P, 2, 0, 300, scale, 1, 0,
                                           2 * P, None, 0, None)
    assert f(3.3e38) == 1 and f(2.5e38) == 1 and f(2.3e38) == 0 and f(1e-45) == 0


def test_small_query_elements_are_off_by_little():
    """Below 2^-14 of its block's largest an element is off by up to 2^-22 of that."""
    m = np.arange(128, 256) / 128.0
    for e in range(-8, -24, -1):
        y = m * 2.0 ** e
        hi = R.code_values(R.round_codes(y, 8), 8)
        lo = R.code_values(R.round_codes((y - hi) * 32, 8), 8) / 32
        assert np.abs(hi + lo - y).max() <= 128 * 2.0 ** -22


def test_tables_of_more_than_2_30_tokens_are_refused(lib, kv):
    """Places from 2^30 on are what attention takes for tokens that are not there, and for no window."""
    h = ctypes.byref(kv)
    for w, want in ((1 << 23, 0), ((1 << 23) + 1, 2), ((1 << 24) - 1, 2)):
        assert lib.oq_kv4_attention(h, P, 1024, 3, 64 * P, 8, 5 * P, w, 6 * P, 7 * P, 2, 0, 300, 0.1, 1, 0, 2 * P, None, 0, None) == want
        assert lib.oq_kv4_read(h, 64 * P, 8, 5 * P, w, 6 * P, 7 * P, 2, 0, P, 2 * P, 0, None) == want
