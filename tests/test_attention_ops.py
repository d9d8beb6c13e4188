"""GPU tests of the operators around attention through the Python binding,
against the plain fp64 reference (attention_reference.py).  Needs a B200.

Bounds.  Norm and rotation: fp32 values off by at most DELTA (|a| + |b|), the sum
of squares 12 half-ulps halved by the root and at most 9 half-ulps after it, below
16 * 2^-24, taken as 32 * 2^-24; and half a step of the output type.  What the
cache holds is compared exactly (an element next to a border between two codes by
less than 2^-40 may have either).  Attention: attention_reference.attention.  The
product: a group's products are exact, its sum takes at most 8 MMAs' additions, the
groups K / group / 8 and the warps and terms 26 more, each off by at most 2^-23 of
the magnitudes added."""

import numpy as np
import pytest

import attention_reference as A
import mx_reference as R

pytestmark = pytest.mark.gpu

DELTA = 32 * 2.0 ** -24
STEP = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


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


def _dt(torch, name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _np(t):
    return t.double().cpu().numpy() if t.dtype.is_floating_point else t.cpu().numpy()


def _heads(torch, rng, T, H, D, dtype, extra=0):
    """[T, H, D] on the GPU, a view with `extra` more heads a token; rows of different magnitude."""
    x = rng.standard_normal((T, H + extra, D)) * np.exp(rng.standard_normal((T, H + extra, 1)))
    return torch.from_numpy(x.astype(np.float32)).cuda().to(_dt(torch, dtype))[:, :H]


def _table(torch, rng, rows, rot):
    a = rng.uniform(-10, 10, (rows, rot // 2))
    return torch.from_numpy(np.stack((np.cos(a), np.sin(a)), -1).astype(np.float32)).cuda()


def _close(got, want, tol, what=""):
    """Within tol where the reference is a number; NaN where it is NaN."""
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), what
    err = np.abs(np.where(nan, 0, got) - np.where(nan, 0, want)) - np.where(nan, 0, tol)
    assert err.max(initial=-1) <= 0, (what, err.max(), np.unravel_index(err.argmax(), err.shape))


# ------------------------------------------------------------------ norm and rotation
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,H,KH,D,rot,inter,norm,gain", [
    (1, 1, 1, 8, 8, True, True, True), (1, 40, 40, 128, 128, True, True, True), (3, 5, 2, 64, 64, False, True, True),
    (257, 3, 0, 72, 48, False, True, False), (33, 7, 3, 96, 96, False, False, False), (129, 24, 8, 256, 128, True, True, True),
    (5, 1, 0, 40, 0, False, True, True), (1000, 2, 1, 128, 64, False, True, True), (2, 300, 7, 32, 32, False, True, True),
    (600, 8, 8, 16, 16, True, False, False)])
def test_norm_rope(env, dtype, T, H, KH, D, rot, inter, norm, gain):
    torch, B = env
    rng = np.random.default_rng(T * 1000 + D)
    q = _heads(torch, rng, T, H, D, dtype, extra=1)
    k = _heads(torch, rng, T, KH, D, dtype, extra=2) if KH else None
    g = [torch.from_numpy(rng.uniform(-2, 2, D).astype(np.float32)).cuda() if gain else None for _ in range(2)]
    table = _table(torch, rng, T + 3, rot) if rot else None
    pos = torch.from_numpy(rng.integers(0, T + 3, T).astype(np.int32)).cuda() if rot else None
    got = B.oq_qk_norm_rope(q, k, g[0], g[1] if KH else None, eps=1e-5, table=table, positions=pos, interleaved=inter, norm=norm)
    for x, y, w in zip((q, k), got, g):
        if x is None:
            assert y is None
            continue
        want, mag = A.turn(_np(x), None if w is None else _np(w), 1e-5, None if table is None else _np(table),
                           None if pos is None else _np(pos), inter, norm)
        assert y.dtype == x.dtype and y.is_contiguous()
        _close(_np(y), want, DELTA * mag + STEP[dtype] * np.abs(want) + 2.0 ** -133)


def test_norm_rope_in_place_in_a_packed_row(env):
    torch, B = env
    rng = np.random.default_rng(1)
    x = _heads(torch, rng, 37, 12, 64, "bf16")
    want = x.clone()
    table = _table(torch, rng, 37, 64)
    gq = torch.rand(64, device="cuda").bfloat16()
    a, b = B.oq_qk_norm_rope(want[:, :8], want[:, 8:10], gq, gq, table=table)
    q, k = x[:, :8], x[:, 8:10]
    r = B.oq_qk_norm_rope(q, k, gq, gq, table=table, q_out=q, k_out=k)
    assert r[0] is q and torch.equal(x[:, :8], a) and torch.equal(x[:, 8:10], b)
    assert torch.equal(x[:, 10:], want[:, 10:])


def test_norm_rope_degenerate_rows(env):
    torch, B = env
    x = np.random.default_rng(2).standard_normal((8, 1, 128))
    x[0] = 0
    x[1] *= 1e30          # squares above fp32
    x[2] *= 1e-30         # below it
    x[3, 0, 5] = np.inf
    x[4, 0, 7] = np.nan
    x[5] *= 1e-42
    t = torch.from_numpy(x.astype(np.float32)).cuda()
    for eps in (1e-6, 0.0):
        got = _np(B.oq_qk_norm_rope(t, eps=eps)[0])
        want, mag = A.turn(_np(t), None, eps)
        _close(got, want, (DELTA + STEP["fp32"]) * np.nan_to_num(mag) + 2.0 ** -149, eps)


@pytest.mark.parametrize("inter", [True, False])
def test_norm_rope_many_tokens(env, inter):
    """Queries and keys of a token in one CTA, a lane group walking over a token's heads."""
    torch, B = env
    rng = np.random.default_rng(30)
    T = 20011
    x = _heads(torch, rng, T, 5, 128, "bf16", extra=1)
    table = _table(torch, rng, T, 64)
    got = B.oq_qk_norm_rope(x[:, :2], x[:, 2:], table=table, interleaved=inter)
    for a, b in zip((x[:, :2], x[:, 2:]), got):
        want, mag = A.turn(_np(a), None, 1e-6, _np(table), np.arange(T), inter)
        _close(_np(b), want, DELTA * mag + STEP["bf16"] * np.abs(want))


def test_norm_rope_rows_out_of_range_among_many(env):
    """More rows than are marked at once, some of them out of fp32's range, in place."""
    torch, B = env
    rng = np.random.default_rng(31)
    x = rng.standard_normal((3000, 300, 8))
    for e in (30, -30):
        x[rng.integers(0, 3000, 50), rng.integers(0, 300, 50)] *= 10.0 ** e
    t = torch.from_numpy(x.astype(np.float32)).cuda()
    table = _table(torch, rng, 3000, 8)
    want, mag = A.turn(_np(t), None, 0.0, _np(table), np.arange(3000), True)
    got = _np(B.oq_qk_norm_rope(t, eps=0.0, table=table, interleaved=True, q_out=t)[0])
    _close(got, want, (DELTA + STEP["fp32"]) * mag + 2.0 ** -149)


def test_positions_outside_the_table_are_nan(env):
    torch, B = env
    rng = np.random.default_rng(3)
    q, table = _heads(torch, rng, 4, 2, 64, "fp32"), _table(torch, rng, 5, 32)
    pos = torch.tensor([0, -1, 5, 4], dtype=torch.int32, device="cuda")
    for inter in (False, True):
        y = _np(B.oq_qk_norm_rope(q, table=table, positions=pos, interleaved=inter)[0])
        want, mag = A.turn(_np(q), None, 1e-6, _np(table), _np(pos), inter)
        assert np.isnan(want[1:3, :, :32]).all() and not np.isnan(want[1:3, :, 32:]).any()
        _close(y, want, (DELTA + STEP["fp32"]) * np.nan_to_num(mag))


# ------------------------------------------------------------------ the cache
class Streams:
    """Sequences with scattered pages over a cache of random bytes."""

    def __init__(self, torch, rng, kv, n, lens, spare=3):
        self.n, self.lens = n, lens
        need = [-(-m // 128) for m in lens]
        pages = sum(need) + spare
        cache = rng.integers(0, 256, (pages, kv.groups, 272, 64)).astype(np.uint8)
        cache[:, :, 256:] = rng.integers(120, 134, cache[:, :, 256:].shape)
        order = rng.permutation(pages)
        self.pages = np.full((len(n), max(need + [1])), pages + 5, np.int32)
        at = 0
        for b, m in enumerate(need):
            self.pages[b, :m] = order[at:at + m]
            at += m
        self.np_cache = cache
        self.free = order[at:]
        self.cache = torch.from_numpy(cache).cuda()
        cu = np.concatenate(([0], np.cumsum(n))).astype(np.int32)
        self.np_cu, self.T = cu, int(cu[-1])
        self.cu = torch.from_numpy(cu).cuda()
        self.table = torch.from_numpy(self.pages).cuda()
        self.len = torch.from_numpy(np.asarray(lens, np.int32)).cuda()

    @property
    def view(self):
        return self.cache, self.table, self.cu, self.len


def _append_expected(s, kv, k, v):
    """The cache after k, v (fp64 [T, KH, D]) joined it."""
    out = s.np_cache.copy()
    for b, (n, m) in enumerate(zip(s.n, s.lens)):
        for i in range(n):
            j = m - n + i
            t = s.np_cu[b] + i
            A.write_token(out, s.pages[b, j // 128], j % 128, k[t].ravel(), v[t].ravel())
    return out


def _same_cache(got, want):
    """Equal but for the sign of zero elements."""
    for x, y in zip(A.cache_values(got), A.cache_values(want)):
        assert np.array_equal(np.isnan(x), np.isnan(y))
        assert np.array_equal(np.nan_to_num(x), np.nan_to_num(y)), np.argwhere(np.nan_to_num(x) != np.nan_to_num(y))[:5]
    assert np.array_equal(got[:, :, 256:], want[:, :, 256:])


APPENDS = [([1], [1]), ([1, 1, 1], [128, 129, 6]), ([0, 3, 1, 2], [50, 3, 260, 34]), ([130, 0, 65], [300, 0, 65]),
           ([33, 31, 32, 2], [64, 95, 32, 33])]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("H,KH,D,inter", [(4, 2, 128, True), (6, 3, 64, False), (1, 1, 64, True)])
@pytest.mark.parametrize("n,lens", APPENDS)
def test_append(env, dtype, H, KH, D, inter, n, lens):
    torch, B = env
    rng = np.random.default_rng(sum(lens) + D)
    kv = B.oq_kv4_create(H, KH, D)
    s = Streams(torch, rng, kv, n, lens)
    x = _heads(torch, rng, s.T, H + 2 * KH, D, dtype)
    q, k, v = x[:, :H], x[:, H:H + KH], x[:, H + KH:]
    g = [torch.from_numpy(rng.uniform(0.5, 2, D).astype(np.float32)).cuda() for _ in range(2)]
    table = _table(torch, rng, max(lens) + 1, D)
    got = B.oq_kv4_append(kv, q, k, v, *s.view, *g, table=table, interleaved=inter)
    place = np.concatenate([np.arange(m - c, m) for c, m in zip(n, lens)]).astype(np.int64)
    want, mag = A.turn(_np(q), _np(g[0]), 1e-6, _np(table), place, inter)
    assert got.dtype == torch.bfloat16
    _close(_np(got), want, DELTA * mag + STEP["bf16"] * np.abs(want))
    kk = A.turn(_np(k), _np(g[1]), 1e-6, _np(table), place, inter)[0]
    _same_cache(_np(s.cache), _append_expected(s, kv, kk, _np(v)))
    # read back: the values of the same tokens
    for dt in (torch.float32, torch.bfloat16):
        rk, rv = B.oq_kv4_read(kv, *s.view, s.T, dtype=dt)
        ck, cv = A.cache_values(_np(s.cache))
        for b in range(len(n)):
            wk, wv, _ = A.sequence(ck, cv, s.pages[b], lens[b], KH, D)
            lo, hi = s.np_cu[b], s.np_cu[b + 1]
            assert np.array_equal(_np(rk)[lo:hi], wk[lens[b] - n[b]:]) and np.array_equal(_np(rv)[lo:hi], wv[lens[b] - n[b]:])


def test_append_many_tokens_of_many_heads(env):
    """Several groups of channels a CTA, windows at every place of a page."""
    torch, B = env
    rng = np.random.default_rng(32)
    kv = B.oq_kv4_create(8, 8, 128)
    s = Streams(torch, rng, kv, [1500, 77], [1713, 300])
    x = _heads(torch, rng, s.T, 24, 128, "bf16")
    q, k, v = x[:, :8], x[:, 8:16], x[:, 16:]
    table = _table(torch, rng, 1713, 128)
    got = B.oq_kv4_append(kv, q, k, v, *s.view, table=table)
    place = np.concatenate([np.arange(m - c, m) for c, m in zip(s.n, s.lens)]).astype(np.int64)
    want, mag = A.turn(_np(q), None, 1e-6, _np(table), place)
    _close(_np(got), want, DELTA * mag + STEP["bf16"] * np.abs(want))
    _same_cache(_np(s.cache), _append_expected(s, kv, A.turn(_np(k), None, 1e-6, _np(table), place)[0], _np(v)))


@pytest.mark.parametrize("norm,rot", [(False, 0), (True, 0), (False, 64), (True, 64)])
def test_append_forms(env, norm, rot):
    """Without norm, rotation or queries; positions given; q in place."""
    torch, B = env
    rng = np.random.default_rng(7)
    kv = B.oq_kv4_create(2, 2, 128)
    s = Streams(torch, rng, kv, [3, 40], [200, 41])
    q, k, v = (_heads(torch, rng, s.T, 2, 128, "bf16") for _ in range(3))
    q, k = q.contiguous(), k.contiguous()
    table = _table(torch, rng, 60, rot) if rot else None
    pos = torch.from_numpy(rng.integers(0, 60, s.T).astype(np.int32)).cuda() if rot else None
    kw = dict(table=table, positions=pos, norm=norm)
    tk = dict(table=None if table is None else _np(table), pos=None if pos is None else _np(pos), norm=norm)
    want, mag = A.turn(_np(q), **tk)
    assert B.oq_kv4_append(kv, None, k, v, *s.view, **kw) is None
    first = s.cache.clone()
    _same_cache(_np(first), _append_expected(s, kv, A.turn(_np(k), **tk)[0], _np(v)))
    r = B.oq_kv4_append(kv, q, k, v, *s.view, q_out=q, **kw)
    assert r is q and torch.equal(first, s.cache)
    _close(_np(q), want, DELTA * mag + STEP["bf16"] * np.abs(want))


def test_append_special_values(env):
    torch, B = env
    rng = np.random.default_rng(8)
    kv = B.oq_kv4_create(1, 1, 128)
    s = Streams(torch, rng, kv, [12], [140])
    x = rng.standard_normal((2, 12, 1, 128)).astype(np.float32)
    x[:, 0] = 0
    x[:, 1, 0, 40] = np.nan
    x[:, 2, 0, 3] = np.inf
    x[:, 3] *= 1e30
    x[:, 4] *= 1e-30
    x[:, 5] = 2.0 ** -140
    x[:, 6, 0, :32] = 0
    x[:, 7] = 3.4e38
    x[:, 8] = np.float32(5.0) * 2.0 ** rng.integers(-3, 3, (2, 1, 128))   # ties
    k, v = (torch.from_numpy(a).cuda() for a in x)
    for norm, gain in ((False, None), (True, np.float32(1.25))):
        g = None if gain is None else torch.full((128,), float(gain), device="cuda")
        B.oq_kv4_append(kv, None, k, v, *s.view, k_gain=g, norm=norm, eps=1e-6)
        kk = A.turn(_np(k), gain, 1e-6, norm=norm)[0]
        _same_cache(_np(s.cache), _append_expected(s, kv, kk, _np(v)))


def test_append_skips_what_has_no_place(env):
    torch, B = env
    rng = np.random.default_rng(9)
    kv = B.oq_kv4_create(2, 2, 64)
    s = Streams(torch, rng, kv, [4, 5, 2, 3], [130, 3, 400, 260])
    s.table[0, 1] = -1                      # sequence 0: tokens 128, 129 have no page
    s.table[3] = torch.tensor([0, 1 << 30, 2, 7], device="cuda", dtype=torch.int32)[: s.table.shape[1]]
    table = s.table[:, :3].contiguous()     # sequence 2: tokens 398, 399 lie behind the table
    k, v = (_heads(torch, rng, s.T, 2, 64, "bf16") for _ in range(2))
    s.pages = _np(table)
    B.oq_kv4_append(kv, None, k, v, s.cache, table, s.cu, s.len, norm=False)
    want = s.np_cache.copy()
    for i in (0, 1):                        # tokens 126, 127; sequence 1 has fewer tokens than the call
        A.write_token(want, s.pages[0, 0], 126 + i, _np(k)[i].ravel(), _np(v)[i].ravel())
    for i in range(3):
        A.write_token(want, s.pages[3, 2], 1 + i, _np(k)[11 + i].ravel(), _np(v)[11 + i].ravel())
    _same_cache(_np(s.cache), want)
    rk, rv = B.oq_kv4_read(kv, s.cache, table, s.cu, s.len, s.T, k=torch.full((s.T, 2, 64), 7.0, device="cuda"))
    assert torch.isnan(rk[2:4]).all() and torch.isnan(rv[2:4]).all() and not torch.isnan(rk[:2]).any()
    assert (rk[4:11] == 7).all()


# ------------------------------------------------------------------ attention
def _check_attention(torch, B, kv, s, q, scale=None, causal=True, window=0, max_q=None, max_len=0, **kw):
    scale = kv.head_dim ** -0.5 if scale is None else scale
    y = B.oq_kv4_attention(kv, q, *s.view, max_q or max(max(s.n), 1), max_len=max_len, scale=scale, causal=causal, window=window, **kw)
    B.oq_kv4_poll_error(kv)
    ck, cv = A.cache_values(_np(s.cache))
    got, pages = _np(y), _np(s.table)
    for b, (n, m) in enumerate(zip(s.n, s.lens)):
        if n:
            K, V, ok = A.sequence(ck, cv, pages[b], m, kv.kv_heads, kv.head_dim)
            lo, hi = s.np_cu[b], s.np_cu[b + 1]
            want, tol = A.attention(_np(q)[lo:hi], K, V, ok, np.float32(scale).astype(np.float64), causal, window)
            _close(got[lo:hi], want, tol, b)
    return y


def _queries(torch, rng, T, H, D):
    return _heads(torch, rng, T, H, D, "bf16", extra=1)


DECODE = [([1], [1]), ([1, 1, 1], [127, 128, 129]), ([1, 0, 1, 1], [300, 70, 0, 1025]), ([1], [5000])]


@pytest.mark.parametrize("H,KH,D", [(1, 1, 128), (4, 4, 64), (8, 2, 128), (5, 1, 64), (6, 3, 64), (24, 1, 128), (32, 2, 64),
                                    (80, 2, 128)])
@pytest.mark.parametrize("n,lens", DECODE)
def test_attention_one_token(env, H, KH, D, n, lens):
    torch, B = env
    rng = np.random.default_rng(sum(lens) * 7 + H)
    kv = B.oq_kv4_create(H, KH, D)
    s = Streams(torch, rng, kv, n, lens)
    _check_attention(torch, B, kv, s, _queries(torch, rng, s.T, H, D))


CHUNKS = [([7, 1, 40], [7, 300, 200], True, 0), ([33, 5], [33, 700], False, 0), ([64, 3], [500, 129], True, 50),
          ([9, 130], [400, 257], False, 1), ([20, 3], [5, 0], True, 0), ([17], [2000], True, 600), ([5, 4], [900, 128], True, 1)]


@pytest.mark.parametrize("H,KH,D", [(2, 2, 128), (3, 3, 64), (10, 2, 128), (8, 1, 64)])
@pytest.mark.parametrize("n,lens,causal,window", CHUNKS)
def test_attention_chunks(env, H, KH, D, n, lens, causal, window):
    """Several tokens a sequence, some of them (more tokens than the cache has) seeing nothing."""
    torch, B = env
    rng = np.random.default_rng(sum(lens) + sum(n) + H)
    kv = B.oq_kv4_create(H, KH, D)
    s = Streams(torch, rng, kv, n, lens)
    y = _check_attention(torch, B, kv, s, _queries(torch, rng, s.T, H, D), causal=causal, window=window)
    if lens[0] == 5:
        assert (y[:15] == 0).all() and (y[20:] == 0).all()


@pytest.mark.parametrize("D,H,KH,n", [(128, 2, 1, 2), (64, 16, 2, 2), (128, 2, 1, 70), (64, 16, 2, 35)])
@pytest.mark.parametrize("scale", [1e-6, 0.5, 4.0, 60.0])
def test_attention_far_scores(env, D, H, KH, n, scale):
    """Scores that grow along the cache (the running reference moves again and again), and flat ones."""
    torch, B = env
    rng = np.random.default_rng(11)
    kv = B.oq_kv4_create(H, KH, D)
    s = Streams(torch, rng, kv, [n, 1], [1400, 600])
    grow = np.linspace(0.0, 3.0, 1400)[:, None, None]
    for b, m in enumerate(s.lens):
        for j in range(m):
            A.write_token(s.np_cache, s.pages[b, j // 128], j % 128, (grow[j] + 0.1 * rng.standard_normal((KH, D))).ravel(),
                          rng.standard_normal((KH, D)).ravel() * 2.0 ** rng.integers(-6, 7))
    s.cache.copy_(torch.from_numpy(s.np_cache))
    q = torch.from_numpy(np.abs(rng.standard_normal((s.T, H, D))).astype(np.float32)).cuda().bfloat16()
    _check_attention(torch, B, kv, s, q, scale=scale / D ** 0.5)
    _check_attention(torch, B, kv, s, -q, scale=scale / D ** 0.5)


def test_attention_scales_of_v(env):
    """V from 2^-90 to 2^90 in one cache, sequences apart."""
    torch, B = env
    rng = np.random.default_rng(12)
    kv = B.oq_kv4_create(2, 1, 128)
    s = Streams(torch, rng, kv, [1, 1, 1], [200, 200, 200])
    for b, e in enumerate((-90, 0, 88)):
        for j in range(200):
            A.write_token(s.np_cache, s.pages[b, j // 128], j % 128, rng.standard_normal(128), rng.standard_normal(128) * 2.0 ** e)
    s.cache.copy_(torch.from_numpy(s.np_cache))
    _check_attention(torch, B, kv, s, _queries(torch, rng, 3, 2, 128))


@pytest.mark.parametrize("D,KH", [(128, 1), (64, 2)])
def test_attention_nan_and_garbage_in_chunks(env, D, KH):
    """The same for many queries: tokens 120 to 199 and 30 to 89 of two sequences are the call's."""
    torch, B = env
    rng = np.random.default_rng(33)
    kv = B.oq_kv4_create(2 * KH, KH, D)
    s = Streams(torch, rng, kv, [80, 60], [200, 90])
    c, p = s.np_cache, s.pages
    rows = c[:, :, 256:].reshape(c.shape[0], kv.groups, 1024)
    rows[p[1, 0], :, 512 + 95 * 4:] = 255
    rows[s.free] = 255
    rows[p[0, 1], :, 512 + (150 - 128) * 4 + 1] = 255          # a value block of token 150
    rows[p[1, 0], :, 85 % 32 * 16 + 85 // 32 * 4] = 255        # a key block of token 85
    c[:, :, 256:] = rows.reshape(c.shape[0], kv.groups, 16, 64)
    s.cache.copy_(torch.from_numpy(c))
    y = _np(_check_attention(torch, B, kv, s, _queries(torch, rng, s.T, 2 * KH, D)))
    assert not np.isnan(y[:30]).any() and np.isnan(y[30:80]).any() and not np.isnan(y[30:80]).all()
    assert not np.isnan(y[80:135]).any() and np.isnan(y[135:]).any()


@pytest.mark.parametrize("D", [64, 128])
def test_attention_chunks_split(env, D):
    """Few tiles of queries over a long cache: parts, joined; and special queries."""
    torch, B = env
    rng = np.random.default_rng(34)
    kv = B.oq_kv4_create(3, 1, D)
    s = Streams(torch, rng, kv, [90, 20], [4000, 2500])
    q = _queries(torch, rng, s.T, 3, D)
    a = _check_attention(torch, B, kv, s, q)
    assert B.oq_kv4_attention_workspace_size(kv, s.T, 2, 90, 4000) > 0
    assert torch.equal(a, B.oq_kv4_attention(kv, q, *s.view, 90))
    _check_attention(torch, B, kv, s, q, max_len=1)
    _check_attention(torch, B, kv, s, q, causal=False, window=300)
    z = q.clone()
    z[5, 1, 3], z[70, 2, 9] = float("inf"), float("nan")
    y = B.oq_kv4_attention(kv, z, *s.view, 90)
    assert torch.isnan(y[5, 1]).all() and torch.isnan(y[70, 2]).all()
    y[5, 1], y[70, 2] = a[5, 1], a[70, 2]
    assert torch.equal(a, y)


def test_attention_many_parts(env):
    """64 parts of a cache."""
    torch, B = env
    rng = np.random.default_rng(35)
    for D in (64, 128):
        kv = B.oq_kv4_create(1, 1, D)
        s = Streams(torch, rng, kv, [1], [8300])
        _check_attention(torch, B, kv, s, _queries(torch, rng, 1, 1, D))


@pytest.mark.parametrize("D,KH", [(128, 1), (64, 2)])
def test_attention_nan_and_garbage(env, D, KH):
    """What no query sees may hold anything; what is seen and NaN reaches the queries that see it, V's in its block of
    32 channels."""
    torch, B = env
    rng = np.random.default_rng(13)
    kv = B.oq_kv4_create(2 * KH, KH, D)
    s = Streams(torch, rng, kv, [6, 3, 4], [200, 70, 90])
    c = s.np_cache
    rows = c[:, :, 256:].reshape(c.shape[0], kv.groups, 1024)
    p = s.pages
    # behind the last token of sequence 1, and pages of nobody
    rows[p[1, 0], :, 512 + 75 * 4:] = 255
    rows[p[1, 0], :, 100 % 32 * 16 + 100 // 32 * 4] = 255
    rows[s.free] = 255
    # sequence 0: a key that the first queries do not see; sequence 2: a value block
    j = 197
    rows[p[0, 1], :, (j % 128) % 32 * 16 + (j % 128) // 32 * 4 + 1] = 255
    rows[p[2, 0], :, 512 + 88 * 4 + 2] = 255
    c[:, :, 256:] = rows.reshape(c.shape[0], kv.groups, 16, 64)
    s.cache.copy_(torch.from_numpy(c))
    y = _np(_check_attention(torch, B, kv, s, _queries(torch, rng, s.T, 2 * KH, D)))
    assert np.isnan(y[3:6]).any() and not np.isnan(y[:3]).any() and not np.isnan(y[6:9]).any()
    assert not np.isnan(y[9:11]).any() and np.isnan(y[11:]).any() and not np.isnan(y[11:]).all()


def test_attention_nan_and_infinite_queries(env):
    torch, B = env
    rng = np.random.default_rng(14)
    kv = B.oq_kv4_create(4, 1, 128)
    s = Streams(torch, rng, kv, [2], [150])
    q = _queries(torch, rng, 2, 4, 128)
    q[0, 1, 3], q[1, 2, 100], q[0, 2] = float("nan"), float("inf"), 0
    q[1, 0] = q[1, 0] * 2.0 ** -120
    y = B.oq_kv4_attention(kv, q, *s.view, 2)
    assert torch.isnan(y[0, 1]).all() and torch.isnan(y[1, 2]).all()
    good = q.clone()
    good[0, 1], good[1, 2] = 0, 0
    z = _check_attention(torch, B, kv, s, good)
    for t, h in ((0, 0), (0, 2), (0, 3), (1, 0), (1, 1), (1, 3)):
        assert torch.equal(y[t, h], z[t, h])


def test_attention_pages_that_are_not_there(env):
    torch, B = env
    rng = np.random.default_rng(15)
    kv = B.oq_kv4_create(4, 2, 128)
    s = Streams(torch, rng, kv, [1, 3, 2], [700, 300, 256])
    s.table[0, 2], s.table[1, 0], s.table[2] = -7, s.cache.shape[0], 1 << 30
    y = _check_attention(torch, B, kv, s, _queries(torch, rng, s.T, 4, 128), causal=False)
    assert (y[4:] == 0).all()
    # more tokens than the table holds: the sequence ends there
    short = s.table[:, :2].contiguous()
    q = _queries(torch, rng, s.T, 4, 128)
    a = B.oq_kv4_attention(kv, q, s.cache, short, s.cu, s.len, 3, causal=False)
    b = B.oq_kv4_attention(kv, q, s.cache, short, s.cu, s.len.clamp(max=256), 3, causal=False)
    assert torch.equal(a[:1], b[:1])


def test_attention_leaves_other_rows_alone(env):
    """Rows before the first sequence, behind the last, past max_q; split and not."""
    torch, B = env
    rng = np.random.default_rng(16)
    kv = B.oq_kv4_create(2, 2, 64)
    s = Streams(torch, rng, kv, [2, 3], [3000, 2000])
    q = _queries(torch, rng, 9, 2, 64)
    cu = s.cu + 1
    for max_len in (1, 3000):
        y = torch.full((9, 2, 64), 3.0, device="cuda", dtype=torch.bfloat16)
        B.oq_kv4_attention(kv, q, s.cache, s.table, cu, s.len, 2, max_len=max_len, y=y)
        assert (y[0] == 3).all() and (y[5:] == 3).all() and not (y[1:5] == 3).all()
    # a sequence that reaches behind q has no output at all
    y.fill_(3.0)
    B.oq_kv4_attention(kv, q[:5], s.cache, s.table, cu, s.len, 3, max_len=1, y=y[:5])
    assert (y[3:] == 3).all()


def test_attention_split_and_repeat(env):
    """The same bits on every call; another split only rounds differently."""
    torch, B = env
    rng = np.random.default_rng(17)
    kv = B.oq_kv4_create(8, 2, 128)
    s = Streams(torch, rng, kv, [1, 2], [3000, 1111])
    q = _queries(torch, rng, 3, 8, 128)
    a = _check_attention(torch, B, kv, s, q)
    assert B.oq_kv4_attention_workspace_size(kv, 3, 2, 2, 3000) > 0
    for _ in range(3):
        assert torch.equal(a, B.oq_kv4_attention(kv, q, *s.view, 2))
    _check_attention(torch, B, kv, s, q, max_len=1)
    _check_attention(torch, B, kv, s, q, max_len=600)


def test_attention_far_in_a_large_cache(env):
    """Pages whose bytes lie past 2^32, and the table's entry for them."""
    torch, B = env
    rng = np.random.default_rng(18)
    kv = B.oq_kv4_create(2, 2, 128)
    s = Streams(torch, rng, kv, [2], [200])
    pages = 130000                          # 4.5 GB
    big = torch.empty((pages, kv.groups, 272, 64), dtype=torch.uint8, device="cuda")
    where = [pages - 1, pages - 3]
    for i, p in enumerate(where):
        big[p] = s.cache[s.pages[0, i]]
    table = torch.tensor([where], dtype=torch.int32, device="cuda")
    q = _queries(torch, rng, 2, 2, 128)
    want = B.oq_kv4_attention(kv, q, *s.view, 2)
    assert torch.equal(want, B.oq_kv4_attention(kv, q, big, table, s.cu, s.len, 2))
    k, v = (_heads(torch, rng, 2, 2, 128, "bf16") for _ in range(2))
    B.oq_kv4_append(kv, None, k, v, *s.view)
    B.oq_kv4_append(kv, None, k, v, big, table, s.cu, s.len)
    for i, p in enumerate(where):
        assert torch.equal(big[p], s.cache[s.pages[0, i]])
    for a, b in zip(B.oq_kv4_read(kv, *s.view, 2), B.oq_kv4_read(kv, big, table, s.cu, s.len, 2)):
        assert torch.equal(a, b)


def test_attention_empty_calls(env):
    torch, B = env
    kv = B.oq_kv4_create(2, 1, 128)
    cache = kv.cache(1)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.zeros(0, 2, 128, device="cuda", dtype=torch.bfloat16)
    assert B.oq_kv4_attention(kv, q, cache, none.view(0, 4), one, none, 0).shape == (0, 2, 128)
    assert B.oq_kv4_append(kv, q, q[:, :1], q[:, :1], cache, none.view(0, 4), one, none).shape == (0, 2, 128)
    # a table without pages: nothing is seen
    q = torch.ones(1, 2, 128, device="cuda", dtype=torch.bfloat16)
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    y = B.oq_kv4_attention(kv, q, cache, torch.zeros(1, 0, dtype=torch.int32, device="cuda"), cu, one + 5, 1)
    assert (y == 0).all()
    a, b = B.oq_qk_norm_rope(q[:0], q[:0, :1])
    assert a.shape == (0, 2, 128) and b.shape == (0, 1, 128)


# ------------------------------------------------------------------ 4-bit weights with group scales
def _weights(rng, N, d):
    w = rng.standard_normal((N, d)) * 0.05 * np.exp(rng.standard_normal((N, 1)))
    return w.astype(np.float32)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("N,d,group", [(1, 32, 32), (17, 160, 32), (40, 192, 64), (16, 1152, 128), (333, 2016, 32)])
def test_w4g_prepare(env, dtype, zeros, N, d, group):
    torch, B = env
    W = _weights(np.random.default_rng(N + d), N, d)
    W[0, :group] = 0
    if N > 3:
        W[1, 5], W[2, 7] = np.inf, np.nan
        W[3, :group] = 1e-41
        W[3, -group:] = np.abs(W[3, -group:])
    t = torch.from_numpy(W).cuda().to(_dt(torch, dtype))
    c, s, z = B.oq_w4g_prepare(t, group, zeros=zeros)
    wc, ws, wz = A.w4g_prepare(t.float().cpu().numpy(), group, zeros)
    assert np.array_equal(s.float().cpu().numpy(), ws, equal_nan=True)
    assert np.array_equal(A.w4g_unpack(_np(c), d), wc)
    assert (z is None) == (not zeros) and (z is None or np.array_equal(_np(z), wz))


def _check_w4g(torch, B, x, c, s, z, d, group, y_dtype):
    y = B.oq_linear_w4g(x, c, s, z, group=group, y_dtype=y_dtype)
    w = A.w4g_values(_np(c), _np(s), None if z is None else _np(z), d, group)
    with np.errstate(all="ignore"):
        want, mags = _np(x) @ w.T, np.abs(_np(x)) @ np.abs(w).T
    tol = (8 + d / group / 8 + 26) * 2.0 ** -23 * np.nan_to_num(mags) + (2.0 ** -8 * np.abs(np.nan_to_num(want)) if y_dtype == torch.bfloat16 else 0)
    _close(_np(y), want, tol)
    return y


@pytest.mark.parametrize("x_dtype,y_dtype", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("T,N,d,group,zeros", [
    (1, 1, 32, 32, False), (1, 5120, 1152, 128, False), (2, 17, 160, 32, True), (3, 130, 4096, 64, True), (8, 33, 96, 32, False),
    (9, 48, 192, 64, False), (13, 512, 5120, 32, True), (16, 16, 13824, 128, True), (17, 100, 640, 128, False),
    (32, 64, 1024, 64, False), (33, 40, 256, 32, True), (70, 50, 384, 128, True), (11, 24, 128, 64, True)])
def test_w4g_linear(env, x_dtype, y_dtype, T, N, d, group, zeros):
    torch, B = env
    rng = np.random.default_rng(T + N + d)
    c, s, z = B.oq_w4g_prepare(torch.from_numpy(_weights(rng, N, d)).cuda(), group, zeros=zeros)
    x = torch.from_numpy((rng.standard_normal((T, d)) * np.exp(rng.standard_normal((T, d)))).astype(np.float32)).cuda()
    x = x.to(_dt(torch, x_dtype))
    y = _check_w4g(torch, B, x, c, s, z, d, group, _dt(torch, y_dtype))
    assert torch.equal(y, B.oq_linear_w4g(x, c, s, z, group=group, y_dtype=_dt(torch, y_dtype)))


@pytest.mark.parametrize("x_dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,N,d,group,zeros", [
    (1, 7301, 160, 32, True), (8, 7500, 1088, 64, False), (2, 14400, 384, 128, True),    # rows in more than one round of CTAs
    (1, 3601, 8320, 64, True), (7, 4000, 8224, 32, False), (2, 3700, 9216, 128, True),   # long rows, split
    (13, 4801, 416, 32, True), (16, 4736, 2176, 64, False), (31, 4750, 672, 32, True)])  # 32 rows a CTA
def test_w4g_linear_many_rows(env, x_dtype, T, N, d, group, zeros):
    torch, B = env
    rng = np.random.default_rng(T * N + d)
    c, s, z = B.oq_w4g_prepare(torch.from_numpy(_weights(rng, N, d)).cuda(), group, zeros=zeros)
    x = torch.from_numpy((rng.standard_normal((T, d)) * np.exp(rng.standard_normal((T, d)))).astype(np.float32)).cuda()
    _check_w4g(torch, B, x.to(_dt(torch, x_dtype)), c, s, z, d, group, torch.float32)


def test_w4g_linear_exact_and_special(env):
    """fp32 tokens enter exactly; infinities and NaN go where the formula says."""
    torch, B = env
    rng = np.random.default_rng(20)
    N, d = 32, 256
    c, s, z = B.oq_w4g_prepare(torch.from_numpy(_weights(rng, N, d)).cuda(), 32, zeros=True)
    s.fill_(1.0)
    x = torch.zeros(4, d, device="cuda")
    x[0, 100] = 1 + 2.0 ** -23
    x[1, 5] = 3.4028234663852886e38 / 16
    x[2, 7] = 2.0 ** -100 * (1 + 2.0 ** -20)
    w = A.w4g_values(_np(c), _np(s), _np(z), d, 32)
    y = B.oq_linear_w4g(x, c, s, z, group=32)
    assert np.array_equal(_np(y), (_np(x) @ w.T).astype(np.float32).astype(np.float64))
    x[3, 9] = float("inf")
    x[0, 3] = float("nan")
    s[5, 2] = float("nan")
    for t in (x, x.bfloat16()):
        y = _np(B.oq_linear_w4g(t, c, s, z, group=32))
        assert np.isnan(y[0]).all() and np.isnan(y[:, 5]).all() and not np.isnan(y[1:3, :5]).any()
        with np.errstate(invalid="ignore"):
            want = np.where(w[:, 9] == 0, np.nan, np.inf * np.sign(w[:, 9]))
        keep = np.arange(N) != 5
        assert np.array_equal(y[3][keep], want[keep], equal_nan=True)


# ------------------------------------------------------------------ together
def _stage_checks(torch, B, kv, s, x, w1, w2, gains, table, group, parts):
    H, KH, D = kv.heads, kv.kv_heads, kv.head_dim
    qkv, q, o, y = parts
    _close(_np(qkv).reshape(s.T, -1), *_product(x, w1, group))
    place = np.concatenate([np.arange(m - c, m) for c, m in zip(s.n, s.lens)]).astype(np.int64)
    want, mag = A.turn(_np(qkv)[:, :H], _np(gains[0]), 1e-6, _np(table), place)
    _close(_np(q), want, DELTA * mag + STEP["bf16"] * np.abs(want))
    kk = A.turn(_np(qkv)[:, H:H + KH], _np(gains[1]), 1e-6, _np(table), place)[0]
    _same_cache(_np(s.cache), _append_expected(s, kv, kk, _np(qkv)[:, H + KH:]))
    _check_attention(torch, B, kv, s, q, y=o)
    _close(_np(y), *_product(o.view(s.T, -1), w2, group))


def _product(x, w, group):
    c, s, z = w
    d = x.shape[1]
    v = A.w4g_values(_np(c), _np(s), None if z is None else _np(z), d, group)
    want = _np(x) @ v.T
    return want, (34 + d / group / 8) * 2.0 ** -23 * (np.abs(_np(x)) @ np.abs(v).T) + 2.0 ** -8 * np.abs(want)


@pytest.mark.parametrize("H,KH,D", [(4, 2, 128), (6, 3, 64)])
def test_a_step_of_streams(env, H, KH, D):
    """Projection, norm with rotation and append, attention, projection; each against the reference on what came before,
    then the same replayed from a graph with other inputs and lengths, on another stream."""
    torch, B = env
    rng = np.random.default_rng(21)
    kv = B.oq_kv4_create(H, KH, D)
    s = Streams(torch, rng, kv, [1, 1, 1], [130, 257, 5])
    d = H * D
    w1 = B.oq_w4g_prepare(torch.from_numpy(_weights(rng, (H + 2 * KH) * D, d)).cuda(), 64)
    w2 = B.oq_w4g_prepare(torch.from_numpy(_weights(rng, d, d)).cuda(), 64, zeros=True)
    gains = [torch.from_numpy(rng.uniform(0.5, 2, D).astype(np.float32)).cuda() for _ in range(2)]
    table = _table(torch, rng, 300, D)
    x = torch.from_numpy(rng.standard_normal((3, d)).astype(np.float32)).cuda().bfloat16()

    def step():
        qkv = B.oq_linear_w4g(x, *w1, group=64, y_dtype=torch.bfloat16).view(3, H + 2 * KH, D)
        q = B.oq_kv4_append(kv, qkv[:, :H], qkv[:, H:H + KH], qkv[:, H + KH:], *s.view, *gains, table=table)
        o = B.oq_kv4_attention(kv, q, *s.view, 1, max_len=300)
        return qkv, q, o, B.oq_linear_w4g(o.view(3, -1), *w2, group=64, y_dtype=torch.bfloat16)

    _stage_checks(torch, B, kv, s, x, w1, w2, gains, table, 64, step())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step()
    with torch.cuda.graph(graph, stream=side):
        parts = step()
    for _ in range(3):
        s.np_cache = _np(s.cache)
        s.lens = [m + 1 for m in s.lens]
        s.len += 1
        x.copy_(torch.from_numpy(rng.standard_normal((3, d)).astype(np.float32)))
        graph.replay()
        torch.cuda.synchronize()
        _stage_checks(torch, B, kv, s, x, w1, w2, gains, table, 64, parts)


def test_calls_on_two_streams(env):
    """One handle, two streams, two workspaces: the results of calls alone."""
    torch, B = env
    rng = np.random.default_rng(22)
    kv = B.oq_kv4_create(8, 2, 128)
    s = [Streams(torch, rng, kv, [1, 3], [2000, 900]) for _ in range(2)]
    q = [_queries(torch, rng, 4, 8, 128) for _ in range(2)]
    want = [B.oq_kv4_attention(kv, a, *b.view, 3) for a, b in zip(q, s)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(B.oq_kv4_attention(kv, q[i], *s[i].view, 3))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(want[i], g) for g in got[i])
    B.oq_kv4_poll_error(kv)


def test_refusals_leave_outputs_alone(env):
    """Arguments that the library refuses; nothing is written."""
    torch, B = env
    rng = np.random.default_rng(23)
    kv = B.oq_kv4_create(8, 2, 128)
    s = Streams(torch, rng, kv, [1], [3000])
    q = _queries(torch, rng, 1, 8, 128)
    y = torch.full((1, 8, 128), 3.0, device="cuda", dtype=torch.bfloat16)
    need = B.oq_kv4_attention_workspace_size(kv, 1, 1, 1, 3000)
    assert need > 0
    small = torch.empty(need - 256, dtype=torch.uint8, device="cuda")
    with pytest.raises(B.OrbitQuantError, match="workspace"):
        B.oq_kv4_attention(kv, q, *s.view, 1, max_len=3000, y=y, workspace=small)
    for kw in (dict(scale=0.0), dict(scale=float("nan")), dict(scale=-1.0), dict(window=-1)):
        with pytest.raises(B.OrbitQuantError):
            B.oq_kv4_attention(kv, q, *s.view, 1, y=y, **kw)
    with pytest.raises(B.OrbitQuantError, match="overlap"):
        B.oq_kv4_attention(kv, y, *s.view, 1, y=y)
    with pytest.raises(ValueError):
        B.oq_kv4_attention(kv, q.float(), *s.view, 1, y=y)
    with pytest.raises(ValueError):
        B.oq_kv4_attention(kv, q, s.cache, s.table, s.cu.long(), s.len, 1, y=y)
    before = s.cache.clone()
    k = _heads(torch, rng, 1, 2, 128, "bf16")
    with pytest.raises(B.OrbitQuantError, match="gains"):
        B.oq_kv4_append(kv, None, k, k, *s.view, k_gain=torch.ones(128, device="cuda"), norm=False)
    with pytest.raises(B.OrbitQuantError):
        B.oq_kv4_append(kv, None, k, k, *s.view, eps=-1.0)
    with pytest.raises(B.OrbitQuantError):
        B.oq_kv4_append(kv, None, k, k, *s.view, table=torch.zeros(4, 12, 2, device="cuda"))
    with pytest.raises(ValueError):
        B.oq_kv4_append(kv, None, k, k.float(), *s.view)
    x = torch.zeros(4, 6, 64, device="cuda")
    with pytest.raises(B.OrbitQuantError, match="overlap"):
        B.oq_qk_norm_rope(x[:, :3], x[:, 3:], q_out=x[:, 1:4], k_out=torch.empty(4, 3, 64, device="cuda"))
    with pytest.raises(ValueError):
        B.oq_qk_norm_rope(x.transpose(0, 1))
    torch.cuda.synchronize()
    assert (y == 3).all() and torch.equal(before, s.cache)
