"""GPU tests of attention and the operators beside it where arithmetic or a mask has a border, against the plain fp64
reference (attention_reference.py, whose bounds they take).  Needs a B200."""

import numpy as np
import pytest

import attention_reference as A
import softmax_emulation as S
from test_attention_ops import Streams, _check_attention, _np, env  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


def _ones_at(s, D, places):
    """Keys of zeros but for ones: {token: channels}, in every sequence; random values."""
    rng = np.random.default_rng(0)
    for b, m in enumerate(s.lens):
        for j in range(m):
            k = np.zeros(D)
            k[places.get(j, [])] = 1
            A.write_token(s.np_cache, s.pages[b, j // 128], j % 128, k, rng.standard_normal(D))


@pytest.mark.parametrize("D", [64, 128])
def test_scores_at_the_border_of_a_move(env, D):
    """A second tile's scores exceed the reference by 2^8 and a fraction of a rounding; every query has its own."""
    torch, B = env
    rng = np.random.default_rng(40)
    c2 = S.log2e(D ** -0.5)
    found = [(m, b) for m in range(8, 401) if (b := S.border_score(m, c2)) is not None]
    kv = B.oq_kv4_create(1, 1, D)
    s = Streams(torch, rng, kv, [len(found)], [700])
    _ones_at(s, D, {5: [32, 33, 34], 130: [0, 1, 2], 333: [0, 1]})
    s.cache.copy_(torch.from_numpy(s.np_cache))
    q = np.zeros((len(found), 1, D), np.float32)
    for i, (m, b) in enumerate(found):
        q[i, 0, :3] = S.parts3(b)
        q[i, 0, 32:35] = S.parts3(np.float32((m - 0.5) / c2))
    q = torch.from_numpy(q).cuda().bfloat16()
    for _ in range(3):
        _check_attention(torch, B, kv, s, q, causal=False)
    for r in (2, 47, 48, 129):      # a few queries a key head, and many
        s.n = [r]
        s.np_cu = np.array([0, r], np.int32)
        s.cu.copy_(torch.from_numpy(s.np_cu))
        _check_attention(torch, B, kv, s, q[:r].contiguous(), causal=False)


FAR = [2.0 ** 20, 2.0 ** 25, 2.0 ** 28 * 1.37, 2.0 ** 31 * 1.11, 2.0 ** 34 * 1.73, 2.0 ** 60 * 1.01, 2.0 ** 95 * 1.9]


def _far(env, D, n, far):
    """Keys of one channel times queries of magnitude `far`, each query its own: the tokens with the largest score share
    the weight and all others have none; a query that sees one token gives its value.  Weights that are equal are rounded
    alike, to 8 bits; the result is rounded to bf16; sums of few terms."""
    torch, B = env
    rng = np.random.default_rng(41)
    kv = B.oq_kv4_create(1, 1, D)
    s = Streams(torch, rng, kv, [n], [400])
    q = np.zeros((n, 1, D))
    q[:, 0, 7] = far * rng.uniform(1, 2, n) * rng.choice([-1, 1], n)
    q = torch.from_numpy(q.astype(np.float32)).cuda().bfloat16()

    def values(key):
        for j in range(400):
            k = np.zeros(D)
            k[7] = key(j)
            A.write_token(s.np_cache, s.pages[0, j // 128], j % 128, k, rng.standard_normal(D))
        s.cache.copy_(torch.from_numpy(s.np_cache))
        V = A.cache_values(s.np_cache)[1]
        return np.stack([V[s.pages[0, j // 128], 0, j % 128, :D] for j in range(400)])

    def check(y, want, V):
        assert (np.abs(_np(y)[:, 0] - want) <= 2 * 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * np.abs(V).max()).all()

    V = values(lambda j: {3: 1, 140: 1, 141: 0.5, 300: 1, 350: -1}.get(j, 0))
    up = _np(q)[:, 0, 7:8] > 0
    check(B.oq_kv4_attention(kv, q, *s.view, n, causal=False), np.where(up, (V[3] + V[140] + V[300]) / 3, V[350]), V)
    V = values(lambda j: 1 - j % 2 * 0.5)
    check(B.oq_kv4_attention(kv, q, *s.view, n, window=1), V[400 - n:], V)
    B.oq_kv4_poll_error(kv)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("far", FAR)
def test_far_scores_of_chunks(env, D, far):
    _far(env, D, 60, far)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 3, 7, 20, 47])
@pytest.mark.parametrize("far", FAR)
def test_far_scores_of_few_queries(env, D, n, far):
    _far(env, D, n, far)


@pytest.mark.parametrize("D,H,KH", [(128, 2, 1), (128, 4, 4), (64, 8, 2), (64, 3, 3), (128, 12, 1), (64, 20, 1)])
@pytest.mark.parametrize("n", [1, 3])
def test_hidden_values_do_not_count(env, D, H, KH, n):
    """A window's border inside 32 tokens, and the causal one: values that no query sees are 2^20 times larger, and the
    result is as exact as without them."""
    torch, B = env
    rng = np.random.default_rng(42)
    kv = B.oq_kv4_create(H, KH, D)
    lens, window = [270, 413, 50], 75
    s = Streams(torch, rng, kv, [n] * 3, lens)
    for b, m in enumerate(lens):
        for j in range(128 * s.pages.shape[1]):
            if s.pages[b, j // 128] < len(s.np_cache):
                big = j >= m or j < m - n - window + 1
                A.write_token(s.np_cache, s.pages[b, j // 128], j % 128, rng.standard_normal(KH * D),
                              rng.standard_normal(KH * D) * (2.0 ** 20 if big else 1))
    s.cache.copy_(torch.from_numpy(s.np_cache))
    q = torch.from_numpy(rng.standard_normal((s.T, H, D)).astype(np.float32)).cuda().bfloat16()
    _check_attention(torch, B, kv, s, q, window=window)
    # fewer queries than columns, the call's tokens among them larger than all: only the last token sees its own
    for b, m in enumerate(lens):
        A.write_token(s.np_cache, s.pages[b, (m - 1) // 128], (m - 1) % 128, rng.standard_normal(KH * D),
                      rng.standard_normal(KH * D) * 2.0 ** 20)
    s.cache.copy_(torch.from_numpy(s.np_cache))
    y = _np(B.oq_kv4_attention(kv, q, *s.view, max(n - 1, 1), window=window))
    ck, cv = A.cache_values(s.np_cache)
    for b, m in enumerate(lens):
        K, V, ok = A.sequence(ck, cv, s.pages[b], m - 1, KH, D)
        if n > 1:
            r = slice(s.np_cu[b], s.np_cu[b + 1] - 1)
            want, tol = A.attention(_np(q)[r], K, V, ok, np.float64(np.float32(D ** -0.5)), True, window)
            assert (np.abs(y[r] - want) <= tol).all()


@pytest.mark.parametrize("n", [2, 60])
def test_a_sequence_behind_the_arrays_has_no_output_in_parts(env, n):
    """Its tokens have no parts to join: what the workspace held before does not become its result."""
    torch, B = env
    rng = np.random.default_rng(43)
    kv = B.oq_kv4_create(1, 1, 128)
    s = Streams(torch, rng, kv, [n, n], [3000, 2000])
    q = torch.from_numpy(rng.standard_normal((2 * n - 1, 1, 128)).astype(np.float32)).cuda().bfloat16()
    need = B.oq_kv4_attention_workspace_size(kv, 2 * n - 1, 2, n, 3000)
    assert need > 0
    w = torch.ones(need // 4, device="cuda")
    y = torch.full((2 * n - 1, 1, 128), 3.0, device="cuda", dtype=torch.bfloat16)
    B.oq_kv4_attention(kv, q, *s.view, n, max_len=3000, y=y, workspace=w)
    assert (y[n:] == 3).all() and not (y[:n] == 3).all()


@pytest.mark.parametrize("D,table,dtype", [(128, True, "bf16"), (64, False, "bf16"), (64, True, "fp32")])
def test_append_leaves_queries_of_no_sequence_alone(env, D, table, dtype):
    """A padded batch: rows before the first sequence and behind the last, in place and not, the sequences' own as in a
    call without them."""
    torch, B = env
    rng = np.random.default_rng(44)
    kv = B.oq_kv4_create(4, 2, D)
    s = Streams(torch, rng, kv, [3, 0, 40], [200, 9, 41])
    T = s.T + 25
    x = torch.from_numpy(rng.standard_normal((T, 8, D)).astype(np.float32)).cuda()
    x = x if dtype == "fp32" else x.bfloat16()
    q, k, v = x[:, :4].contiguous(), x[:, 4:6], x[:, 6:]
    t = torch.from_numpy(rng.standard_normal((250, D // 2, 2)).astype(np.float32)).cuda() if table else None
    pos = torch.from_numpy(rng.integers(0, 250, T).astype(np.int32)).cuda() if table else None
    rows = slice(2, 2 + s.T)
    for p in (None, pos):
        part = B.oq_kv4_append(kv, q[rows], k[rows], v[rows], *s.view, table=t, positions=None if p is None else p[rows].contiguous())
        cache = s.cache.clone()
        outs = [torch.full((T, 4, D), 3.0, device="cuda", dtype=torch.bfloat16)]
        if dtype == "bf16":
            outs.append(q.clone())
        for out in outs:
            before = out.clone()
            y = B.oq_kv4_append(kv, out if out is not outs[0] else q, k, v, s.cache, s.table, s.cu + 2, s.len, table=t, positions=p,
                                q_out=out)
            assert y is out and torch.equal(out[rows], part) and torch.equal(cache, s.cache)
            assert torch.equal(out[:2], before[:2]) and torch.equal(out[2 + s.T:], before[2 + s.T:])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 4, 47, 60])
@pytest.mark.parametrize("far", [2.0 ** 103 * 1.2, 2.0 ** 110, 2.0 ** 124 * 1.6])
def test_scores_up_to_the_end_of_fp32(env, D, n, far):
    """Among them queries all of whose scores are below -10^30."""
    _far(env, D, n, far)


@pytest.mark.parametrize("D,H,KH", [(128, 2, 1), (64, 8, 2), (128, 16, 1)])
def test_small_query_channels_meet_large_keys(env, D, H, KH):
    """Channels from 2^-10 to 2^-22 of their block's largest, under keys that make up for it."""
    torch, B = env
    rng = np.random.default_rng(45)
    kv = B.oq_kv4_create(H, KH, D)
    s = Streams(torch, rng, kv, [2, 1], [300, 41])
    down = 2.0 ** -(10 + np.arange(D) % 13)
    down[::32] = 1                              # a block's largest
    up = np.where(down == 1, 2.0 ** -4, 2.0 ** 12)   # (one scale for a block: keys of 2^12 beside keys of 0)
    for b, m in enumerate(s.lens):
        for j in range(m):
            k = rng.standard_normal((KH, D)) * up * (rng.random((KH, D)) < 0.3)
            A.write_token(s.np_cache, s.pages[b, j // 128], j % 128, k.ravel(), rng.standard_normal(KH * D))
    s.cache.copy_(torch.from_numpy(s.np_cache))
    q = torch.from_numpy((rng.uniform(1, 2, (s.T, H, D)) * rng.choice([-1, 1], (s.T, H, D)) * down).astype(np.float32)).cuda().bfloat16()
    _check_attention(torch, B, kv, s, q)


@pytest.mark.parametrize("D,H,KH", [(128, 1, 1), (64, 4, 2), (64, 8, 1), (128, 16, 1), (64, 32, 2), (128, 60, 1), (64, 128, 2)])
def test_far_queries_beside_others(env, D, H, KH):
    """Of neighbouring queries one has scores of 10^9, one of 10^30 and one is NaN: the others keep their bounds."""
    torch, B = env
    rng = np.random.default_rng(46)
    kv = B.oq_kv4_create(H, KH, D)
    s = Streams(torch, rng, kv, [1, 3], [700, 300])
    for b, m in enumerate(s.lens):
        for j in range(m):
            A.write_token(s.np_cache, s.pages[b, j // 128], j % 128, rng.standard_normal(KH * D), rng.standard_normal(KH * D))
    s.cache.copy_(torch.from_numpy(s.np_cache))
    q = rng.standard_normal((s.T, H, D)).astype(np.float32)
    q[0, ::5] *= 1e9
    q[1:, 2::7] *= 1e30
    q[2, 1::6] = np.nan
    q = torch.from_numpy(q).cuda().bfloat16()
    for window in (0, 100):
        _check_attention(torch, B, kv, s, q, window=window)
