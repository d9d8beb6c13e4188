"""Plain fp64 numpy statement of the operators around attention, for the tests:
norm and rotation of heads, the 4-bit cache's layout (include/orbitquant.h),
attention over it with bounds of the kernel's error, and 4-bit weights with
group scales.  No code of the library."""

import numpy as np

import mx_reference as R

PAGE = 128


def turn(x, gain=None, eps=1e-6, table=None, pos=None, inter=False, norm=True):
    """fp64 [T, H, D] -> (result, |a| + |b| of the pair each value was turned from)."""
    n = x.astype(np.float64)
    with np.errstate(all="ignore"):
        if norm:
            n = n / np.sqrt((n * n).mean(-1, keepdims=True) + eps)
            if gain is not None:
                n = n * gain
    mag = np.abs(n)
    if table is None:
        return n, mag
    half = table.shape[1]
    bad = (pos < 0) | (pos >= table.shape[0])
    t = np.where(bad[:, None, None], np.nan, table[np.where(bad, 0, pos)].astype(np.float64))
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)
    c, s = t[:, None, :, 0], t[:, None, :, 1]
    out, m = n.copy(), mag.copy()
    with np.errstate(all="ignore"):
        out[..., a] = n[..., a] * c - n[..., b] * s
        out[..., b] = n[..., b] * c + n[..., a] * s
        m[..., a] = m[..., b] = mag[..., a] + mag[..., b]
    return out, m


# ------------------------------------------------------------------ the cache
def groups_of(kv_heads, D):
    return -(-kv_heads * D // 128)


def cache_values(cache):
    """uint8 [pages, G, 272, 64] -> K, V values [pages, G, 128 tokens, 128 channels]."""
    P, G = cache.shape[:2]
    nib = np.stack((cache & 15, cache >> 4), -1).reshape(P, G, 272, 128)
    flat = cache[:, :, 256:].reshape(P, G, 1024)
    ks = flat[..., :512].reshape(P, G, 32, 4, 4).transpose(0, 1, 3, 2, 4).reshape(P, G, 128, 4)
    vs = flat[..., 512:].reshape(P, G, 128, 4)
    k = R.code_values(nib[:, :, :128], 4)
    v = R.code_values(nib[:, :, 128:256], 4).transpose(0, 1, 3, 2)
    return k * R.scale_values(ks).repeat(32, -1), v * R.scale_values(vs).repeat(32, -1)


def write_token(cache, page, row, k, v):
    """One token's heads (fp64 [kv_heads * D]) into a numpy cache, element by element."""
    G = cache.shape[1]
    pad = np.zeros(G * 128)
    for which, x in (("k", k), ("v", v)):
        pad[:] = 0
        pad[:x.size] = x
        codes, sc = R.quantize(pad.reshape(1, -1), 4)
        for g in range(G):
            c, s = codes[0, g * 128:(g + 1) * 128], sc[0, g * 4:(g + 1) * 4]
            if which == "k":
                cache[page, g, row] = c[0::2] | (c[1::2] << 4)
                at = 256 * 64 + row % 32 * 16 + row // 32 * 4
            else:
                col = cache[page, g, 128:256, row // 2]
                cache[page, g, 128:256, row // 2] = (col & 0x0F) | (c << 4) if row % 2 else (col & 0xF0) | c
                at = 264 * 64 + row * 4
            cache[page, g].reshape(-1)[at:at + 4] = s


def sequence(k, v, pages, length, kv_heads, D):
    """Values of a sequence's tokens from cache_values' arrays -> K, V [length, kv_heads, D], and which are there."""
    P, G = k.shape[:2]
    j = np.arange(length)
    p = pages[j // PAGE]
    ok = (p >= 0) & (p < P)
    p = np.where(ok, p, 0)
    return (*(x[p, :, j % PAGE].reshape(length, G * 128)[:, :kv_heads * D].reshape(length, kv_heads, D) for x in (k, v)), ok)


def attention(q, K, V, there, scale, causal, window):
    """q [n, H, D] fp64 (exact bf16), K, V [len, KH, D], there [len] -> (y, tolerance) [n, H, D].

    The kernel's error.  Scores: fp32 sums of exact products in the tensor core,
    each of the at most 16 additions off by 2^-23 of the magnitudes, the second term of
    an element small against its block 2^-21 of the block's largest; times scale
    log2 e and less the reference in fp32, 2^-22 of the score's magnitude, ex2
    2^-22.  Weights: two e4m3 terms, 2^-4 of 2^-4, and below their range 2^-16 of
    the largest product with V's scales in the 32 tokens (2^-10 of 256, the power
    of two up to twice the weight, elements up to 6 of a scale that is a quarter of
    the largest at most).  Sums: one addition a tile and 32-token block, and the
    reductions.  The result: half a bf16 step, 2^-8."""
    n, H, D = q.shape
    L, KH = K.shape[:2]
    G = H // KH
    y, tol = np.zeros((n, H, D)), np.zeros((n, H, D))
    i, j = np.arange(n)[:, None] + (L - n), np.arange(L)[None]
    see = np.broadcast_to(there[None], (n, L)).copy()
    if causal:
        see &= j <= i
    if window:
        see &= j > i - window
    nb = -(-L // 32)
    for h in range(H):
        k, v = K[:, h // G], V[:, h // G]
        with np.errstate(all="ignore"):
            s = q[:, h] @ k.T * scale
            mags = np.abs(q[:, h]) @ np.abs(k).T * scale
            small = np.abs(q[:, h]).max(-1, keepdims=True) * np.abs(k).sum(-1)[None] * scale
            s[~see] = -np.inf
            top = np.where(see.any(-1), s.max(-1, initial=-np.inf), 0)[:, None]
            p = np.where(see, np.exp(s - top), 0)
            l = p.sum(-1, keepdims=True)
            p = p / np.where(l == 0, 1, l)   # a NaN score makes the row NaN
            keep = see.any(0)   # a hidden token's NaN goes nowhere
            kv = np.where(keep[:, None], v, 0)
            y[:, h] = p @ kv
            if np.isnan(kv).any():   # 0 * NaN for tokens hidden from some queries only
                for t in range(n):
                    y[t, h] = np.where(see[t][:, None], p[t][:, None] * v, 0).sum(0)
            es = np.where(see, mags * 16 * 2.0 ** -23 + small * 2.0 ** -21 + (np.abs(s) + np.abs(top)) * 2.0 ** -21 + 2.0 ** -20, 0)
            es = np.where(np.isfinite(es), es, 0).max(-1, initial=0.0)[:, None]
            av = np.nan_to_num(np.abs(kv))
            pv = np.nan_to_num(p) @ av
            pad = nb * 32 - L
            pm = np.pad(np.nan_to_num(p), ((0, 0), (0, pad))).reshape(n, nb, 32).max(-1)
            vm = np.pad(av, ((0, pad), (0, 0))).reshape(nb, 32, D // 32, 32).max((1, 3)).repeat(32, -1)
            tol[:, h] = 2.0 ** -8 * np.abs(np.nan_to_num(y[:, h])) \
                + (2.0 ** -8 + 2 * es + (2 * nb + 40) * 2.0 ** -23) * pv + 2.0 ** -16 * 32 * (pm @ vm)
    return y, tol


# ------------------------------------------------------------------ 4-bit weights
def w4g_places(d):
    """For each element of a row: (byte, whether in its high half)."""
    e = np.arange(-(-d // 128) * 128)
    r = e % 128
    word, nib = e // 128 * 16 + r // 8 % 4 * 4 + r // 32, r % 2 * 4 + r % 8 // 2
    return word * 4 + nib // 2, nib % 2


def bf16_round(x):
    """fp32 -> the nearest bf16 (ties to even), in fp32."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isfinite(x), r, x).astype(np.float32)


def w4g_prepare(W, group, zeros):
    """fp32 rows -> (element codes [N, d], scales fp32 (bf16 values), zeros [N, groups]) by the header's rules."""
    N, d = W.shape
    b = W.astype(np.float32).reshape(N, -1, group)
    bad = ~np.isfinite(b).all(-1)
    with np.errstate(all="ignore"):
        lo, hi = np.minimum(b.min(-1), np.float32(0)), np.maximum(b.max(-1), np.float32(0))
        s = bf16_round((hi - lo) / np.float32(15) if zeros else np.maximum(hi, -lo) / np.float32(7))
        bad |= ~np.isfinite(s)
        use = ~bad & (s > 0)
        s1 = np.where(use, s, np.float32(1))
        z = np.where(use, np.clip(np.rint(-lo / s1), 0, 15), 0) if zeros else np.full(s.shape, 8.0)
        c = np.clip(np.rint(b / s1[..., None]) + z[..., None], 0, 15)
    c = np.where(use[..., None], c, z[..., None])
    return c.reshape(N, d).astype(np.uint8), np.where(bad, np.float32(np.nan), s), z.astype(np.uint8)


def w4g_unpack(codes, d):
    byte, high = w4g_places(d)
    return np.where(high, codes[:, byte] >> 4, codes[:, byte] & 15)[:, :d]


def w4g_values(codes, scales, zeros, d, group):
    """fp64 [N, d] of packed codes."""
    c = w4g_unpack(codes, d).astype(np.float64)
    z = np.full(scales.shape, 8.0) if zeros is None else zeros.astype(np.float64)
    return (c - z.repeat(group, 1)) * scales.astype(np.float64).repeat(group, 1)
