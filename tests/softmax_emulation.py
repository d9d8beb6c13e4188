"""The running softmax reference of the attention kernels, restated in fp32 on the host."""

import numpy as np

F = np.float32
LAZY, NONE = F(8), -np.finfo(F).max


def fma(a, b, c):
    """fp32 a * b + c, rounded once: the product is exact in 64 bits, and the sum too where it cancels or fits."""
    return F(np.float64(a) * np.float64(b) + np.float64(c))


def log2e(scale):
    return F(scale) * F(1.4426950408889634)


def parts3(x):
    """fp32 -> three bf16 numbers whose sum it is."""
    out = []
    for _ in range(3):
        h = (np.asarray(x, F).view(np.uint32) & np.uint32(0xFFFF0000)).view(F)
        out.append(h)
        x = F(x - h)
    assert (x == 0).all()
    return out


def border_score(m, c2):
    """An fp32 s whose s * c2 rounds to m + 8 and yet exceeds it, or None."""
    s = F(np.float64(m + 8) / np.float64(c2))
    for _ in range(4):
        s = np.nextafter(s, F(0))
    for _ in range(9):
        if F(s * c2) == F(m + 8) and fma(s, c2, F(-m)) > LAZY:
            return s
        s = np.nextafter(s, F(np.inf))
    return None


FAR = F(2 ** 22)


def weights(s, c2, M, far=True):
    with np.errstate(over="ignore"):
        x = F(F(s * c2) - M) if far and abs(M) > FAR and M != NONE else fma(s, c2, -M)
        return np.exp2(x.astype(np.float64)).astype(F)


def chunk_tile(s, c2, M, passes=2, far=True):
    """A tile's scores of one query relative to the reference M -> (weights, M, passes made).  `passes`: after so many
    the weights are taken as they are; `far`: whether products are rounded by themselves from FAR on."""
    move, made = M == NONE, 0
    while True:
        if made == passes - 1 or not move:
            w = weights(s, c2, M, far)
            move = w.max() > 256
            if made == passes - 1 or not move:
                return w, M, made + 1
        made += 1
        m = F(s.max() * c2)
        M = np.ceil(m) if m > M + LAZY else M
