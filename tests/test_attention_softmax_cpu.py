"""CPU restatement of how the attention kernels move the softmax reference: at which scores, how often, and what the
weights become."""

import numpy as np
import pytest

import softmax_emulation as S

F = np.float32
MANY = 50          # passes after which a rule counts as one that does not end


@pytest.mark.parametrize("D", [64, 128])
def test_scores_at_the_border_of_a_move_end(D):
    """Scores that round to M + 8 and exceed it by less than a rounding, for every M from 8 to 400."""
    c2 = S.log2e(D ** -0.5)
    found = stuck = 0
    for m in range(8, 401):
        s = S.border_score(m, c2)
        if s is None:
            continue
        found += 1
        tile = np.array([s, F(0), F(1)], F)
        stuck += S.chunk_tile(tile, c2, F(m), MANY)[2] == MANY      # asking until no weight exceeds 2^8
        w, M, made = S.chunk_tile(tile, c2, F(m))
        assert made <= 2 and M == m and 256 < w.max() < 256.1
    assert found > 100 and stuck == found


def test_large_scores_end():
    """Normal scores times 1 to 10^10, several tiles."""
    rng = np.random.default_rng(0)
    c2 = S.log2e(128 ** -0.5)
    stuck = 0
    for e in range(11):
        for _ in range(40):
            M = old = S.NONE
            for _ in range(8):
                s = (rng.standard_normal(16) * 10.0 ** e).astype(F)
                if old is not None:
                    w, old, made = S.chunk_tile(s, c2, old, MANY, far=False)
                    if made == MANY:
                        stuck, old = stuck + 1, None
                w, M, made = S.chunk_tile(s, c2, M)
                assert made <= 2 and not np.isnan(w).any()
    assert stuck > 10


def test_weights_of_far_scores():
    """From 2^22 on: no weight above 2^8, the largest score's not below 1 / 2, whatever the scores' magnitude."""
    rng = np.random.default_rng(1)
    c2 = S.log2e(128 ** -0.5)
    wrong = 0
    for e in range(4, 38):
        for _ in range(20):
            M = S.NONE
            for t in range(4):
                s = (rng.standard_normal(16) * 10.0 ** e).astype(F)
                last, (w, M, _) = M, S.chunk_tile(s, c2, M)
                assert w.max() <= 256.1
                if M != last:
                    assert w.max() >= 0.5
                one = S.weights(s, c2, M, far=False)
                wrong += not (one.max() <= 256.1 and (M == last or one.max() >= 0.5))
    assert wrong > 100


def test_weights_of_a_far_block_fit_e4m3():
    """Few queries: a block's largest weight times 2^8 over its power of two, at most 2^8 (e4m3 ends at 448)."""
    rng = np.random.default_rng(2)
    c2 = S.log2e(128 ** -0.5)
    beyond = 0
    for e in np.arange(0, 37, 0.25):
        s = (rng.uniform(1, 10, 400) * rng.choice([-1, 1], 400) * 10.0 ** e).astype(F)   # blocks of one token each
        m = np.ceil(F(s * c2))
        once = S.fma(s, c2, F(F(8) - m))
        x = np.where(np.abs(m) > S.FAR, F(F(F(s * c2) - m) + F(8)), once)
        assert x.max() <= 8.71 and x.min() >= 7 - 2.0 ** -20
        beyond += (once > np.log2(448)).sum()
    assert beyond > 100
