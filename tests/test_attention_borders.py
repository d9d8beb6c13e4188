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
