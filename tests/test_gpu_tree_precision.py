"""sparse_paged_tree_attn: how much of a weight reaches the output.  Against 64 bits, beyond the output's own rounding."""
import numpy as np
import pytest

from tests.test_gpu_tree_attn import Case

pytestmark = pytest.mark.gpu


def half_step(x):
    """Half a step of bf16 (8 bits) at x."""
    return np.ldexp(1.0, np.frexp(np.maximum(np.abs(x), 1e-30))[1] - 9)


@pytest.mark.parametrize("lens,n,G,K", [([3], 2, 1, 0), ([40, 7], 5, 4, 0), ([200], 16, 8, 0), ([900], 40, 8, 0), ([900, 300], 64, 8, 0),
                                        ([300], 6, 4, 7), ([500], 64, 4, 12), ([2000, 1000], 9, 4, 0)])
@pytest.mark.parametrize("D,T", [(64, 16), (128, 16), (128, 32)])
def test_weights_keep_sixteen_bits(lens, n, G, K, D, T):
    """An output is rounded to bf16 once: off by half a step, and by what it was off before.  That is, of the sum of weight *
    |value|: 2^-16 by the weights, which are held in two halves of 8 bits (half a step of half a step: 2^-8 2^-8); the
    scores' error, as tree_plain.out_bound has it; 2^-22 by exp2; and by the sums, where 16 products are added at once to
    what was summed before: each such addition loses less than 2^-22 of the sum, two for each 16 tokens, and the streams' and
    CTAs' parts are joined by some 20 more."""
    c = Case(lens, [n] * len(lens), n, Hkv=2, G=G, D=D, T=T, K=K, seed=n + G)
    c.call()
    c.check()
    for b in range(c.B):
        for h in range(c.Hkv):
            (o, _, weighted, size), N = c.expect(b, h)
            z = size[:, None] * (D + 8) * 2.0 ** -23
            before = (2.0 ** -16 + 2 * z + 2.0 ** -22 * (N / 8 + 20)) * weighted
            got = c.out[b, :n, h * G:(h + 1) * G].double().cpu().numpy().reshape(n * G, D)
            far = np.abs(got - o) - 1.0001 * before - half_step(np.abs(o) + before)
            assert far.max() <= 0, (b, h, far.max(), (far > 0).mean())
