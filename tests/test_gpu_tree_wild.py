"""sparse_paged_tree_attn: values of nodes that are NaN or infinite reach the rows that see the node and no others."""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_tree_attn import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,n,G,K,Pmax", [([100, 0, 517, 128], 9, 4, 0, None), ([300, 121], 64, 4, 0, None), ([300, 50], 64, 8, 0, None),
                                             ([1000, 47], 13, 3, 6, None), ([130], 3, 1, 0, None), ([900, 60, 0], 40, 2, 0, 4000),
                                             ([60] * 40, 7, 8, 0, 4000), ([20000], 30, 4, 0, None)])
@pytest.mark.parametrize("T,D", [(16, 128), (32, 64), (32, 128)])
@pytest.mark.parametrize("what", ["value", "key"])
def test_nodes_that_are_not_finite(lens, n, G, K, Pmax, T, D, what):
    """Against the same call with zeros in their place: equal bit by bit where the node is not seen, and in other channels."""
    c = Case(lens, [max(1, n - b % 3) for b in range(len(lens))], n, Hkv=2, G=G, D=D, T=T, K=K, Pmax=Pmax, seed=n + T)
    r = np.random.RandomState(n)
    wild = {}
    for b in range(c.B):
        for h in range(2):
            for j in sorted(set(r.randint(0, c.nodes[b], 1 + c.nodes[b] // 6).tolist() + [c.nodes[b] - 1])):
                wild[b, h, j] = sorted(set(r.randint(0, D, 2).tolist() + [D - 1] * (j % 2)))

    def put(values):
        for i, ((b, h, j), channels) in enumerate(sorted(wild.items())):
            t = c.lens[b] + j
            page = int(c.table[b, 0, h, t // T])
            for x, d in enumerate(channels):
                at = (page, d, t % T) if what == "value" else (page, t % T, d)
                (c.v_pool if what == "value" else c.k_pool)[at] = values[(i + x) % len(values)]

    put([0.0])
    c.call()
    want, want_lse = c.out.clone(), c.lse.clone()
    put([math.nan, math.inf, -math.inf])
    c.call()
    torch.cuda.synchronize()
    assert int(c.err) == 0
    sees = np.zeros((c.B, 2, n, D), dtype=bool)
    for (b, h, j), channels in wild.items():
        for i in range(c.nodes[b]):
            if int(c.bits[b, i]) >> j & 1:
                sees[b, h, i, channels if what == "value" else slice(None)] = True
    hurt = torch.from_numpy(sees).cuda().permute(0, 2, 1, 3).repeat_interleave(G, 2)  # [B, n, Hq, D]
    assert torch.equal(c.out[~hurt], want[~hurt])
    assert not hurt.all()
    if what == "value":
        assert c.out[hurt].isnan().all()
        assert torch.equal(c.lse, want_lse)
    else:
        rows = hurt.any(-1)
        assert torch.equal(c.lse[~rows], want_lse[~rows])


def test_a_replaced_value_does_not_last():
    """Nothing of it is kept for the CTA's next units, or the next call."""
    c = Case([60] * 90, [5] * 90, 5, Hkv=2, G=4, D=128, Pmax=1000, seed=3)
    c.call()
    want = c.out.clone()
    for b in range(0, 90, 3):
        at = int(c.table[b, 0, 1, 62 // 16]), 7, 62 % 16
        was = c.v_pool[at].clone()
        c.v_pool[at] = math.inf
        c.call()
        c.v_pool[at] = was
        seen = [i for i in range(5) if int(c.bits[b, i]) >> 2 & 1]
        spoilt = c.out[b, seen, 4:, 7]
        assert spoilt.isnan().all()
        c.out[b, seen, 4:, 7] = want[b, seen, 4:, 7]
        assert torch.equal(c.out, want)
    c.call()
    assert torch.equal(c.out, want)
    c.check()
