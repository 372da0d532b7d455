"""sparse_paged_tree_attn over the longest tables, a unit a CTA: the tensor cores' sums, which are rounded toward zero, do not
drift, and what is summed in runs is put together again."""
import math

import numpy as np
import pytest
import torch

from paged_kv_cache_minmax_gb300 import kvmm
from tests.test_gpu_tree_precision import half_step
from tests import test_gpu_tree_sums as sums
from tests.test_gpu_tree_sums import Case, lse_is

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,G", [(1, 1), (64, 4)])
@pytest.mark.parametrize("T,D", [(16, 64), (32, 128)])
def test_long_runs_do_not_drift(n, G, T, D):
    """As many units as there are SMs, each of 2^19 or 2^20 tokens of positive values: a CTA sums whole units.  An addition
    that truncates is off by at most 2^-23 of the sum, always downwards; of 1,024 in a row, on a sum that grows steadily, the
    result is off by at most half of 1,024 * 2^-23 = 2^-14.  Each 1,024 are added to the others with one addition to nearest
    (64 at most, 2^-24 each), 1 / l and its product are rounded to nearest likewise: 2^-17.  Then half a step of bf16."""
    B, Hkv, P = 20, 8, 32768
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    values = (torch.rand(64, D, T, generator=g, device="cuda") + 0.5).to(torch.bfloat16)
    table = torch.randint(0, 64, (B, Hkv, P), generator=g, device="cuda")
    seq = P * T - 64
    c = Case(values, table, [seq] * B, n, G, mask=torch.zeros(B, n, dtype=torch.int64, device="cuda"))  # no node sees a node
    lse_is(c.lse, torch.full_like(c.lse, seq))
    times = torch.zeros(B, Hkv, 64, dtype=torch.float64, device="cuda")
    times.scatter_add_(2, table[..., :seq // T], torch.ones(B, Hkv, seq // T, dtype=torch.float64, device="cuda"))
    want = (times @ values.double().sum(-1)) / seq  # [B, Hkv, D]
    far = c.out.view(B, n, Hkv, G, D).double() / want.view(B, 1, Hkv, 1, D) - 1
    print(f"mean signed error {far.mean().item():.3e}, the largest {far.abs().max().item():.3e}")
    assert (c.out.view(B, n, Hkv, G, D) == c.out.view(B, n, Hkv, G, D)[:, :1, :, :1]).all()  # rows are alike
    want, got = want.cpu().numpy(), c.out.view(B, n, Hkv, G, D)[:, 0, :, 0].double().cpu().numpy()
    before = (2.0 ** -14 + 2.0 ** -17) * want
    over = np.abs(got - want) - before - half_step(want + before)
    assert over.max() <= 0, (over.max(), (over > 0).mean())


@pytest.mark.parametrize("n,G", [(1, 1), (7, 4), (16, 8), (33, 5), (64, 8)])
@pytest.mark.parametrize("T,D", [(16, 128), (32, 64)])
@pytest.mark.parametrize("B,Hkv,tokens", [(40, 4, 33001), (19, 8, 16523), (1, 2, 524007)])
def test_every_block_of_long_runs_counts_once(n, G, T, D, B, Hkv, tokens):
    sums.test_every_block_counts_once(n, G, T, D, B, Hkv, tokens, None)


@pytest.mark.parametrize("order", ["up", "down", "any"])
@pytest.mark.parametrize("n,G", [(1, 3), (13, 5), (64, 4)])
@pytest.mark.parametrize("T,D,tokens", [(16, 128, 40000), (32, 64, 300000)])
def test_long_runs_against_64_bits(order, n, G, T, D, tokens):
    """The table leads to 64 pages, in the order of their scores or in any: the exact softmax weighs each by the times that it
    is listed.  The outputs' bound is test_gpu_tree_precision's with the additions of a run, 1,024 of 16 products, each off
    by less than 2^-22 of the sum (2^-12), and those of the runs; lse's has an addition to nearest (2^-24) a block, and some 60 within."""
    B, Hkv, P = 20, 8, tokens // T
    seq = P * T - 64
    g = torch.Generator(device="cuda")
    g.manual_seed(n + T)
    values = torch.randn(64, D, T, generator=g, device="cuda").to(torch.bfloat16)
    table = torch.randint(0, 64, (B, Hkv, P), generator=g, device="cuda")
    if order != "any":
        table = table.sort(-1, descending=order == "down").values
    mask = torch.zeros(B, n, dtype=torch.int64, device="cuda")
    c = Case(values, table, [seq] * B, n, G, mask=mask)  # (once with queries of zero)
    keys = torch.randn(64, T, D, generator=g, device="cuda")
    keys[..., 0] = torch.arange(64, device="cuda").view(64, 1) / 4.0
    c.k_pool = keys.to(torch.bfloat16)
    c.q = torch.randn(B, n, Hkv * G, D, generator=g, device="cuda").to(torch.bfloat16)
    c.q[..., 0] = 8.0
    kvmm.sparse_paged_tree_attn(c.shape, 0, c.q, c.k_pool, c.v_pool, c.table,
                                torch.full((B,), seq, dtype=torch.int32, device="cuda"), c.out, c.ws, tree_mask=mask, lse=c.lse,
                                err=c.err)
    torch.cuda.synchronize()
    assert int(c.err) == 0
    times = torch.zeros(B, Hkv, 64, dtype=torch.float64, device="cuda")
    times.scatter_add_(2, table[..., :seq // T], torch.ones(B, Hkv, seq // T, dtype=torch.float64, device="cuda"))
    k, v = c.k_pool.double().view(64 * T, D), c.v_pool.double().transpose(1, 2).reshape(64 * T, D)
    many = times.repeat_interleave(T, -1)  # [B, Hkv, 64 T]
    q = c.q.double().view(B, n, Hkv, G, D)
    for b in (0, 7, 19):
        for h in (0, 5):
            rows = q[b, :, h].reshape(n * G, D)
            z = rows @ k.T / math.sqrt(D)
            live = many[b, h] > 0
            z[:, ~live] = -math.inf
            e = (z - z.amax(-1, keepdim=True)).exp() * many[b, h]
            l = e.sum(-1, keepdim=True)
            o, weighted = (e / l @ v).cpu().numpy(), (e / l @ v.abs()).cpu().numpy()
            size = (rows.abs() @ k[live].abs().T / math.sqrt(D)).amax(-1).cpu().numpy()[:, None] * (D + 8) * 2.0 ** -23
            before = (2.0 ** -16 + 2 * size + 2.0 ** -12 + 2.0 ** -16) * weighted
            got = c.out.view(B, n, Hkv, G, D)[b, :, h].double().cpu().numpy().reshape(n * G, D)
            far = np.abs(got - o) - 1.0001 * before - half_step(np.abs(o) + before)
            assert far.max() <= 0, (b, h, far.max())
            want = (z.amax(-1) + l.log().squeeze(-1)).cpu().numpy()
            off = np.abs(c.lse.view(B, n, Hkv, G)[b, :, h].double().cpu().numpy().reshape(-1) - want)
            assert (off <= size[:, 0] + (tokens / 128 + 60) * 2.0 ** -24 + np.abs(want) * 2.0 ** -21).all(), (b, h, off.max())
