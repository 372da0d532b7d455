"""sparse_paged_tree_attn where the sums are known: queries of zero, so that every weight is 1, lse is the logarithm of the
tokens that a row sees and the output their values' mean.  Tables lead to a few physical pages again and again, so that a
sequence may be as long as the table allows."""
import math

import pytest
import torch

from paged_kv_cache_minmax_gb300 import kvmm

pytestmark = pytest.mark.gpu


class Case:
    """values [pages, D, T]: the physical pages; table [B, Hkv, Pmax]: entries."""

    def __init__(self, values, table, lens, n, G, mask=None, sel=None, cnt=None):
        B, Hkv, P = table.shape
        pages, D, T = values.shape
        dev = dict(device="cuda")
        self.v_pool, self.k_pool = values, torch.randn(pages, T, D, **dev).to(torch.bfloat16)
        self.table = table.to(torch.int32).view(B, 1, Hkv, P).contiguous()
        self.shape = kvmm.make_shape(B, 1, Hkv * G, Hkv, D, T, P, 1 if sel is None else sel.shape[-1], pages)
        self.q = torch.zeros(B, n, Hkv * G, D, dtype=torch.bfloat16, **dev)
        self.out = torch.full((B, n, Hkv * G, D), 7.0, dtype=torch.bfloat16, **dev)
        self.lse = torch.full((B, n, Hkv * G), 7.0, **dev)
        self.err = torch.zeros(1, dtype=torch.int32, **dev)
        self.ws = kvmm.alloc_tree_workspace(self.shape, n)
        self.ws.fill_(255)  # (NaN)
        kvmm.sparse_paged_tree_attn(self.shape, 0, self.q, self.k_pool, self.v_pool, self.table,
                                    torch.tensor(lens, dtype=torch.int32, **dev), self.out, self.ws, tree_mask=mask,
                                    sel_idx=sel, sel_cnt=cnt, lse=self.lse, err=self.err)
        torch.cuda.synchronize()
        assert int(self.err) == 0


def lse_is(lse, count):
    """log of a whole number that fp32 holds: log2f is off by an ulp, its product with ln 2 and that constant by half each."""
    want = torch.as_tensor(count, dtype=torch.float64, device="cuda").log()
    off = (lse.double() - want).abs() - 2.0 ** -21 * want.abs()
    assert (off <= 0).all(), off.max().item()


# units: how they are taken (a cluster each, or blocks dealt to the SMs, a CTA with a part of one or parts of several)
UNITS = [(1, 1, 1000, None), (1, 8, 3991, None), (2, 8, 8200, None), (1, 1, 40003, None), (3, 3, 9017, None), (1, 8, 131050, None),
         (5, 8, 20011, None), (40, 4, 6007, None), (4, 2, 1500, 5000)]


@pytest.mark.parametrize("n,G", [(1, 1), (7, 4), (16, 8), (33, 5), (64, 4), (64, 8)])
@pytest.mark.parametrize("T,D", [(16, 128), (32, 64)])
@pytest.mark.parametrize("B,Hkv,tokens,Pmax", UNITS)
def test_every_block_counts_once(n, G, T, D, B, Hkv, tokens, Pmax):
    """A block's values are 1 in the channel of its number and 0 elsewhere: one that is lost or taken twice changes a channel
    by a share of blocks / D, one token changes lse by more than its bound."""
    lens = [max(0, tokens - 977 * b) for b in range(B)]
    P = -(-(tokens + n) // T) if Pmax is None else Pmax
    marks = torch.eye(D, device="cuda").to(torch.bfloat16).unsqueeze(-1).expand(D, D, T).contiguous()
    entry = torch.arange(P, device="cuda") * T // 128 % D
    c = Case(marks, entry.expand(B, Hkv, P), lens, n, G)
    for b in range(B):
        count = lens[b] + 1 + torch.arange(n, device="cuda")  # a chain
        lse_is(c.lse[b], count.view(n, 1).expand(n, Hkv * G))
        blocks = torch.arange(-(-(lens[b] + n) // 128), device="cuda")
        held = (count.view(n, 1) - 128 * blocks).clamp(0, 128)  # [n, blocks]
        want = torch.zeros(n, D, dtype=torch.float64, device="cuda").index_add_(1, blocks % D, held.double()) / count.view(n, 1)
        # sums of ones are exact; 1 / l, its product and the rounding to bf16 are not
        off = (c.out[b].double() - want.unsqueeze(1)).abs() - (2.0 ** -8 + 2.0 ** -22) * want.unsqueeze(1)
        assert (off <= 0).all(), (b, off.max().item())


@pytest.mark.parametrize("n,G", [(1, 2), (16, 4), (64, 4), (50, 8)])
@pytest.mark.parametrize("T", [16, 32])
@pytest.mark.parametrize("B,Hkv,K", [(1, 1, 37), (8, 8, 128), (3, 2, 700), (30, 8, 41)])
def test_every_selected_page_counts_once(n, G, T, B, Hkv, K):
    """Selections: a page's values mark its place in the list."""
    D, P, seq = 64, 900, 880 * 16 // T * T
    P = P * 16 // T
    K = min(K, seq // T)
    g = torch.Generator(device="cuda")
    g.manual_seed(K)
    marks = torch.eye(D, device="cuda").to(torch.bfloat16).unsqueeze(-1).expand(D, D, T).contiguous()
    marks = torch.cat([marks, torch.zeros(1, D, T, dtype=torch.bfloat16, device="cuda")])  # D: the nodes' pages
    sel = torch.rand(B, Hkv, seq // T, generator=g, device="cuda").argsort(-1)[..., :K]
    cnt = torch.randint(0, K + 1, (B, Hkv), generator=g, device="cuda")
    cnt[0, 0] = K
    table = torch.full((B, Hkv, P), D, device="cuda")
    table.scatter_(2, sel, (torch.arange(K, device="cuda") % D).expand(B, Hkv, K).contiguous())
    c = Case(marks, table, [seq] * B, n, G, sel=sel.to(torch.int32).view(B, 1, Hkv, K).contiguous(),
             cnt=cnt.to(torch.int32).view(B, 1, Hkv).contiguous())
    seen = cnt.view(B, 1, Hkv) * T + 1 + torch.arange(n, device="cuda").view(n, 1)  # [B, n, Hkv]
    lse_is(c.lse.view(B, n, Hkv, G), seen.unsqueeze(-1).expand(B, n, Hkv, G))
    pages = torch.zeros(B, Hkv, D, dtype=torch.float64, device="cuda")
    pages.scatter_add_(2, (torch.arange(K, device="cuda") % D).expand(B, Hkv, K).contiguous(),
                       (torch.arange(K, device="cuda") < cnt.unsqueeze(-1)).double())
    want = (pages * T).view(B, 1, Hkv, 1, D) / seen.view(B, n, Hkv, 1, 1)
    off = (c.out.view(B, n, Hkv, G, D).double() - want).abs() - (2.0 ** -8 + 2.0 ** -22) * want
    assert (off <= 0).all(), off.max().item()
