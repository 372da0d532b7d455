"""sparse_paged_tree_attn against a plain implementation in 64 bits.  Slots of the pools that no settled token and no
node has hold NaN."""
import math

import numpy as np
import pytest
import torch

from paged_kv_cache_minmax_gb300 import kvmm
from tests import tree_plain

pytestmark = pytest.mark.gpu

NAN, INF = 0x7FC0, 0x7F80


def bits_of(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


class Case:
    """A layer's pools with the given settled lengths and nodes; other layers' pages and unused slots hold NaN."""

    def __init__(self, lens, nodes, n, Hkv=2, G=4, D=64, T=16, L=1, layer=0, K=0, mask="tree", seed=0, Pmax=None, scale=0.0,
                 spare=3):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        r = np.random.RandomState(seed)
        self.lens, self.nodes, self.n = list(lens), list(nodes), n
        B = len(lens)
        self.B, self.Hkv, self.G, self.D, self.T, self.L, self.layer = B, Hkv, G, D, T, L, layer
        Hq = Hkv * G
        P = max(1, max(-(-(a + b) // T) for a, b in zip(lens, nodes))) + 1 if Pmax is None else Pmax
        n_phys = B * L * Hkv * P + spare
        perm = torch.randperm(n_phys, generator=g, device="cuda")[:B * L * Hkv * P]
        self.table = perm.to(torch.int32).view(B, L, Hkv, P).contiguous()
        self.shape = kvmm.make_shape(B, L, Hq, Hkv, D, T, P, max(K, 1), n_phys)
        self.k_pool = torch.full((n_phys, T, D), math.nan, dtype=torch.bfloat16, device="cuda")
        self.v_pool = torch.full((n_phys, D, T), math.nan, dtype=torch.bfloat16, device="cuda")
        self.kv = {}
        for b in range(B):
            N = min(lens[b] + nodes[b], P * T)
            for h in range(Hkv):
                k = torch.randn(N, D, generator=g, device="cuda").to(torch.bfloat16)
                k[:, :3] *= 6
                v = (torch.randn(N, D, generator=g, device="cuda") + 0.5).to(torch.bfloat16)
                t = torch.arange(N, device="cuda")
                phys = self.table[b, layer, h].long()[t // T]
                self.k_pool[phys, t % T] = k
                self.v_pool[phys, :, t % T] = v
                self.kv[b, h] = k.double().cpu().numpy(), v.double().cpu().numpy()
        self.q = torch.randn(B, n, Hq, D, generator=g, device="cuda").to(torch.bfloat16)
        self.seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.n_nodes = torch.tensor(nodes, dtype=torch.int32, device="cuda")
        self.out = torch.full((B, n, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((B, n, Hq), 7.0, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = torch.randint(0, 255, (kvmm.tree_workspace_size(self.shape, n),), dtype=torch.uint8, device="cuda",
                                generator=g)
        if mask == "chain":
            self.bits, self.mask = np.array([[(1 << (i + 1)) - 1 for i in range(n)]] * B, dtype=np.uint64), None
        else:
            if mask == "tree":
                parent = np.full((B, n), -1)
                for i in range(1, n):
                    parent[:, i] = r.randint(max(0, i - 3), i, B)
                self.bits = tree_plain.masks(parent)
            elif mask == "random":
                self.bits = r.randint(0, 1 << 62, (B, n)).astype(np.uint64) * np.uint64(4) + r.randint(0, 4, (B, n)).astype(np.uint64)
            elif mask == "none":
                self.bits = np.zeros((B, n), dtype=np.uint64)
            else:
                self.bits = np.full((B, n), ~np.uint64(0))
            self.mask = torch.from_numpy(self.bits.view(np.int64)).cuda()
        self.sel = self.cnt = None
        self.K = K
        if K:
            sel, cnt = np.zeros((B, L, Hkv, K), dtype=np.int32), np.zeros((B, L, Hkv), dtype=np.int32)
            for b in range(B):
                pages = -(-lens[b] // T)
                for h in range(Hkv):
                    m = min(K, pages) if h % 2 == 0 else r.randint(0, min(K, pages) + 1)
                    sel[b, layer, h, :m] = np.sort(r.permutation(pages)[:m])
                    cnt[b, layer, h] = m
            self.sel, self.cnt = torch.from_numpy(sel).cuda(), torch.from_numpy(cnt).cuda()
        self.scale = scale

    def call(self, **kw):
        a = dict(n_nodes=self.n_nodes, tree_mask=self.mask, sel_idx=self.sel, sel_cnt=self.cnt, lse=self.lse, err=self.err,
                 sm_scale=self.scale)
        a.update(kw)
        kvmm.sparse_paged_tree_attn(self.shape, self.layer, self.q, self.k_pool, self.v_pool, self.table, self.seq, self.out,
                                    self.ws, **a)

    def expect(self, b, h, skip=()):
        """Rows of (b, h) in 64 bits; pages in `skip` contribute nothing."""
        seq, m, T = self.lens[b], self.nodes[b], self.T
        k, v = self.kv[b, h]
        N = k.shape[0]
        tok = np.arange(N)
        old = tok < seq
        if self.K:
            got = self.sel[b, self.layer, h, :int(self.cnt[b, self.layer, h])].cpu().numpy()
            old &= np.isin(tok // T, got)
        fine = ~np.isin(tok // T, skip)
        shown = np.zeros((m, N), dtype=bool)
        for i in range(m):
            j = tok - seq
            bit = np.array([(int(self.bits[b, i]) >> int(x)) & 1 if 0 <= x < 64 else 0 for x in j], dtype=bool)
            shown[i] = (old | ((j >= 0) & (j < m) & bit)) & fine
        G, D = self.G, self.D
        q = self.q[b, :m, h * G:(h + 1) * G].double().cpu().numpy().reshape(m * G, D)
        scale = self.scale if self.scale > 0 else 1 / math.sqrt(D)
        return tree_plain.attend(q, k, v, shown.repeat(G, 0), scale), N

    def check(self, err=0, skip=()):
        torch.cuda.synchronize()
        assert int(self.err) == err
        G, D = self.G, self.D
        for b in range(self.B):
            m = self.nodes[b]
            assert (self.out[b, m:] == 7.0).all() and (self.lse[b, m:] == 7.0).all(), "rows that do not exist were written"
            if not m:
                continue
            for h in range(self.Hkv):
                (o, lse, weighted, size), N = self.expect(b, h, skip)
                got = self.out[b, :m, h * G:(h + 1) * G].double().cpu().numpy().reshape(m * G, D)
                got_lse = self.lse[b, :m, h * G:(h + 1) * G].double().cpu().numpy().reshape(m * G)
                far = np.abs(got - o) - tree_plain.out_bound(o, weighted, size, D, N)
                assert far.max() <= 0, (b, h, np.unravel_index(far.argmax(), far.shape), far.max())
                assert np.array_equal(np.isneginf(lse), np.isneginf(got_lse)), (b, h)
                with np.errstate(invalid="ignore"):
                    off = np.where(np.isneginf(lse), 0.0, np.abs(got_lse - lse))
                assert (off <= tree_plain.lse_bound(lse, size, D, N)).all(), (b, h, off.max())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [16, 32])
@pytest.mark.parametrize("G", [1, 4, 7, 8])
@pytest.mark.parametrize("n", [1, 5, 33])
def test_every_page(D, T, G, n):
    c = Case([100, 0, 517, 128], [n, max(1, n - 2), n, 1], n, Hkv=2, G=G, D=D, T=T, seed=n + G)
    c.call()
    c.check()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [16, 32])
@pytest.mark.parametrize("K", [1, 9, 40])
@pytest.mark.parametrize("n", [1, 12, 64])
def test_selected_pages(D, T, K, n):
    c = Case([0, 1000, 47, 320], [n, n, 0, max(1, n - 5)], n, Hkv=3, G=3, D=D, T=T, K=K, seed=n + K, L=2, layer=1)
    c.call()
    c.check()


@pytest.mark.parametrize("mask", ["chain", "tree", "random", "none", "all"])
@pytest.mark.parametrize("n,G", [(64, 8), (64, 4), (64, 2), (40, 8), (17, 8), (16, 8), (3, 1)])
@pytest.mark.parametrize("lens", [[0, 0], [1, 255], [300, 16]])
def test_masks_and_row_counts(mask, n, G, lens):
    """Up to 512 rows a KV head, masks that leave rows empty where nothing is settled."""
    c = Case(lens, [n, max(1, n // 3)], n, Hkv=1, G=G, D=128, mask=mask, seed=n)
    c.call()
    c.check()


@pytest.mark.parametrize("T", [16, 32])
@pytest.mark.parametrize("at", list(range(0, 34)) + [111, 112, 113, 120, 127, 128, 129, 143, 144])
def test_tree_starts_anywhere_in_a_page(T, at):
    c = Case([at], [5], 5, Hkv=1, G=2, T=T, seed=at)
    c.call()
    c.check()
    c = Case([at], [40], 40, Hkv=1, G=2, T=T, seed=at, K=4)
    c.call()
    c.check()


@pytest.mark.parametrize("lens,n,K", [([40000], 8, 0), ([30000, 5, 9000], 24, 0), ([30000, 5, 9000], 7, 200), ([20011], 64, 0)])
def test_long_sequences(lens, n, K):
    c = Case(lens, [n] * len(lens), n, Hkv=2, G=4, D=128, K=K, seed=5)
    c.call()
    c.check()


@pytest.mark.parametrize("B", [33, 160])
def test_many_short_sequences(B):
    lens = [(37 * b) % 211 for b in range(B)]
    c = Case(lens, [b % 4 for b in range(B)], 3, Hkv=2, G=2, D=64, seed=B)
    c.call()
    c.check()


def test_no_optional_arguments():
    """No lse, no err, no n_nodes: every node exists."""
    c = Case([77, 130], [6, 6], 6, seed=2)
    c.call(lse=None, err=None, n_nodes=None)
    c.lse.fill_(0)
    want = c.out.clone()
    c.call()
    c.check()
    assert torch.equal(want, c.out)


@pytest.mark.parametrize("scale", [0.02, 3.0])
def test_scales(scale):
    c = Case([700], [9], 9, D=128, scale=scale, seed=3)
    c.call()
    c.check()


def test_growing_scores():
    """Every later page's scores lie above the earlier ones': the running maximum moves all the time; and the reverse."""
    for sign in (1, -1):
        c = Case([2000], [4], 4, Hkv=1, G=4, D=64, seed=8)
        ramp = torch.arange(2004, device="cuda").double().mul(sign * 0.02).to(torch.bfloat16)
        c.q[..., 0] = 8.0
        k, v = c.kv[0, 0]
        k[:, 0] = ramp.double().cpu().numpy()
        t = torch.arange(2004, device="cuda")
        c.k_pool[c.table[0, 0, 0].long()[t // 16], t % 16, 0] = ramp
        c.call()
        c.check()


def test_large_scores():
    """Scores in the hundreds: one token of each row holds nearly all the weight."""
    c = Case([900], [6], 6, Hkv=2, G=4, D=128, seed=9)
    c.q.mul_(16)
    c.call()
    c.check()


def test_every_slot_of_the_table():
    """A sequence that fills its table to the last slot; nodes beyond it are told and not attended, their rows written."""
    c = Case([250], [6], 6, Pmax=16, seed=4, Hkv=1)
    c.call()
    c.check()
    c = Case([250], [9], 9, Pmax=16, seed=4, Hkv=1, mask="all")  # three nodes have no place
    c.call()
    c.check(err=kvmm.ERR_OUT_OF_RANGE)
    c = Case([256], [4], 4, Pmax=16, seed=4, Hkv=1, mask="all", K=3)
    c.call()
    c.check(err=kvmm.ERR_OUT_OF_RANGE)


@pytest.mark.parametrize("K", [0, 30])
@pytest.mark.parametrize("page", [0, 3, 19, 20])
@pytest.mark.parametrize("entry", [-1, 1 << 30])
def test_pages_without_a_place(K, page, entry):
    """A null or impossible entry: told, and the page contributes nothing (page 20 holds nodes alone)."""
    c = Case([310], [14], 14, Hkv=1, G=4, K=K, seed=6)
    c.table[0, 0, 0, page] = entry
    c.call()
    c.check(err=kvmm.ERR_NULL_BLOCK if entry < 0 else kvmm.ERR_OUT_OF_RANGE, skip=(page,))


def test_no_page_has_a_place():
    c = Case([310], [14], 14, Hkv=1, G=4, seed=6)
    c.table.fill_(-1)
    c.call()
    torch.cuda.synchronize()
    assert int(c.err) == kvmm.ERR_NULL_BLOCK
    assert (c.out == 0).all() and torch.isneginf(c.lse).all()


def test_impossible_selections():
    c = Case([310], [3], 3, Hkv=1, G=4, K=6, seed=6)
    c.sel[0, 0, 0] = torch.tensor([0, 5, 20, -1, 7, 1 << 30], dtype=torch.int32)
    c.cnt.fill_(6)
    c.call()
    c.check(err=kvmm.ERR_OUT_OF_RANGE)  # (20 is a page of nodes, not of settled tokens; the plain form finds no token there)
    c = Case([310], [3], 3, Hkv=1, G=4, K=6, seed=6)
    c.cnt.fill_(-5)
    c.call()
    c.cnt.fill_(0)
    c.check(err=kvmm.ERR_OUT_OF_RANGE)
    c = Case([310], [3], 3, Hkv=1, G=4, K=6, seed=6)
    c.cnt.fill_(99)
    c.call()
    c.cnt.fill_(6)
    c.check(err=kvmm.ERR_OUT_OF_RANGE)


def test_impossible_lengths():
    c = Case([310, 20], [3, 5], 5, Hkv=1, seed=6)
    c.seq[1] = -9
    c.n_nodes[0] = -2
    c.call()
    torch.cuda.synchronize()
    assert int(c.err) == kvmm.ERR_OUT_OF_RANGE
    assert (c.out[0] == 7.0).all() and not (c.out[1, :5] == 7.0).all() and not c.out[1].isnan().any()
    c = Case([310, 20], [5, 5], 5, Hkv=1, seed=6)
    c.n_nodes[0] = 6  # as 5
    c.call()
    c.check(err=kvmm.ERR_OUT_OF_RANGE)
    c = Case([256, 20], [5, 5], 5, Pmax=16, Hkv=1, seed=6)
    c.seq[0] = 300  # as 256: no node has a place
    c.call()
    c.check(err=kvmm.ERR_OUT_OF_RANGE)


def test_stream_and_graph():
    """On another stream, and captured: replays with changed inputs, beside eager calls with a workspace of their own."""
    c = Case([1500, 33], [8, 6], 8, Hkv=2, D=128, seed=12)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.call(stream=side)
    side.synchronize()
    c.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call()
    other = Case([700], [5], 5, Hkv=2, D=128, seed=13)
    c.q.copy_(c.q.flip(0))
    c.out.fill_(7)
    c.lse.fill_(7)
    g.replay()
    other.call()
    g.replay()
    c.check()
    other.check()


def test_two_calls_at_once():
    """Two streams with a workspace each."""
    cs = [Case([9000, 100], [8, 8], 8, Hkv=4, D=128, seed=s) for s in (21, 22)]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, s in zip(cs, streams):
            c.call(stream=s)
    for c in cs:
        c.check()


def test_the_same_bits_every_time():
    c = Case([9000, 1200, 40], [16, 16, 3], 16, Hkv=4, D=128, seed=30)
    c.call()
    out, lse = c.out.clone(), c.lse.clone()
    for _ in range(5):
        c.ws.random_(0, 255)
        c.call()
        assert torch.equal(out, c.out) and torch.equal(lse, c.lse)
    c.check()


def test_pool_beyond_32_bit_offsets():
    """Pages whose byte offsets pass 2^32 and whose element offsets pass 2^31."""
    c = Case([200], [6], 6, Hkv=1, G=4, D=128, seed=31)
    n_phys = (1 << 31) // (16 * 128) + 40
    k = torch.zeros(n_phys, 16, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros(n_phys, 128, 16, dtype=torch.bfloat16, device="cuda")
    old = c.table.view(-1).long()
    new = n_phys - 1 - torch.arange(old.numel(), device="cuda")
    k[new], v[new] = c.k_pool[old], c.v_pool[old]
    c.k_pool, c.v_pool, c.table = k, v, new.to(torch.int32).view(c.table.shape)
    c.shape.n_phys = n_phys
    c.call()
    c.check()


@pytest.mark.parametrize("n,G", [(6, 4), (40, 8), (64, 8)])
@pytest.mark.parametrize("K", [0, 12])
@pytest.mark.parametrize("lens", [[500], [500, 3, 0, 129, 900], [60] * 37])
def test_short_sequences_of_a_long_table(lens, n, G, K):
    """A table for far longer sequences: the blocks are dealt to the SMs where a table of their length has clusters."""
    for Pmax in (None, 6000):
        c = Case(lens, [n] * len(lens), n, Hkv=2, G=G, D=64, K=K, seed=40, Pmax=Pmax)
        if K and Pmax:  # and selections far shorter than their list may be
            wide = torch.zeros(c.B, 1, 2, 4000, dtype=torch.int32, device="cuda")
            wide[..., :K] = c.sel
            c.sel, c.shape.Kmax = wide, 4000
        c.call()
        c.check()


def test_more_units_than_one_launch_takes():
    c = Case([(5 * b) % 90 for b in range(300)], [1 + b % 3 for b in range(300)], 3, Hkv=8, G=1, D=64, seed=41, Pmax=7)
    c.call()
    c.check()


def test_a_batch_of_nothing_but_empty_rows():
    """Selections of no page and nodes without a place: zeros and -inf, whichever way the units are taken."""
    for Pmax, B in ((16, 1), (16, 90), (2000, 3)):
        c = Case([Pmax * 16] * B, [3] * B, 3, Hkv=2, G=4, D=64, seed=42, Pmax=Pmax, K=2)
        c.cnt.zero_()
        c.call()
        torch.cuda.synchronize()
        assert int(c.err) == kvmm.ERR_OUT_OF_RANGE
        assert (c.out == 0).all() and torch.isneginf(c.lse).all()


def test_nan_in_a_query_stays_in_its_row():
    for lens in ([300], [40000]):
        c = Case(lens, [5], 5, Hkv=1, G=4, D=64, seed=43)
        c.call()
        want = c.out.clone()
        c.q[0, 2, 1, 7] = math.nan
        c.call()
        torch.cuda.synchronize()
        assert c.out[0, 2, 1].isnan().all() and c.lse[0, 2, 1].isnan()
        want[0, 2, 1] = c.out[0, 2, 1] = 0
        assert torch.equal(want, c.out)


def test_refusals():
    c = Case([20], [4], 4, Hkv=1, seed=1)
    for kw, what in ((dict(tree_mask=c.mask[:, :3]), "tree_mask"), (dict(lse=c.lse[:, :3]), "lse"),
                     (dict(sel_idx=c.table), "together"), (dict(n_nodes=c.n_nodes.long()), "n_nodes"),
                     (dict(tree_mask=c.mask.int()), "tree_mask")):
        with pytest.raises(ValueError, match=what):
            c.call(**kw)
    with pytest.raises(ValueError, match="out"):
        kvmm.sparse_paged_tree_attn(c.shape, 0, c.q, c.k_pool, c.v_pool, c.table, c.seq, c.out[:, :3], c.ws)
    with pytest.raises(ValueError, match="q"):
        kvmm.sparse_paged_tree_attn(c.shape, 0, c.q[0], c.k_pool, c.v_pool, c.table, c.seq, c.out, c.ws)
    with pytest.raises(kvmm.KvmmError, match="workspace"):
        kvmm.sparse_paged_tree_attn(c.shape, 0, c.q, c.k_pool, c.v_pool, c.table, c.seq, c.out, c.ws[:8])
