"""The 4-bit cache read back (kv4_gather) and attended over (sparse_paged_decode_attn_kv4), against numpy in 64 bits,
and a run of the operators together through the runtime's decode state."""
import math

import numpy as np
import pytest
import torch

from paged_kv_cache_minmax_gb300 import kvmm
from paged_kv_cache_minmax_gb300.runtime import DecodeState, Kv4DecodeState
from tests import kv4_plain as kp

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    from paged_kv_cache_minmax_gb300 import build

    build.build_library()
    kvmm.load()
    yield
    torch.cuda.empty_cache()


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class Cache:
    """A 4-bit pool of random codes and scales, sequences of given lengths, a permuted table."""

    def __init__(self, seq, Hq=8, Hkv=2, D=64, T=16, L=2, layer=1, Pmax=None, Kmax=4, seed=0, scales=(0x20, 0x48)):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.seq, self.B, self.Hq, self.Hkv, self.D, self.T, self.L, self.layer = list(seq), len(seq), Hq, Hkv, D, T, L, layer
        self.Pmax = Pmax or max(1, -(-max(seq) // T))
        self.n_phys = self.B * L * Hkv * self.Pmax + 2
        self.shape = kvmm.make_shape(self.B, L, Hq, Hkv, D, T, self.Pmax, Kmax, self.n_phys)
        n = self.B * L * Hkv * self.Pmax
        self.table = torch.randperm(self.n_phys, generator=g, device="cuda")[:n].to(torch.int32).view(
            self.B, L, Hkv, self.Pmax).contiguous()
        self.pool = torch.randint(0, 256, (self.n_phys, kvmm.kv4_page_bytes(self.shape)), generator=g, device="cuda",
                                  dtype=torch.uint8)
        o = kp.offsets(T, D)
        for i in (1, 3):
            self.pool[:, o[i]:o[i + 1]] = torch.randint(*scales, (self.n_phys, o[i + 1] - o[i]), generator=g,
                                                        device="cuda", dtype=torch.uint8)
        self.seq_len = torch.tensor(self.seq, dtype=torch.int32, device="cuda")
        self.q = torch.randn(self.B, Hq, D, generator=g, device="cuda").to(torch.bfloat16)
        self.out = torch.full((self.B, Hq, D), 7.0, device="cuda")
        self.lse = torch.full((self.B, Hq), 7.0, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = kvmm.alloc_kv4_workspace(self.shape)
        self.ws[1024:] = 0xFF  # NaN behind the counters: nothing of it may be read before it is written
        self.sel = self.cnt = None

    def spoil_behind(self):
        """What pages hold behind a sequence's last token: codes and scales of every bit pattern, NaN among them."""
        o = kp.offsets(self.T, self.D)
        for b, s in enumerate(self.seq):
            if s % self.T:
                for h in range(self.Hkv):
                    page = self.pool[int(self.table[b, self.layer, h, s // self.T])]
                    for i, w in ((0, self.D // 2), (1, self.D // 16), (2, self.D // 2), (3, self.D // 16)):
                        page[o[i] + (s % self.T) * w:o[i + 1]] = 0xFF if i % 2 else 0x9C

    def select(self, K, seed=1, cnt=None):
        """K random pages of every unit, ascending."""
        rng = np.random.default_rng(seed)
        self.shape = kvmm.make_shape(self.B, self.L, self.Hq, self.Hkv, self.D, self.T, self.Pmax, K, self.n_phys)
        sel = np.full((self.B, self.L, self.Hkv, K), -5, dtype=np.int32)
        n = np.zeros((self.B, self.L, self.Hkv), dtype=np.int32)
        for b in range(self.B):
            P = -(-self.seq[b] // self.T)
            for h in range(self.Hkv):
                m = min(P, K if cnt is None else cnt[b * self.Hkv + h])
                sel[b, self.layer, h, :m] = np.sort(rng.permutation(P)[:m])
                n[b, self.layer, h] = m
        self.sel, self.cnt = torch.from_numpy(sel).cuda(), torch.from_numpy(n).cuda()

    def rows(self, b, h, pages=None):
        """Keys and values [n, D] float64 (without factors) of the given logical pages (all), valid tokens only."""
        pool = getattr(self, "_np", None)
        if pool is None:
            pool = self._np = self.pool.cpu().numpy()
            self._tab = self.table.cpu().numpy()
        ks, vs = [], []
        for p in range(-(-self.seq[b] // self.T)) if pages is None else pages:
            phys = self._tab[b, self.layer, h, p]
            if not 0 <= phys < self.n_phys:
                continue
            n = min(self.T, self.seq[b] - p * self.T)
            for out, values in ((ks, False), (vs, True)):
                out.append(kp.value(*(x[:n] for x in kp.page_rows(pool[phys], self.T, self.D, values))))
        empty = np.zeros((0, self.D))
        return np.concatenate(ks + [empty]), np.concatenate(vs + [empty])

    def attend(self, **kw):
        kvmm.sparse_paged_decode_attn_kv4(self.shape, self.layer, self.q, self.pool, self.table, self.seq_len, self.sel,
                                          self.cnt, self.out, self.ws, lse=self.lse, err=self.err, **kw)

    def check(self, k_scale=1.0, v_scale=1.0, sm_scale=None, units=None):
        G = self.Hq // self.Hkv
        sm = sm_scale or 1 / math.sqrt(self.D)
        out, lse, q = f64(self.out), f64(self.lse), f64(self.q)
        for b in range(self.B):
            for h in range(self.Hkv):
                if units is not None and (b, h) not in units:
                    continue
                pages = None
                if self.sel is not None:
                    pages = self.sel[b, self.layer, h, :int(self.cnt[b, self.layer, h])].cpu().numpy()
                k, v = self.rows(b, h, pages)
                g = slice(h * G, (h + 1) * G)
                want, wl, zsum = kp.unit_attention(q[b, g], k * k_scale, v * v_scale, sm)
                if k.shape[0] == 0:
                    assert (out[b, g] == 0).all() and (lse[b, g] == -np.inf).all(), (b, h)
                    continue
                tol = kp.out_tolerance(self.D, zsum, np.abs(v * v_scale).max())
                assert np.abs(out[b, g] - want).max() <= tol, (b, h, np.abs(out[b, g] - want).max(), tol)
                assert (np.abs(lse[b, g] - wl) <= kp.lse_tolerance(self.D, zsum, wl)).all(), (b, h)


# ---- gather ---------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("D,T", [(64, 16), (64, 32), (128, 16), (128, 32)])
@pytest.mark.parametrize("k_scale,v_scale", [(1.0, 1.0), (0.37, 3.0)])
def test_gather_is_exact(D, T, k_scale, v_scale):
    c = Cache([70, 1, 0, 33, 96], D=D, T=T, Hkv=3, Hq=3, scales=(0, 0x7F))
    begin, end, n = [5, 0, 0, 32, 60], [70, 1, 0, 33, 92], 66
    tb, te = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (begin, end))
    k, v = (torch.full((5, n, 3, D), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kvmm.kv4_gather(c.shape, 1, c.pool, c.table, tb, te, k, v, k_scale=k_scale, v_scale=v_scale, err=c.err)
    torch.cuda.synchronize()
    assert int(c.err) == 0
    for b in range(5):
        m = end[b] - begin[b]
        assert (f64(k[b, m:]) == 9.0).all() and (f64(v[b, m:]) == 9.0).all()
        for h in range(3):
            kk, vv = c.rows(b, h)
            assert np.array_equal(f64(k[b, :m, h]), kp.bf16(kp.f32(kk[begin[b]:end[b]] * float(np.float32(k_scale)))))
            assert np.array_equal(f64(v[b, :m, h]), kp.bf16(kp.f32(vv[begin[b]:end[b]] * float(np.float32(v_scale)))))


def test_gather_from_the_start_one_side_and_bad_ranges():
    c = Cache([40, 40], Pmax=3)
    te = torch.tensor([40, 17], dtype=torch.int32, device="cuda")
    k = torch.full((2, 40, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    kvmm.kv4_gather(c.shape, 1, c.pool, c.table, None, te, k, None, err=c.err)
    v = torch.full((2, 40, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    kvmm.kv4_gather(c.shape, 1, c.pool, c.table, None, te, None, v, err=c.err)
    torch.cuda.synchronize()
    assert int(c.err) == 0
    for b, n in ((0, 40), (1, 17)):
        kk, vv = c.rows(b, 1)
        assert np.array_equal(f64(k[b, :n, 1]), kk[:n]) and np.array_equal(f64(v[b, :n, 1]), vv[:n])
        assert (f64(k[b, n:]) == 9.0).all()
    # longer than the rows: cut; outside the table: cut; a null page: its rows are left
    c.table[1, 1, 0, 1] = -1
    for te_, tb_, want in (([40, 30], None, kvmm.ERR_OUT_OF_RANGE | kvmm.ERR_NULL_BLOCK), ([49, 30], [44, 28],
                                                                                        kvmm.ERR_OUT_OF_RANGE | kvmm.ERR_NULL_BLOCK),
                           ([3, 2], [5, 1], kvmm.ERR_OUT_OF_RANGE), ([3, 2], [-4, 1], kvmm.ERR_OUT_OF_RANGE)):
        c.err.zero_()
        k = torch.full((2, 20, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda")
        te = torch.tensor(te_, dtype=torch.int32, device="cuda")
        tb = None if tb_ is None else torch.tensor(tb_, dtype=torch.int32, device="cuda")
        kvmm.kv4_gather(c.shape, 1, c.pool, c.table, tb, te, k, None, err=c.err)
        torch.cuda.synchronize()
        assert int(c.err) == want, (te_, tb_)
        for b in range(2):
            lo = max(0, tb_[b] if tb_ else 0)
            hi = min(te_[b], 48, lo + 20)
            got = f64(k[b])
            for j in range(20):
                for h in range(2):
                    t = lo + j
                    if t < hi and not (b == 1 and h == 0 and t // 16 == 1):
                        cc = kp.value(*(x[t % 16:t % 16 + 1] for x in kp.page_rows(
                            c.pool[int(c.table[b, 1, h, t // 16])].cpu().numpy(), 16, 64, False)))[0]
                        assert np.array_equal(got[j, h], cc), (b, j, h)
                    else:
                        assert (got[j, h] == 9.0).all(), (b, j, h)


# ---- attention ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 7, 8])
@pytest.mark.parametrize("D,T", [(64, 16), (64, 32), (128, 16), (128, 32)])
def test_every_page_of_ragged_sequences(D, T, G):
    c = Cache([1, 0, T - 1, T, T + 1, 5 * T + 3, 200], Hq=2 * G, D=D, T=T)
    c.spoil_behind()
    c.attend()
    torch.cuda.synchronize()
    assert int(c.err) == 0
    c.check()


@pytest.mark.parametrize("G", [1, 4, 6, 8])
@pytest.mark.parametrize("D,T", [(64, 16), (64, 32), (128, 16), (128, 32)])
def test_selected_pages(D, T, G):
    c = Cache([777, 300, 31, 0, 16 * T], Hq=3 * G, Hkv=3, D=D, T=T, L=1, layer=0)
    c.spoil_behind()
    c.select(9, cnt=[9, 1, 5, 9, 9, 0, 1, 1, 0, 0, 0, 0, 9, 3, 2])
    c.attend(k_scale=0.3, v_scale=2.5, sm_scale=0.2)
    torch.cuda.synchronize()
    assert int(c.err) == 0
    c.check(k_scale=float(np.float32(0.3)), v_scale=2.5, sm_scale=float(np.float32(0.2)))


@pytest.mark.parametrize("G", [4, 5])
def test_one_long_sequence_falls_on_every_cta(G):
    """Few units, one long axis: every unit is merged from many CTAs' parts."""
    c = Cache([40003], Hq=2 * G, Hkv=2, D=128, L=1, layer=0)
    c.attend()
    torch.cuda.synchronize()
    assert int(c.err) == 0
    c.check()
    # every page selected: the same values through a cluster a unit
    c.out.zero_(), c.lse.zero_()
    c.select(c.Pmax)
    c.attend()
    torch.cuda.synchronize()
    assert int(c.err) == 0
    c.check()


@pytest.mark.parametrize("G,T", [(4, 16), (5, 32)])
def test_long_sequences_are_dealt_evenly(G, T):
    """Longer than a cluster a unit is taken for: pieces that hold parts of units, whole ones and empty ones."""
    c = Cache([70003, 3, 0, 33000], Hq=2 * G, Hkv=2, D=64, T=T, L=1, layer=0, Pmax=-(-70003 // T) + 9)
    c.spoil_behind()
    for _ in range(2):  # the counters are back at zero
        c.out.fill_(5.0)
        c.attend(v_scale=0.5)
        torch.cuda.synchronize()
        assert int(c.err) == 0
        c.check(v_scale=0.5)
    assert int(c.ws[:1024].max()) == 0


@pytest.mark.parametrize("G", [1, 4, 5, 8])
@pytest.mark.parametrize("D,T", [(64, 16), (64, 32), (128, 16), (128, 32)])
def test_ragged_sequences_share_clusters(D, T, G):
    """A cluster of several CTAs a unit over every page: lengths that leave most of its CTAs, or all, without a page."""
    c = Cache([2001, 0, 1, 777, 16 * T, 1234], Hq=2 * G, Hkv=2, D=D, T=T, L=1, layer=0)
    c.spoil_behind()
    c.table[0, 0, 1, 2:5] = -1
    c.attend(early_reads=G == 4)
    torch.cuda.synchronize()
    assert int(c.err) == kvmm.ERR_NULL_BLOCK
    c.check()


@pytest.mark.parametrize("K", [1, 16, 17, 47, 130, 300])
@pytest.mark.parametrize("B,Hkv,G,D,T", [(1, 1, 8, 128, 16), (1, 3, 1, 64, 16), (3, 2, 5, 128, 32), (7, 5, 4, 64, 32)])
def test_clusters_of_every_size(K, B, Hkv, G, D, T):
    """Few units: the more places a unit has, the more CTAs share it; counts below Kmax leave some of them idle."""
    c = Cache([4000 - 900 * (b % 4) for b in range(B)], Hq=Hkv * G, Hkv=Hkv, D=D, T=T, L=1, layer=0)
    rng = np.random.default_rng(K)
    c.select(K, cnt=[int(x) for x in rng.integers(0, K + 1, B * Hkv)])
    c.attend()
    torch.cuda.synchronize()
    assert int(c.err) == 0
    c.check()


@pytest.mark.parametrize("Pmax", [40, 1000, 32768])
def test_short_sequences_in_a_long_table(Pmax):
    """Far fewer pages than the table has room for: fewer than the CTAs launched, too."""
    c = Cache([70, 1, 0, 150], Hkv=2, Hq=8, D=64, L=1, layer=0, Pmax=Pmax)
    for _ in range(2):  # the counters are back at zero
        c.out.fill_(5.0)
        c.attend()
        torch.cuda.synchronize()
        assert int(c.err) == 0
        c.check()
    assert int(c.ws[:1024].max()) == 0
    d = Cache([17], Hkv=1, Hq=8, D=128, L=1, layer=0, Pmax=Pmax)
    d.attend()
    torch.cuda.synchronize()
    d.check()


def test_selections_of_more_units_than_sms():
    """320 units: the selected pages of all are dealt evenly."""
    rng = np.random.default_rng(5)
    c = Cache([int(x) for x in rng.integers(0, 700, 40)], Hq=24, Hkv=8, D=64, L=1, layer=0)
    c.select(20, cnt=[int(x) for x in rng.integers(0, 21, 320)])
    c.attend()
    torch.cuda.synchronize()
    assert int(c.err) == 0
    c.check()


def test_more_units_than_one_launch_takes():
    """2,600 units of 0 to 3 pages: two launches, many units a CTA, most of them whole."""
    B, Hkv = 325, 8
    rng = np.random.default_rng(0)
    c = Cache([int(x) for x in rng.integers(0, 49, B)], Hq=16, Hkv=Hkv, L=1, layer=0, Pmax=3)
    c.attend()
    torch.cuda.synchronize()
    assert int(c.err) == 0
    c.check()


def test_all_empty():
    c = Cache([0, 0], Pmax=4)
    c.attend()
    torch.cuda.synchronize()
    assert int(c.err) == 0
    c.check()
    c.select(3)
    c.out.fill_(3.0)
    c.attend()
    torch.cuda.synchronize()
    assert int(c.err) == 0
    c.check()


def test_large_scores_and_wide_values():
    """Scores of hundreds, scales over e4m3's whole range, queries over bf16's: the reference is raised often, and
    most probabilities vanish."""
    c = Cache([600, 333], D=128, Hq=8, scales=(0, 0x7F), seed=4)
    c.q = (c.q.float() * torch.exp2(torch.randint(-12, 3, c.q.shape, device="cuda").float())).to(torch.bfloat16)
    for sm in (1e-4, 0.002):
        c.attend(sm_scale=sm)
        torch.cuda.synchronize()
        assert int(c.err) == 0
        c.check(sm_scale=float(np.float32(sm)))


def test_zero_and_tiny_queries():
    c = Cache([100, 50])
    c.q[0] = 0
    c.q[1] = 1e-38
    c.attend()
    torch.cuda.synchronize()
    c.check()


def test_invalid_entries_are_reported_and_skipped():
    c = Cache([300, 300], T=16)
    c.table[0, 1, 0, 3] = -1
    c.attend()
    torch.cuda.synchronize()
    assert int(c.err) == kvmm.ERR_NULL_BLOCK
    c.check()
    c.err.zero_()
    c.table[1, 1, 1, 0] = c.n_phys
    c.__dict__.pop("_np")
    c.attend()
    torch.cuda.synchronize()
    assert int(c.err) == kvmm.ERR_NULL_BLOCK | kvmm.ERR_OUT_OF_RANGE
    c.check()
    # a unit none of whose pages can be read
    c.err.zero_()
    c.table[0, 1, 1] = -1
    c.__dict__.pop("_np")
    c.attend()
    torch.cuda.synchronize()
    c.check()
    # selections outside the sequence, counts outside the list, lengths outside the table
    d = Cache([300, 300])
    d.select(4)
    d.sel[0, 1, 0, 3] = 19
    d.sel[0, 1, 1, 0] = -2
    d.attend()
    torch.cuda.synchronize()
    assert int(d.err) == kvmm.ERR_OUT_OF_RANGE
    keep = d.sel.clone()
    d.check(units=[(1, 0), (1, 1)])
    d.sel, d.cnt[0, 1, 0] = keep, 3
    d.check(units=[(0, 0)])
    d.sel = keep[..., 1:].contiguous()
    d.cnt[0, 1, 1] = 3
    d.check(units=[(0, 1)])
    e = Cache([300, 300])
    e.select(4)
    e.cnt[1, 1, 0], e.cnt[1, 1, 1] = 5, -1
    e.attend()
    torch.cuda.synchronize()
    assert int(e.err) == kvmm.ERR_OUT_OF_RANGE
    e.cnt[1, 1, 0], e.cnt[1, 1, 1] = 4, 0
    e.check()
    f = Cache([300, 304], Pmax=19)
    f.seq_len[1] = 9999
    f.seq_len[0] = -3
    f.attend()
    torch.cuda.synchronize()
    assert int(f.err) == kvmm.ERR_OUT_OF_RANGE
    f.seq = [0, 304]
    f.check()


def test_pages_beyond_32_bits():
    """Pages more than 2^32 bytes into the pool: the bits of a small pool's."""
    c = Cache([700, 333], D=128, T=32, Hq=8)
    c.attend()
    n_phys = (5 << 30) // c.pool.shape[1]
    far = n_phys - c.n_phys
    pool = torch.empty(n_phys, c.pool.shape[1], dtype=torch.uint8, device="cuda")
    pool[far:] = c.pool
    shape = kvmm.make_shape(c.B, c.L, c.Hq, c.Hkv, c.D, c.T, c.Pmax, 4, n_phys)
    out = torch.zeros_like(c.out)
    kvmm.sparse_paged_decode_attn_kv4(shape, 1, c.q, pool, c.table + far, c.seq_len, None, None, out, c.ws, err=c.err)
    rows = [torch.zeros(2, 700, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    kvmm.kv4_gather(c.shape, 1, c.pool, c.table, None, c.seq_len, rows[0], None, err=c.err)
    kvmm.kv4_gather(shape, 1, pool, c.table + far, None, c.seq_len, rows[1], None, err=c.err)
    torch.cuda.synchronize()
    assert int(c.err) == 0
    assert torch.equal(out, c.out) and torch.equal(*rows)


@pytest.mark.parametrize("every", [False, True])
def test_padded_batch_and_repeated_pages(every):
    """Entries without a token, whose table rows and selections hold anything, and table rows behind a sequence's last
    page; a page that is selected twice, or that two sequences share, counts for each."""
    c = Cache([0, 100, 0, 100, 0], Pmax=40)
    c.table[1::2, :, :, 7:] = 0x7FFFFFFF
    c.table[0::2] = -0x80000000
    c.table[3, 1, :, :4] = c.table[1, 1, :, :4]  # a shared prefix
    if not every:
        c.select(5)
        c.sel[0::2] = 0x7FFFFFFF
        c.sel[1, 1, 0, :5] = torch.tensor([2, 2, 6, 6, 6], dtype=torch.int32)
    c.attend()
    torch.cuda.synchronize()
    assert int(c.err) == 0
    c.check()


def test_without_lse_and_error_word():
    c = Cache([300, 40])
    c.attend()
    out = c.out.clone()
    kvmm.sparse_paged_decode_attn_kv4(c.shape, 1, c.q, c.pool, c.table, c.seq_len, None, None, c.out.zero_(), c.ws)
    torch.cuda.synchronize()
    assert torch.equal(out, c.out)


def test_graphs_streams_and_two_calls_at_once():
    """Captured and replayed with new inputs in the same buffers; two calls on two streams with their own workspaces."""
    c = Cache([5000, 3000], D=128, Hq=8)
    d = Cache([4000, 100], D=128, Hq=10, seed=9)
    c.attend()
    d.attend()
    torch.cuda.synchronize()
    want_c, want_d = c.out.clone(), d.out.clone()
    c.out.zero_(), d.out.zero_()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        c.attend(stream=s1)
        d.attend(stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(c.out, want_c) and torch.equal(d.out, want_d)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.attend()
        c.attend()
    c.out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.out, want_c)
    c.q.copy_(torch.randn_like(c.q.float()))
    c.seq_len.copy_(torch.tensor([77, 4999], dtype=torch.int32))
    c.table.copy_(c.table.flip(0))  # another sequence's pages
    c.seq = [77, 4999]
    c.__dict__.pop("_np", None)
    graph.replay()
    torch.cuda.synchronize()
    assert int(c.err) == 0
    c.check()


def test_early_reads_give_the_same_bits():
    c = Cache([5000, 3000, 17], D=128, Hq=8)
    for sel in (False, True):
        if sel:
            c.select(40)
        c.attend()
        torch.cuda.synchronize()
        want = c.out.clone()
        for _ in range(3):
            c.out.zero_()
            c.attend(early_reads=True)
            c.attend(early_reads=True)
        torch.cuda.synchronize()
        assert torch.equal(c.out, want)


@pytest.mark.parametrize("seq,Hkv,T", [([70000, 0, 1200], 2, 16), ([70000, 40000], 2, 32), ([50, 0, 333, 17] * 50, 2, 16)])
def test_units_across_ctas_early_captured_and_on_two_streams(seq, Hkv, T):
    """Pages dealt evenly: early reads, two calls at once with their own workspaces, and a captured pair of calls
    replayed with other lengths, all give the bits of a call by itself."""
    c, d = (Cache(seq, Hq=Hkv * G, Hkv=Hkv, D=64, T=T, L=1, layer=0, seed=G, Pmax=4500) for G in (4, 7))
    want = []
    for x in (c, d):
        x.attend()
        torch.cuda.synchronize()
        x.check(units={(b, h) for b in list(range(8)) + [len(seq) - 1] for h in range(Hkv)})
        want.append((x.out.clone(), x.lse.clone()))
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for early in (False, True):
        for x in (c, d):
            x.out.fill_(3.0), x.lse.fill_(3.0)
        torch.cuda.synchronize()
        for _ in range(4):
            c.attend(stream=streams[0], early_reads=early)
            d.attend(stream=streams[1], early_reads=early)
        torch.cuda.synchronize()
        for x, (out, lse) in zip((c, d), want):
            assert int(x.err) == 0
            assert torch.equal(x.out, out) and torch.equal(x.lse, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.attend(early_reads=True)
        c.attend()
    other = [(7 * n + 11) % (max(seq) + 1) for n in seq]
    for lengths in (other, seq, [0] * len(seq), seq):
        c.seq_len.copy_(torch.tensor(lengths, dtype=torch.int32))
        c.out.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert int(c.err) == 0
        if lengths is seq:
            assert torch.equal(c.out, want[0][0]) and torch.equal(c.lse, want[0][1])
        c.seq = lengths
        c.check(units={(b, h) for b in range(min(3, len(seq))) for h in range(Hkv)})
        c.seq = list(seq)
    assert int(c.ws[:1024].max()) == 0


def test_early_reads_behind_an_append():
    """The append writes the pool, not the lengths or the table: the attention behind it may read those early."""
    D, T, Hkv, B = 128, 16, 2, 3
    c = Cache([900, 333, 17], D=D, T=T, Hq=8, Hkv=Hkv, L=1, layer=0, Pmax=60)
    g = torch.Generator(device="cuda").manual_seed(0)
    rows = torch.randn(20, 2, B, 1, Hkv, D, generator=g, device="cuda").to(torch.bfloat16)
    begin = c.seq_len - 1
    outs = []
    for early in (False, True):
        got = []
        for i in range(20):
            kvmm.kv4_append_rope(c.shape, 0, None, rows[i, 0], rows[i, 1], begin, c.seq_len, c.pool, c.table, None,
                                 err=c.err)
            c.attend(early_reads=early)
            got.append(c.out.clone())
        outs.append(torch.stack(got))
    torch.cuda.synchronize()
    assert int(c.err) == 0
    assert torch.equal(outs[0], outs[1])
    c.check()


# ---- the operators together -----------------------------------------------------------------------------------
def rope_table(rows, dim):
    ang = torch.arange(rows, dtype=torch.float64)[:, None] * 10000.0 ** (
        -2.0 * torch.arange(dim // 2, dtype=torch.float64) / dim)
    return torch.stack([ang.cos(), ang.sin()], 1).float().cuda()


@pytest.mark.parametrize("D,T,Hq,Hkv", [(128, 16, 8, 2), (64, 32, 10, 2)])
def test_prompt_then_decode_steps_in_four_bits(D, T, Hq, Hkv):
    """A ragged prompt, then decode steps: the selection is the top of the scores over the held keys' bounds, the
    attention is that of the held values, and reading the cache back gives those values."""
    B, K, steps, k_scale, v_scale = 3, 6, 5, 1.5, 0.4
    lens = [230, 97, 0]
    Pmax = -(-(max(lens) + steps) // T)
    g = torch.Generator(device="cuda").manual_seed(2)
    n_phys = B * Hkv * Pmax
    table = torch.randperm(n_phys, generator=g, device="cuda").to(torch.int32).view(B, 1, Hkv, Pmax)
    rope = kvmm.Rope(rope_table(Pmax * T, D), D)
    seq_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    pool = torch.zeros(n_phys, T * (D + D // 8), dtype=torch.uint8, device="cuda")
    st = Kv4DecodeState(B, 1, Hq, Hkv, D, T, Pmax, K, pool, table, seq_len, k_scale=k_scale, v_scale=v_scale)
    n = max(lens)
    x = torch.randn(B, n, Hq + 2 * Hkv, D, generator=g, device="cuda").to(torch.bfloat16)
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    st.append_prompt(0, x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], zero, seq_len, rope=rope)
    angles = f64(rope.table)
    held = [[None] * Hkv for _ in range(B)]

    def turn(rows, pos):
        t = angles[pos]
        return kp.rotate(f64(rows), t[:, 0][:, None], t[:, 1][:, None], D, False)

    hold = lambda r, s: kp.value(*kp.hold(r, s))  # noqa: E731
    for b in range(B):
        k = hold(turn(x[b, :lens[b], Hq:Hq + Hkv], np.arange(lens[b])), k_scale)
        v = hold(f64(x[b, :lens[b], Hq + Hkv:]), v_scale)
        for h in range(Hkv):
            held[b][h] = [k[:, h], v[:, h]]
    for step in range(steps):
        seq_len += (seq_len > 0).int()
        y = torch.randn(B, Hq + 2 * Hkv, D, generator=g, device="cuda").to(torch.bfloat16)
        st.layer_step_rope(0, y[:, :Hq], y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:], rope)
        scores = torch.zeros(B, Hkv, Pmax, device="cuda")
        st.select(0, st.q_turned[0], scores_out=scores)
        torch.cuda.synchronize()
        assert st.read_err() == 0
        for b in range(B):
            s = int(seq_len[b])
            P = -(-s // T)
            G = Hq // Hkv
            if s == 0:
                assert (f64(st.out[0, b]) == 0).all() and int(st.sel_cnt[b, 0].max()) == 0
                continue
            q = kp.bf16(turn(y[b:b + 1, :Hq], np.array([s - 1])))[0]
            assert np.array_equal(f64(st.q_turned[0, b]), q)
            for h in range(Hkv):
                kk, vv = held[b][h]
                kk = np.concatenate([kk, hold(turn(y[b:b + 1, Hq:Hq + Hkv], np.array([s - 1]))[0, h:h + 1], k_scale)])
                vv = np.concatenate([vv, hold(f64(y[b, Hq + Hkv + h]), v_scale)[None]])
                held[b][h] = [kk, vv]
                qg = q[h * G:(h + 1) * G]
                want = np.array([np.maximum(qg * kk[p * T:(p + 1) * T].min(0), qg * kk[p * T:(p + 1) * T].max(0)).sum()
                                 for p in range(P)])
                got = f64(scores[b, h, :P])
                assert np.abs(got - want).max() <= 1e-5 * np.abs(want).max()
                sel = st.sel_idx[b, 0, h, :int(st.sel_cnt[b, 0, h])].cpu().numpy()
                assert sel.tolist() == sorted(np.lexsort((np.arange(P), -got))[:K].tolist())
                tok = np.concatenate([np.arange(p * T, min(s, (p + 1) * T)) for p in sel])
                sm = 1 / math.sqrt(D)
                out, lse, zsum = kp.unit_attention(qg, kk[tok] * k_scale, vv[tok] * float(np.float32(v_scale)), sm)
                gs = slice(h * G, (h + 1) * G)
                assert np.abs(f64(st.out[0, b, gs]) - out).max() <= kp.out_tolerance(D, zsum, np.abs(vv[tok]).max() * v_scale)
                assert (np.abs(f64(st.lse[0, b, gs]) - lse) <= kp.lse_tolerance(D, zsum, lse)).all()
    st.attend(0, st.q_turned[0], every_page=True)
    rows = int(seq_len.max())
    k, v = (torch.zeros(B, rows, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    st.gather(0, k, v)
    torch.cuda.synchronize()
    assert st.read_err() == 0
    for b in range(B):
        s = int(seq_len[b])
        for h in range(Hkv):
            kk, vv = held[b][h]
            assert np.array_equal(f64(k[b, :s, h]), kp.bf16(kp.f32(kk * k_scale)))
            assert np.array_equal(f64(v[b, :s, h]), kp.bf16(kp.f32(vv * float(np.float32(v_scale)))))
            if s:
                q = f64(st.q_turned[0, b, h * (Hq // Hkv):(h + 1) * (Hq // Hkv)])
                out, _, zsum = kp.unit_attention(q, kk * k_scale, vv * float(np.float32(v_scale)), 1 / math.sqrt(D))
                assert np.abs(f64(st.out[0, b, h * (Hq // Hkv):(h + 1) * (Hq // Hkv)]) - out).max() <= kp.out_tolerance(
                    D, zsum, np.abs(vv).max() * v_scale)


def test_decode_step_from_projection_rows_in_bf16():
    """DecodeState.layer_step_rope leaves what layer_step leaves on rows turned beforehand."""
    from paged_kv_cache_minmax_gb300 import workloads

    cfg = workloads.scaled(workloads.CONFIGS[2], B=2, L=1, S=1000, K=16, n_planted=8, steps=2)
    a, b = (workloads.generate(cfg, device="cuda") for _ in range(2))
    sa, sb = DecodeState.for_workload(a), DecodeState.for_workload(b)
    sa.build_metadata()
    sb.build_metadata()
    rope = kvmm.Rope(rope_table(cfg.Pmax * cfg.T, cfg.D), cfg.D)
    y = torch.randn(2, cfg.Hq + 2 * cfg.Hkv, cfg.D, device="cuda").to(torch.bfloat16)
    q, k, v = y[:, :cfg.Hq], y[:, cfg.Hq:cfg.Hq + cfg.Hkv], y[:, cfg.Hq + cfg.Hkv:]
    sa.layer_step_rope(0, q, k, v, rope)
    t = f64(rope.table)[cfg.S - 1]
    turn = lambda x: torch.from_numpy(kp.bf16(kp.rotate(f64(x), t[0], t[1], cfg.D, False))).cuda().to(torch.bfloat16)  # noqa: E731
    sb.layer_step(0, turn(q), turn(k).unsqueeze(2), v.unsqueeze(2).contiguous())
    torch.cuda.synchronize()
    assert sa.read_err() == sb.read_err() == 0
    for x, z in ((a.k_pool, b.k_pool), (a.v_pool, b.v_pool), (sa.meta, sb.meta), (sa.sel_idx, sb.sel_idx),
                 (sa.sel_cnt, sb.sel_cnt), (sa.out, sb.out), (sa.promoted_cnt, sb.promoted_cnt)):
        assert torch.equal(x, z)
