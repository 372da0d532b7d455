"""The rotated appends and the 4-bit cache at the edges of their formats: values beyond a format's range, infinities,
NaN, signed zeros, and batches that take more than one launch."""
import math

import numpy as np
import pytest
import torch

from paged_kv_cache_minmax_gb300 import kvmm
from tests import kv4_plain as kp
from tests.test_gpu_append_rope import Case, check_four, fill_pool4
from tests.test_gpu_kv4 import Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    from paged_kv_cache_minmax_gb300 import build

    build.build_library()
    kvmm.load()
    yield
    torch.cuda.empty_cache()


def append4(c, pool, **kw):
    kvmm.kv4_append_rope(c.shape, c.layer, None, c.k, c.v, c.tb, c.te, pool, c.table, c.meta, rope=c.rope, err=c.err, **kw)
    torch.cuda.synchronize()
    assert int(c.err) == 0


# ---- values beyond the range ----------------------------------------------------------------------------------
@pytest.mark.parametrize("scales", [(1.0, 1.0), (0.5, 1e-38), (1e-38, 0.5), (3.0, 8.0)])
@pytest.mark.parametrize("D,T", [(64, 16), (128, 32)])
@pytest.mark.filterwarnings("ignore::RuntimeWarning")
def test_values_beyond_the_range_saturate(D, T, scales):
    """Infinities, and finite values that leave fp32 times 1 / factor: the scale is 448 and the code +-6."""
    c = Case(Hq=2, D=D, T=T, n=24, begin=(4, 9), end=(28, 33), rope="none", spread=3.0)
    g = np.random.default_rng(11)
    big = float(torch.finfo(torch.bfloat16).max)
    for rows in (c.k, c.v):
        for i in range(24):
            for h in range(2):
                rows[0, i, h, g.integers(D)] = [math.inf, -math.inf, big, -big][i % 4]
                if i % 5 == 0:  # both signs, and next to each other
                    rows[1, i, h, 16:18] = torch.tensor([-math.inf, math.inf])
                    rows[1, i, h, 40] = -big
    pool = fill_pool4(c)
    pool0, meta0 = pool.clone(), c.meta.clone()
    append4(c, pool, k_scale=scales[0], v_scale=scales[1])
    check_four(c, pool0, pool, meta0, *scales)


@pytest.mark.parametrize("rope", ["half", "pairs"])
@pytest.mark.filterwarnings("ignore::RuntimeWarning")
def test_rotations_beyond_the_range_saturate(rope):
    """Pairs whose rotation leaves fp32's range."""
    c = Case(Hq=2, n=24, begin=(4, 9), end=(28, 33), rope=rope)
    big = float(torch.finfo(torch.bfloat16).max)
    c.k.copy_(torch.where(c.k.float().abs() > 1, torch.copysign(torch.full_like(c.k, big), c.k), c.k))
    pool = fill_pool4(c)
    pool0, meta0 = pool.clone(), c.meta.clone()
    append4(c, pool)
    check_four(c, pool0, pool, meta0, 1.0, 1.0)


# ---- NaN ------------------------------------------------------------------------------------------------------
def value_bits(codes, scales):
    """bf16 bits of held values; 0x7fff where the scale is the NaN."""
    v = kp.value(codes, scales).astype(np.float32).view(np.uint32) >> 16
    return np.where(np.repeat(scales == 0x7F, 16, -1), 0x7FFF, v).astype(np.int64)


def ordered(bits):
    """bf16 bits -> integers in the order of the values (-0 below +0, NaN of either sign outermost)."""
    return np.where(bits & 0x8000, 0x7FFF - bits, bits)


def bounds_bits(bits):
    at = ordered(bits)
    take = lambda i: np.take_along_axis(bits, i[None], 0)[0]  # noqa: E731
    return np.stack([take(at.argmin(0)), take(at.argmax(0))])


def hold_nan(x, scale):
    """kp.hold, with the groups that have a NaN: scale 0x7f, codes 7."""
    bad = np.isnan(x).reshape(*x.shape[:-1], -1, 16).any(-1)
    codes, scales = kp.hold(np.where(np.isnan(x), 0.0, x), scale)
    return np.where(np.repeat(bad, 16, -1), 7, codes).astype(np.uint8), np.where(bad, 0x7F, scales).astype(np.uint8)


@pytest.mark.parametrize("D,T", [(64, 16), (64, 32), (128, 16), (128, 32)])
@pytest.mark.parametrize("payload", [0x7FC0, 0xFFC0, 0x7F81])
@pytest.mark.filterwarnings("ignore::RuntimeWarning")
def test_nan_stays_nan(D, T, payload):
    """A NaN, of either sign, alone or beside an infinity, makes its group's scale the NaN, and no other group's."""
    c = Case(Hq=2, D=D, T=T, n=24, begin=(4, 9), end=(28, 33), rope="none")
    nan = torch.tensor([payload], dtype=torch.int32).to(torch.int16).view(torch.bfloat16).cuda()
    rng = np.random.default_rng(D + T)
    for rows in (c.k, c.v):
        for b in range(2):
            for i in range(0, 24, 3):
                d = int(rng.integers(D))
                rows[b, i, i % 2, d:d + 1] = nan
                if i % 2:
                    rows[b, i, i % 2, d ^ 1] = math.inf
        rows[1, 5, 0] = nan  # a whole row
    pool = fill_pool4(c)
    want, meta0 = pool.cpu().numpy().copy(), c.meta.clone()
    append4(c, pool, k_scale=2.0, v_scale=0.37)
    want_m = meta0.view(torch.int16).cpu().numpy().astype(np.int64) & 0xFFFF
    k, v = (x.float().cpu().numpy().astype(np.float64) for x in (c.k, c.v))
    for b, tb, te in c.ranges():
        (kc, ks), (vc, vs) = hold_nan(k[b], 2.0), hold_nan(v[b], 0.37)
        for h in range(c.Hkv):
            row = c.table[b, c.layer, h].cpu().numpy()
            for t in range(tb, te):
                for side, (codes, scales) in enumerate(((kc, ks), (vc, vs))):
                    kp.put_row(want[row[t // T]], T, D, t % T, bool(side), codes[t - tb, h], scales[t - tb, h])
            for p in range(tb // T, -(-te // T)):
                held = value_bits(*kp.page_rows(want[row[p]], T, D, False))[:min(T, te - p * T)]
                want_m[b, c.layer, h, p] = bounds_bits(held)
    assert np.array_equal(pool.cpu().numpy(), want)
    assert np.array_equal(c.meta.view(torch.int16).cpu().numpy().astype(np.int64) & 0xFFFF, want_m)
    # read back: NaN in those groups, numbers elsewhere
    out = [torch.zeros(2, 24, 2, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    kvmm.kv4_gather(c.shape, c.layer, pool, c.table, c.tb, c.te, *out, k_scale=2.0, v_scale=0.37, err=c.err)
    torch.cuda.synchronize()
    assert int(c.err) == 0
    for x, got in zip((k, v), out):
        bad = np.repeat(np.isnan(x).reshape(2, 24, 2, -1, 16).any(-1), 16, -1)
        assert np.array_equal(torch.isnan(got).cpu().numpy(), bad)


# ---- signed zeros ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("rope", ["none", "half"])
def test_zeros_keep_their_signs(rope):
    """-0 is held as code 8 where its group's scale is not zero, as a negative value that rounds to zero is."""
    c = Case(Hq=2, D=64, n=24, begin=(4, 9), end=(28, 33), rope=rope)
    for rows in (c.k, c.v):
        rows[:, :, :, 0::3] = -0.0
        rows[:, :, :, 1::7] = 0.0
        rows[:, ::2, :, 32:48] = -0.0  # groups of nothing else
        rows[:, 1::2, :, 5] = -1e-3    # next to values near 1: rounds to zero
    pool = fill_pool4(c)
    pool0, meta0 = pool.clone(), c.meta.clone()
    append4(c, pool)
    check_four(c, pool0, pool, meta0, 1.0, 1.0)


# ---- NaN in the attention -------------------------------------------------------------------------------------
class Poisoned(Cache):
    """A cache whose numbers (`rows`) are kept as they were before some became NaN."""

    def keep(self):
        self.rows(0, 0)
        self.q0 = self.q.clone()
        G = self.Hq // self.Hkv
        self.bad_out = np.zeros((self.B, self.Hkv, G, self.D), dtype=bool)
        self.bad_lse = np.zeros((self.B, self.Hkv, G), dtype=bool)

    def token(self, b, h, t):
        """The page of token t and where its key and value scales begin."""
        o, w = kp.offsets(self.T, self.D), self.D // 16
        page = self.pool[int(self.table[b, self.layer, h, t // self.T])]
        return page, o[1] + t % self.T * w, o[3] + t % self.T * w

    def nan_query(self, b, head):
        G = self.Hq // self.Hkv
        self.q[b, head, 3] = math.nan
        self.bad_out[b, head // G, head % G] = self.bad_lse[b, head // G, head % G] = True

    def nan_key(self, b, h, t, group=1):
        page, k, _ = self.token(b, h, t)
        page[k + group] = 0x7F
        self.bad_out[b, h] = self.bad_lse[b, h] = True

    def nan_value(self, b, h, t, group=2):
        page, _, v = self.token(b, h, t)
        page[v + group] = 0x7F
        self.bad_out[b, h, :, 16 * group:16 * group + 16] = True

    def check_nan(self, units):
        G = self.Hq // self.Hkv
        out, lse, q = (x.float().cpu().numpy().astype(np.float64) for x in (self.out, self.lse, self.q0))
        for b, h in units:
            pages = None
            if self.sel is not None:
                pages = self.sel[b, self.layer, h, :int(self.cnt[b, self.layer, h])].cpu().numpy()
            k, v = self.rows(b, h, pages)
            g = slice(h * G, (h + 1) * G)
            assert np.array_equal(np.isnan(out[b, g]), self.bad_out[b, h]), (b, h)
            assert np.array_equal(np.isnan(lse[b, g]), self.bad_lse[b, h]), (b, h)
            if k.shape[0] == 0:
                assert (out[b, g] == 0).all() and (lse[b, g] == -np.inf).all(), (b, h)
                continue
            want, wl, zsum = kp.unit_attention(q[b, g], k, v, 1 / math.sqrt(self.D))
            tol = kp.out_tolerance(self.D, zsum, np.abs(v).max())
            assert np.nanmax(np.abs(out[b, g] - want), initial=0.0) <= tol, (b, h)
            ok = ~self.bad_lse[b, h]
            assert (np.abs(lse[b, g] - wl) <= kp.lse_tolerance(self.D, zsum, wl))[ok].all(), (b, h)


@pytest.mark.parametrize("G,D,T", [(1, 128, 16), (4, 64, 32), (5, 128, 32), (8, 64, 16)])
@pytest.mark.parametrize("mode", ["one CTA a unit", "clusters", "selections", "dealt, short", "dealt, long",
                                  "dealt, selections"])
def test_nan_reaches_the_results(mode, G, D, T):
    """A NaN in a query reaches its head's results, one in a key its unit's, one in a value its channels', however the
    pages were dealt; no other number changes its place among the tolerances."""
    if mode == "one CTA a unit":
        c = Poisoned([200, 33, 0], Hq=2 * G, D=D, T=T)
    elif mode == "clusters":
        c = Poisoned([2001, 777, 0], Hq=2 * G, D=D, T=T, L=1, layer=0)
    elif mode == "selections":
        c = Poisoned([2001, 777, 0], Hq=2 * G, D=D, T=T, L=1, layer=0)
        c.select(c.Pmax, seed=3)
    elif mode == "dealt, long":
        c = Poisoned([70003, 20000, 0], Hq=2 * G, D=D, T=T, L=1, layer=0)
    else:
        c = Poisoned([200, 33, 0, 17] * 30, Hq=2 * G, D=D, T=T, L=1, layer=0)
        if mode == "dealt, selections":
            c.select(c.Pmax, seed=3)
    c.keep()
    c.nan_query(0, G - 1)      # the last head of the first group
    c.nan_value(0, 1, 130)     # the other unit of that sequence
    c.nan_key(1, 0, 0)         # the first token
    c.nan_value(1, 1, 32, group=0)
    c.nan_query(1, 2 * G - 1)
    if c.B > 3:
        c.nan_key(4, 1, 199)   # the last token
        c.nan_value(5, 0, 15)
    for _ in range(2):
        c.attend()
        torch.cuda.synchronize()
        assert int(c.err) == 0
        c.check_nan([(b, h) for b in range(min(c.B, 9)) for h in range(2)])
    assert int(c.ws[:1024].max()) == 0


# ---- positions replaced between calls -------------------------------------------------------------------------
def test_positions_replaced_between_calls():
    """A call turns its rows by the positions that its rope has then, whatever it had when it was made."""
    a, b = (Case(n=5, begin=(3, 20), end=(8, 25)) for _ in range(2))
    rope = kvmm.Rope(a.angles, a.dim, positions=torch.zeros(2, 5, dtype=torch.int32, device="cuda"))
    for pos in ([[9, 1, 7, 30, 2], [5, 5, 6, 8, 0]], None, [[0, 1, 2, 3, 4], [90, 91, 92, 93, 94]]):
        rope.positions = None if pos is None else torch.tensor(pos, dtype=torch.int32, device="cuda")
        junk = torch.full((2, 5), 95, dtype=torch.int32, device="cuda")  # may take the memory of the ones before
        fresh = kvmm.Rope(b.angles, b.dim, positions=rope.positions)
        for c, r in ((a, rope), (b, fresh)):
            kvmm.kv_append_rope(c.shape, 1, c.q, c.k, c.v, c.tb, c.te, c.k_pool, c.v_pool, c.table, c.meta, rope=r,
                                q_out=c.q_out, err=c.err)
        torch.cuda.synchronize()
        assert int(a.err) == int(b.err) == 0 and int(junk[0, 0]) == 95
        at = np.array(pos) if pos is not None else np.array([range(3, 8), range(20, 25)])
        for i in range(2):
            want = kp.bf16(a.turned(a.q[i].float().cpu().numpy().astype(np.float64), at[i]))
            assert np.array_equal(a.q_out[i].float().cpu().numpy().astype(np.float64), want)
        assert torch.equal(a.q_out, b.q_out) and torch.equal(a.k_pool, b.k_pool) and torch.equal(a.meta, b.meta)


# ---- batches of more than one launch --------------------------------------------------------------------------
def many(B, **kw):
    """Short sequences, empty ones where the launches meet, longer ones among the last."""
    rng = np.random.default_rng(B)
    seq = [int(x) for x in rng.integers(0, 40, B)]
    for b in (0, 511, 512, 1023, 1024, B - 2):
        if b < B:
            seq[b] = 0
    seq[B - 1], seq[B - 3] = 630, 333
    return Cache(seq, L=1, layer=0, Pmax=40, **kw)


@pytest.mark.parametrize("early", [False, True])
@pytest.mark.parametrize("B,Hkv,G,D,T", [(1030, 2, 4, 64, 16), (1030, 1, 3, 64, 32), (520, 1, 8, 128, 16), (517, 2, 5, 128, 32)])
def test_every_page_in_several_launches(B, Hkv, G, D, T, early):
    """More than 512 sequences: each launch's offsets into queries, outputs, lengths and table, its own way of dealing
    the pages (the last few sequences by clusters), one workspace."""
    c = many(B, Hq=Hkv * G, Hkv=Hkv, D=D, T=T)
    c.spoil_behind()
    for _ in range(2):
        c.out.fill_(5.0), c.lse.fill_(5.0)
        torch.cuda.synchronize()
        c.attend(early_reads=early, v_scale=0.5)
        torch.cuda.synchronize()
        assert int(c.err) == 0
        c.check(v_scale=0.5)
    assert int(c.ws[:1024].max()) == 0


@pytest.mark.parametrize("early", [False, True])
@pytest.mark.parametrize("B,Hkv,G,D,T", [(1030, 2, 4, 64, 16), (520, 1, 8, 128, 32)])
def test_selections_in_several_launches(B, Hkv, G, D, T, early):
    c = many(B, Hq=Hkv * G, Hkv=Hkv, D=D, T=T)
    rng = np.random.default_rng(7)
    c.select(20, cnt=[int(x) for x in rng.integers(0, 21, B * Hkv)])
    c.attend(early_reads=early)
    torch.cuda.synchronize()
    assert int(c.err) == 0
    c.check()
    assert int(c.ws[:1024].max()) == 0


def test_bad_entries_in_a_later_launch():
    """A length, a table entry and a selection out of their ranges in the second launch set their bits, and the other
    sequences have their results."""
    c = many(520, Hq=4, Hkv=1, D=64, T=16)
    c.seq_len[515] = 9999
    c.attend()
    torch.cuda.synchronize()
    assert int(c.err) == kvmm.ERR_OUT_OF_RANGE
    units = {(b, 0) for b in range(520)} - {(515, 0)}
    c.check(units=units)
    c.seq_len[515] = c.seq[515]
    c.err.zero_()
    c.table[519, 0, 0, 5] = -1
    c.__dict__.pop("_np")
    c.attend()
    torch.cuda.synchronize()
    assert int(c.err) == kvmm.ERR_NULL_BLOCK
    c.check()


# ---- long sums ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("G,D,T", [(4, 128, 16), (8, 128, 32), (2, 64, 32), (5, 64, 16)])
@pytest.mark.parametrize("mode", ["every page", "selections, clusters", "selections, one CTA a unit", "a few tiles"])
def test_long_sums_are_not_rounded_one_way(mode, G, D, T):
    """Hundreds of tiles a warp: the mean error of outputs that are means of positive values.

    With a query of zeros every probability is the same power of two and the sum of weights is exact, so all that is
    rounded is the values' sum.  The tensor core rounds toward zero, at most 2^-23 of what it has, and may add up 32
    products of one run at most, the k-th onto k/32 of the sum: (32 + 1) / 2 * 2^-23 = 2^-18.95 of it; on average over
    the places in a step (half of it) and over where a sum lies between powers of two (0.72), 2^-20.4.  What is rounded
    to nearest has no direction, and its mean over thousands of outputs vanishes beside that.  Longer runs rounded
    toward zero would be off by their length over 32 times as much.
    """
    n_phys = 700
    if mode == "every page":
        B, Hkv, Pmax, K = 6, 4, 32768, 1
    elif mode == "selections, clusters":
        B, Hkv, Pmax, K = 2, 4, 64, 32768
    elif mode == "selections, one CTA a unit":
        B, Hkv, Pmax, K = 20, 5, 64, 6000
    else:
        B, Hkv, Pmax, K = 9, 2, 200, 1
    g = torch.Generator(device="cuda").manual_seed(D + T)
    shape = kvmm.make_shape(B, 1, Hkv * G, Hkv, D, T, Pmax, K, n_phys)
    pool = torch.randint(0, 256, (n_phys, kvmm.kv4_page_bytes(shape)), generator=g, device="cuda", dtype=torch.uint8)
    pool &= 0x77  # no signs; scales up to 2^7 * 15/8, with low bits that a long sum cannot keep
    table = torch.randint(0, n_phys, (B, 1, Hkv, Pmax), generator=g, device="cuda", dtype=torch.int32)
    seq = torch.full((B,), Pmax * T, dtype=torch.int32, device="cuda")
    sel = cnt = None
    pages = table[:, 0]
    if K > 1:
        sel = torch.randint(0, Pmax, (B, 1, Hkv, K), generator=g, device="cuda", dtype=torch.int32)
        cnt = torch.full((B, 1, Hkv), K, dtype=torch.int32, device="cuda")
        pages = table[:, 0].gather(2, sel[:, 0].long())
    q = torch.zeros(B, Hkv * G, D, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.zeros(B, Hkv * G, D, device="cuda"), torch.zeros(B, Hkv * G, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvmm.sparse_paged_decode_attn_kv4(shape, 0, q, pool, table, seq, sel, cnt, out, kvmm.alloc_kv4_workspace(shape),
                                      lse=lse, err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    held = pool.cpu().numpy()
    mean = np.stack([kp.value(*kp.page_rows(held[i], T, D, True)).mean(0) for i in range(n_phys)])  # a page's
    count = np.stack([np.bincount(x, minlength=n_phys) for x in pages.reshape(B * Hkv, -1).cpu().numpy()])
    want = (count @ mean / pages.shape[-1]).reshape(B, Hkv, 1, D)
    off = out.double().cpu().numpy().reshape(B, Hkv, G, D) / want - 1
    mean_off = float(off.mean())
    assert abs(mean_off) <= 2.0 ** -20.4
    tokens = pages.shape[-1] * T
    assert np.abs(lse.cpu().numpy() - math.log(tokens)).max() <= 2.0 ** -22 * math.log(tokens) + 2.0 ** -22
