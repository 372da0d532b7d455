"""kv_append_rope and kv4_append_rope against the plain arithmetic, bit for bit, and against kv_minmax_update.

Covers every (D, T), both pairings, partly turned rows, rows of any strides (cut from one projection, head by head,
broadcast over the batch), ragged ranges that begin and end inside pages, single tokens, empty ranges, explicit
positions, null and out-of-range entries, and what has to be left as it was.
"""
import numpy as np
import pytest
import torch

from paged_kv_cache_minmax_gb300 import kvmm
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


def bits(t):
    return t.detach().contiguous().cpu().view(torch.int16).numpy()


class Case:
    """Pools, table and new rows of one shape."""

    def __init__(self, B=2, L=2, Hq=8, Hkv=2, D=64, T=16, Pmax=6, n=5, begin=(3, 20), end=(8, 25), rope="half", dim=None,
                 rows="fused", seed=0, layer=1, spread=1.0, rope_rows=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.L, self.Hq, self.Hkv, self.D, self.T, self.Pmax, self.n, self.layer = B, L, Hq, Hkv, D, T, Pmax, n, layer
        self.n_phys = B * L * Hkv * Pmax + 3
        self.shape = kvmm.make_shape(B, L, Hq, Hkv, D, T, Pmax, 4, self.n_phys)
        self.table = torch.randperm(self.n_phys, generator=g, device="cuda")[:B * L * Hkv * Pmax].to(torch.int32)
        self.table = self.table.view(B, L, Hkv, Pmax).contiguous()

        def normal(*s):
            x = torch.randn(*s, generator=g, device="cuda")
            if spread != 1.0:
                x = x * torch.exp2(spread * torch.randn(*s[:-1], 1, generator=g, device="cuda"))
            return x.to(torch.bfloat16)

        self.k_pool, self.v_pool = normal(self.n_phys, T, D), normal(self.n_phys, D, T)
        self.meta = normal(B, L, Hkv, Pmax, 2, D)
        if rows == "fused":
            x = normal(B, n, Hq + 2 * Hkv, D)
            self.q, self.k, self.v = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
        elif rows == "heads":
            self.q, self.k, self.v = (normal(B, H, n, D).transpose(1, 2) for H in (Hq, Hkv, Hkv))
        elif rows == "tokens":
            self.q, self.k, self.v = (normal(n, B, H, D).transpose(0, 1) for H in (Hq, Hkv, Hkv))
        else:  # one batch entry's rows for all
            self.q, self.k, self.v = (normal(1, n, H, D).expand(B, n, H, D) for H in (Hq, Hkv, Hkv))
        self.begin, self.end = list(begin), list(end)
        self.tb, self.te = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (self.begin, self.end))
        self.q_out = torch.full((B, n, Hq, D), 77.0, dtype=torch.bfloat16, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.rope, self.style = None, rope
        if rope != "none":
            self.dim = dim or D
            R = rope_rows or Pmax * T
            ang = torch.arange(R, dtype=torch.float64)[:, None] * 10000.0 ** (
                -2.0 * torch.arange(self.dim // 2, dtype=torch.float64) / self.dim)
            self.angles = torch.stack([ang.cos(), ang.sin()], 1).float().cuda()
            self.rope = kvmm.Rope(self.angles, self.dim, interleaved=rope == "pairs")

    def turned(self, x, pos, rounded=True):
        """x [n, H, D] float64 at positions pos [n]."""
        if self.rope is None:
            return x
        t = f64(self.angles)[pos]
        return kp.rotate(x, t[:, 0][:, None], t[:, 1][:, None], self.dim, self.style == "pairs", rounded)

    def ranges(self):
        cap = self.Pmax * self.T
        for b in range(self.B):
            tb, te = self.begin[b], self.end[b]
            if 0 <= tb <= te and tb <= cap:
                te = min(te, cap)
                yield b, tb, min(te, tb + self.n)


CASES = {
    "half-d64": dict(),
    "half-d128-t16": dict(D=128, Hq=4, n=40, begin=(0, 17), end=(40, 57), Pmax=4),
    "pairs-d128-t32": dict(D=128, T=32, Hq=10, rope="pairs", n=33, begin=(31, 0), end=(64, 33), Pmax=3, rows="heads"),
    "part-d64-t32": dict(T=32, dim=32, n=70, begin=(5, 63), end=(75, 96), Pmax=4, rows="tokens"),
    "part-pairs-d128": dict(D=128, dim=96, rope="pairs", n=16, begin=(16, 1), end=(32, 17)),
    "part-half-d128": dict(D=128, dim=32, n=3, begin=(14, 0), end=(17, 3), rows="one"),
    "none": dict(rope="none", n=9, begin=(0, 30), end=(9, 39)),
    "token": dict(n=1, begin=(15, 16), end=(16, 17)),
    "token-first": dict(n=1, begin=(0, 95), end=(1, 96), D=128, Hq=2),
    "ragged": dict(B=5, n=20, begin=(0, 7, 16, 90, 3), end=(20, 7, 17, 96, 22), Hkv=3, Hq=3),
    "wide-range": dict(spread=6.0, n=24, begin=(4, 9), end=(28, 33)),
    "blocks-d64-t32": dict(Hq=32, Hkv=4, T=32, n=35, begin=(30, 0), end=(65, 20), Pmax=4, rope="pairs"),
    "rows-d128": dict(B=3, Hq=12, Hkv=3, D=128, T=32, n=5, begin=(30, 0, 96), end=(35, 0, 101), Pmax=4),
    "eight-heads": dict(Hq=64, Hkv=8, D=128, n=2, begin=(3, 31), end=(5, 33), L=1, layer=0),
}


def expected_rows(c, four_scale=None):
    """(b, token, key rows, value rows) float64 as the pools take them: turned, bf16-rounded (or fp32, for 4 bits)."""
    for b, tb, te in c.ranges():
        n = te - tb
        k = c.turned(f64(c.k[b, :n]), np.arange(tb, te))
        v = f64(c.v[b, :n])
        yield b, tb, te, k, v


@pytest.mark.parametrize("name", sorted(CASES))
def test_bf16_append_is_exact(name):
    c = Case(**CASES[name])
    k0, v0, m0 = (t.clone() for t in (c.k_pool, c.v_pool, c.meta))
    kvmm.kv_append_rope(c.shape, c.layer, c.q, c.k, c.v, c.tb, c.te, c.k_pool, c.v_pool, c.table, c.meta, rope=c.rope,
                        q_out=c.q_out, err=c.err)
    torch.cuda.synchronize()
    assert int(c.err) == 0
    want_k, want_v, want_m = f64(k0), f64(v0), f64(m0)
    want_q = np.full((c.B, c.n, c.Hq, c.D), 77.0)
    for b, tb, te, k, v in expected_rows(c):
        kb = kp.bf16(k)
        want_q[b, :te - tb] = kp.bf16(c.turned(f64(c.q[b, :te - tb]), np.arange(tb, te)))
        # the rounded rotation is within half a bf16 step, and three fp32 roundings of its products, of the true one
        true = c.turned(f64(c.k[b, :te - tb]), np.arange(tb, te), rounded=False)
        x = np.abs(f64(c.k[b, :te - tb])).max(-1, keepdims=True)
        assert (np.abs(kb - true) <= 2.0 ** -8 * np.abs(true) + 4 * 2.0 ** -24 * 2 * x).all()
        for h in range(c.Hkv):
            row = c.table[b, c.layer, h].cpu().numpy()
            for t in range(tb, te):
                want_k[row[t // c.T], t % c.T] = kb[t - tb, h]
                want_v[row[t // c.T], :, t % c.T] = v[t - tb, h]
            for p in range(tb // c.T, -(-te // c.T)) if te > tb else ():
                rows = want_k[row[p], :min(c.T, te - p * c.T)]
                want_m[b, c.layer, h, p] = rows.min(0), rows.max(0)
    assert np.array_equal(f64(c.k_pool), want_k)
    assert np.array_equal(f64(c.v_pool), want_v)
    assert np.array_equal(f64(c.meta), want_m)
    assert np.array_equal(f64(c.q_out), want_q)


@pytest.mark.parametrize("name", sorted(CASES))
def test_bf16_append_equals_minmax_update_on_turned_rows(name):
    """The operator beside it, given dense rows that are already turned, leaves the same bytes."""
    c = Case(**CASES[name])
    d = Case(**CASES[name])
    kvmm.kv_append_rope(c.shape, c.layer, None, c.k, c.v, c.tb, c.te, c.k_pool, c.v_pool, c.table, c.meta, rope=c.rope,
                        err=c.err)
    k = torch.zeros(c.B, c.Hkv, c.n, c.D, dtype=torch.bfloat16, device="cuda")
    for b, tb, te, rows, _ in expected_rows(d):
        k[b, :, :te - tb] = torch.from_numpy(kp.bf16(rows)).cuda().transpose(0, 1).to(torch.bfloat16)
    v = d.v.transpose(1, 2).contiguous()
    kvmm.kv_minmax_update(d.shape, d.layer, k, v, d.n, d.tb, d.te, d.k_pool, d.v_pool, d.table, d.meta, d.err)
    torch.cuda.synchronize()
    assert int(c.err) == int(d.err) == 0
    for x, y in ((c.k_pool, d.k_pool), (c.v_pool, d.v_pool), (c.meta, d.meta)):
        # a turned zero may be -0 on one side: compare values, and bits where they are not zero
        assert torch.equal(x, y)


def fill_pool4(c, seed=5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    pool = torch.randint(0, 256, (c.n_phys, kvmm.kv4_page_bytes(c.shape)), generator=g, device="cuda", dtype=torch.uint8)
    o = kp.offsets(c.T, c.D)
    for i in (1, 3):
        pool[:, o[i]:o[i + 1]] = torch.randint(0, 0x7F, (c.n_phys, o[i + 1] - o[i]), generator=g, device="cuda",
                                               dtype=torch.uint8)
    return pool


def check_four(c, pool0, pool, meta0, k_scale, v_scale):
    want, want_m = pool0.cpu().numpy().copy(), f64(meta0)
    for b, tb, te, k, v in expected_rows(c):
        if te <= tb:
            continue
        kc, ks = kp.hold(k, k_scale)
        vc, vs = kp.hold(v, v_scale)
        for h in range(c.Hkv):
            row = c.table[b, c.layer, h].cpu().numpy()
            for t in range(tb, te):
                kp.put_row(want[row[t // c.T]], c.T, c.D, t % c.T, False, kc[t - tb, h], ks[t - tb, h])
                kp.put_row(want[row[t // c.T]], c.T, c.D, t % c.T, True, vc[t - tb, h], vs[t - tb, h])
            for p in range(tb // c.T, -(-te // c.T)):
                held = kp.value(*kp.page_rows(want[row[p]], c.T, c.D, False))[:min(c.T, te - p * c.T)]
                want_m[b, c.layer, h, p] = held.min(0), held.max(0)
    assert np.array_equal(pool.cpu().numpy(), want)
    assert np.array_equal(f64(c.meta), want_m)


@pytest.mark.parametrize("scales", [(1.0, 1.0), (0.37, 2.5)])
@pytest.mark.parametrize("name", sorted(CASES))
def test_4bit_append_is_exact(name, scales):
    c = Case(**CASES[name])
    pool = fill_pool4(c)
    pool0, meta0 = pool.clone(), c.meta.clone()
    kvmm.kv4_append_rope(c.shape, c.layer, c.q, c.k, c.v, c.tb, c.te, pool, c.table, c.meta, rope=c.rope, q_out=c.q_out,
                         k_scale=scales[0], v_scale=scales[1], err=c.err)
    torch.cuda.synchronize()
    assert int(c.err) == 0
    check_four(c, pool0, pool, meta0, *scales)
    for b, tb, te in c.ranges():
        want_q = kp.bf16(c.turned(f64(c.q[b, :te - tb]), np.arange(tb, te)))
        assert np.array_equal(f64(c.q_out[b, :te - tb]), want_q)
        assert (f64(c.q_out[b, te - tb:]) == 77.0).all()


def test_4bit_borders():
    """Values on and next to every border of a code, zero groups, scales that vanish, saturate or are subnormal."""
    D, T, n = 64, 16, 48
    c = Case(B=1, Hq=2, Hkv=2, D=D, T=T, Pmax=3, n=n, begin=(0,), end=(n,), rope="none", L=1, layer=0)
    rng = np.random.default_rng(3)
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    x = np.zeros((n, 2, D))
    for i in range(n):
        for h in range(2):
            for g in range(D // 16):
                s = kp.E4M3[rng.integers(1, 0x7F)]
                y = rng.choice(borders, 16) * s * rng.choice([-1, 1], 16)
                y[0] = 6 * s  # fixes the scale at s
                kind = (i * 8 + h * 4 + g) % 6
                if kind == 1:  # the next bf16 up or down
                    y = y * (1 + rng.choice([-1, 1], 16) * 2.0 ** -7)
                elif kind == 2:
                    y = np.zeros(16)
                elif kind == 3:
                    y = y / np.abs(y).max() * rng.choice([1e-4, 0.003, 0.0058, 0.01, 0.02, 0.05])
                elif kind == 4:
                    y = y / np.abs(y).max() * rng.choice([2600.0, 2688.0, 2900.0, 1e5])
                x[i, h, 16 * g:16 * g + 16] = y
    rows = torch.from_numpy(x).float().to(torch.bfloat16).cuda().unsqueeze(0)
    c.k, c.v = rows, rows.flip(1).contiguous()
    pool = fill_pool4(c)
    pool0, meta0 = pool.clone(), c.meta.clone()
    kvmm.kv4_append_rope(c.shape, 0, None, c.k, c.v, c.tb, c.te, pool, c.table, c.meta, err=c.err)
    torch.cuda.synchronize()
    assert int(c.err) == 0
    check_four(c, pool0, pool, meta0, 1.0, 1.0)


@pytest.mark.parametrize("four", [False, True])
def test_token_by_token_equals_a_prompt(four):
    a = Case(D=128, n=37, begin=(2, 11), end=(39, 48), rows="heads")
    b = Case(D=128, n=37, begin=(2, 11), end=(39, 48), rows="heads")
    pa, pb = (fill_pool4(c) for c in (a, b))

    def append(c, pool, k, v, q, tb, te, q_out):
        if four:
            kvmm.kv4_append_rope(c.shape, 1, q, k, v, tb, te, pool, c.table, c.meta, rope=c.rope, q_out=q_out, err=c.err)
        else:
            kvmm.kv_append_rope(c.shape, 1, q, k, v, tb, te, c.k_pool, c.v_pool, c.table, c.meta, rope=c.rope,
                                q_out=q_out, err=c.err)

    append(a, pa, a.k, a.v, a.q, a.tb, a.te, a.q_out)
    for j in range(37):
        q_out = torch.zeros(2, 1, b.Hq, b.D, dtype=torch.bfloat16, device="cuda")
        append(b, pb, b.k[:, j:j + 1], b.v[:, j:j + 1], b.q[:, j:j + 1], b.tb + j, b.tb + j + 1, q_out)
        b.q_out[:, j] = q_out[:, 0]
    torch.cuda.synchronize()
    assert int(a.err) == int(b.err) == 0
    for x, y in ((a.k_pool, b.k_pool), (a.v_pool, b.v_pool), (a.meta, b.meta), (a.q_out, b.q_out)):
        assert np.array_equal(bits(x), bits(y))
    assert torch.equal(pa, pb)


@pytest.mark.parametrize("four", [False, True])
def test_explicit_positions_and_rows_without_one(four):
    """Positions that are not the indices; a row whose position the table lacks is left out, all else is written."""
    c = Case(n=6, begin=(3, 20), end=(9, 26), rope_rows=40)
    pos = torch.tensor([[39, 0, 7, 40, 7, 1], [5, -1, 6, 8, 2, 2]], dtype=torch.int32, device="cuda")
    rope = kvmm.Rope(c.angles, c.dim, positions=pos)
    pool = fill_pool4(c)
    pool0, k0, v0, meta0 = pool.clone(), c.k_pool.clone(), c.v_pool.clone(), c.meta.clone()
    if four:
        kvmm.kv4_append_rope(c.shape, 1, c.q, c.k, c.v, c.tb, c.te, pool, c.table, c.meta, rope=rope, q_out=c.q_out,
                             err=c.err)
    else:
        kvmm.kv_append_rope(c.shape, 1, c.q, c.k, c.v, c.tb, c.te, c.k_pool, c.v_pool, c.table, c.meta, rope=rope,
                            q_out=c.q_out, err=c.err)
    torch.cuda.synchronize()
    assert int(c.err) == kvmm.ERR_OUT_OF_RANGE
    at = pos.cpu().numpy()
    want, wk, wv, wq = pool0.cpu().numpy().copy(), f64(k0), f64(v0), np.full((2, 6, c.Hq, c.D), 77.0)
    wm = f64(meta0)
    for b in range(2):
        good = [j for j in range(6) if 0 <= at[b, j] < 40]
        k = c.turned(f64(c.k[b, good]), at[b, good])
        q = c.turned(f64(c.q[b, good]), at[b, good])
        v = f64(c.v[b, good])
        (kc, ks), (vc, vs) = kp.hold(k, 1.0), kp.hold(v, 1.0)
        for i, j in enumerate(good):
            wq[b, j] = kp.bf16(q[i])
            t = c.begin[b] + j
            for h in range(c.Hkv):
                phys = int(c.table[b, 1, h, t // c.T])
                kp.put_row(want[phys], c.T, c.D, t % c.T, False, kc[i, h], ks[i, h])
                kp.put_row(want[phys], c.T, c.D, t % c.T, True, vc[i, h], vs[i, h])
                wk[phys, t % c.T], wv[phys, :, t % c.T] = kp.bf16(k[i, h]), v[i, h]
        for h in range(c.Hkv):
            for p in range(c.begin[b] // c.T, -(-c.end[b] // c.T)):
                phys, n = int(c.table[b, 1, h, p]), min(c.T, c.end[b] - p * c.T)
                rows = kp.value(*kp.page_rows(want[phys], c.T, c.D, False)) if four else wk[phys]
                wm[b, 1, h, p] = rows[:n].min(0), rows[:n].max(0)
    assert np.array_equal(f64(c.q_out), wq)
    assert np.array_equal(f64(c.meta), wm)
    if four:
        assert np.array_equal(pool.cpu().numpy(), want)
    else:
        assert np.array_equal(f64(c.k_pool), wk) and np.array_equal(f64(c.v_pool), wv)


@pytest.mark.parametrize("four", [False, True])
def test_bad_ranges_and_entries(four):
    """Ranges outside the table append nothing, long ones are cut, bad entries skip their page; each sets its bit."""
    def go(bits_wanted, change, touched, **kw):
        c = Case(**{**dict(n=8, begin=(3, 20), end=(8, 25)), **kw})
        pool = fill_pool4(c)
        change(c)
        before = [t.clone() for t in (c.k_pool, c.v_pool, pool, c.meta)]
        if four:
            kvmm.kv4_append_rope(c.shape, 1, c.q, c.k, c.v, c.tb, c.te, pool, c.table, c.meta, rope=c.rope,
                                 q_out=c.q_out, err=c.err)
        else:
            kvmm.kv_append_rope(c.shape, 1, c.q, c.k, c.v, c.tb, c.te, c.k_pool, c.v_pool, c.table, c.meta, rope=c.rope,
                                q_out=c.q_out, err=c.err)
        torch.cuda.synchronize()
        assert int(c.err) == bits_wanted
        now = [c.k_pool, c.v_pool, pool, c.meta]
        changed = {int(i) for x, y in zip(before[:3], now[:3]) for i in torch.nonzero((x != y).flatten(1).any(1)).flatten()}
        assert changed == touched(c)
        return c

    pages = lambda c, *bp: {int(c.table[b, 1, h, p]) for b, p in bp for h in range(c.Hkv)}  # noqa: E731
    both = lambda c: pages(c, (0, 0), (1, 1))  # noqa: E731
    go(0, lambda c: None, both)
    c = go(kvmm.ERR_OUT_OF_RANGE, lambda c: c.tb.copy_(torch.tensor([-1, 20])), lambda c: pages(c, (1, 1)))
    assert (f64(c.q_out[0]) == 77.0).all()
    go(kvmm.ERR_OUT_OF_RANGE, lambda c: c.te.copy_(torch.tensor([2, 25])), lambda c: pages(c, (1, 1)))
    c = go(kvmm.ERR_OUT_OF_RANGE, lambda c: c.te.copy_(torch.tensor([2 ** 31 - 1, 25])), both)  # cut to eight rows
    assert (f64(c.q_out[0]) != 77.0).any(-1).all()
    go(kvmm.ERR_OUT_OF_RANGE, lambda c: (c.tb.copy_(torch.tensor([93, 20])), c.te.copy_(torch.tensor([99, 25]))),
       lambda c: pages(c, (0, 5), (1, 1)))
    go(0, lambda c: (c.tb.copy_(torch.tensor([96, 20])), c.te.copy_(torch.tensor([96, 25]))), lambda c: pages(c, (1, 1)))

    def entry(v):
        def change(c):
            c.keep = c.table.clone()
            c.table[0, 1, 1, 0] = v
        return change

    one = lambda c: {int(c.table[0, 1, 0, 0])} | pages(c, (1, 1))  # noqa: E731
    c = go(kvmm.ERR_NULL_BLOCK, entry(-1), one)
    assert (f64(c.q_out[0, :5]) != 77.0).any(-1).all()  # the queries do not depend on their keys' pages
    go(kvmm.ERR_OUT_OF_RANGE, entry(c.n_phys), one)


def test_without_metadata_queries_or_error_word():
    a, b = (Case(D=128, n=20, begin=(3, 20), end=(23, 40)) for _ in range(2))
    kvmm.kv_append_rope(a.shape, 1, a.q, a.k, a.v, a.tb, a.te, a.k_pool, a.v_pool, a.table, a.meta, rope=a.rope,
                        q_out=a.q_out, err=a.err)
    keep = b.meta.clone()
    kvmm.kv_append_rope(b.shape, 1, None, b.k, b.v, b.tb, b.te, b.k_pool, b.v_pool, b.table, None, rope=b.rope)
    pa, pb = fill_pool4(a), fill_pool4(b)
    kvmm.kv4_append_rope(a.shape, 1, a.q, a.k, a.v, a.tb, a.te, pa, a.table, a.meta, rope=a.rope, q_out=a.q_out)
    kvmm.kv4_append_rope(b.shape, 1, None, b.k, b.v, b.tb, b.te, pb, b.table, None, rope=b.rope)
    torch.cuda.synchronize()
    assert torch.equal(a.k_pool, b.k_pool) and torch.equal(a.v_pool, b.v_pool) and torch.equal(pa, pb)
    assert torch.equal(b.meta, keep)


def test_queries_turn_in_place():
    a, b = (Case(D=128, n=1, begin=(3, 20), end=(4, 21)) for _ in range(2))
    kvmm.kv_append_rope(a.shape, 1, a.q, a.k, a.v, a.tb, a.te, a.k_pool, a.v_pool, a.table, a.meta, rope=a.rope,
                        q_out=a.q_out, err=a.err)
    q = b.q.contiguous()
    kvmm.kv_append_rope(b.shape, 1, q, b.k, b.v, b.tb, b.te, b.k_pool, b.v_pool, b.table, b.meta, rope=b.rope, q_out=q,
                        err=b.err)
    torch.cuda.synchronize()
    assert np.array_equal(bits(q), bits(a.q_out))


def test_many_query_rows_and_pages():
    """Enough rows that a warp takes several query rows, at an odd count."""
    c = Case(B=3, L=1, layer=0, Hq=24, Hkv=3, D=64, T=16, Pmax=64, n=1001, begin=(0, 9, 1), end=(1001, 1010, 3))
    kvmm.kv_append_rope(c.shape, 0, c.q, c.k, c.v, c.tb, c.te, c.k_pool, c.v_pool, c.table, c.meta, rope=c.rope,
                        q_out=c.q_out, err=c.err)
    torch.cuda.synchronize()
    assert int(c.err) == 0
    for b, tb, te in c.ranges():
        n = te - tb
        assert np.array_equal(f64(c.q_out[b, :n]), kp.bf16(c.turned(f64(c.q[b, :n]), np.arange(tb, te))))
        assert (f64(c.q_out[b, n:]) == 77.0).all()
        t = np.arange(tb, te)
        for h in range(c.Hkv):
            phys = c.table[b, 0, h].cpu().numpy()[t // c.T]
            assert np.array_equal(f64(c.k_pool)[phys, t % c.T], kp.bf16(c.turned(f64(c.k[b, :n]), t))[:, h])
            assert np.array_equal(f64(c.v_pool)[phys, :, t % c.T], f64(c.v[b, :n, h]))


def test_binding_refuses():
    c = Case()
    with pytest.raises(ValueError, match="new_v must be"):
        kvmm.kv_append_rope(c.shape, 1, None, c.k, c.v[:, :3], c.tb, c.te, c.k_pool, c.v_pool, c.table, c.meta)
    with pytest.raises(ValueError, match="consecutive"):
        kvmm.kv_append_rope(c.shape, 1, None, c.k.transpose(2, 3).contiguous().transpose(2, 3), c.v, c.tb, c.te, c.k_pool,
                            c.v_pool, c.table, c.meta)
    with pytest.raises(ValueError, match="positions"):
        rope = kvmm.Rope(c.angles, c.dim, positions=torch.zeros(3, dtype=torch.int32, device="cuda"))
        kvmm.kv_append_rope(c.shape, 1, None, c.k, c.v, c.tb, c.te, c.k_pool, c.v_pool, c.table, c.meta, rope=rope)
    odd = torch.zeros(2, 5, 2, 68, dtype=torch.bfloat16, device="cuda")[..., 4:]
    with pytest.raises(kvmm.KvmmError, match="invalid"):
        kvmm.kv_append_rope(c.shape, 1, None, odd, c.v, c.tb, c.te, c.k_pool, c.v_pool, c.table, c.meta)
    with pytest.raises(kvmm.KvmmError, match="unsupported"):
        t = torch.zeros(9, 2, 8, device="cuda")
        kvmm.kv_append_rope(c.shape, 1, None, c.k, c.v, c.tb, c.te, c.k_pool, c.v_pool, c.table, c.meta,
                            rope=kvmm.Rope(t, 16))


@pytest.mark.parametrize("four", [False, True])
def test_offsets_beyond_32_bits(four):
    """Pages and rows that lie more than 2^31 elements and 2^32 bytes into their buffers: the bits of a small pool's."""
    c = Case(D=128, T=32, n=70, begin=(5, 0), end=(75, 70), Pmax=3, L=1, layer=0, Hq=4, Hkv=2)
    page = kvmm.kv4_page_bytes(c.shape)
    n_phys = (5 << 30) // (page if four else 32 * 128 * 2)
    far = n_phys - c.n_phys
    shape = kvmm.make_shape(c.B, c.L, c.Hq, c.Hkv, c.D, c.T, c.Pmax, 4, n_phys)
    wide = torch.empty(70 << 25, dtype=torch.bfloat16, device="cuda")

    def strided(x):  # (one at a time: they share the buffer)
        y = wide.as_strided(x.shape, (x.shape[2] * x.shape[3], 1 << 25, x.shape[3], 1))
        y.copy_(x)
        return y

    def run(shape, q, k, v, pools, table):
        meta, q_out = torch.zeros_like(c.meta), torch.zeros_like(c.q_out)
        if four:
            kvmm.kv4_append_rope(shape, 0, q, k, v, c.tb, c.te, *pools, table, meta, rope=c.rope, q_out=q_out, err=c.err)
        else:
            kvmm.kv_append_rope(shape, 0, q, k, v, c.tb, c.te, *pools, table, meta, rope=c.rope, q_out=q_out, err=c.err)
        torch.cuda.synchronize()
        assert int(c.err) == 0
        return meta, q_out

    if four:
        near_pools = [torch.zeros(c.n_phys, page, dtype=torch.uint8, device="cuda")]
    else:
        near_pools = [torch.zeros_like(c.k_pool), torch.zeros_like(c.v_pool)]
    far_pools = [torch.empty(n_phys, *p.shape[1:], dtype=p.dtype, device="cuda") for p in near_pools]
    for p in far_pools:
        p[far:] = 0
    want = run(c.shape, c.q, c.k, c.v, near_pools, c.table)
    got = run(shape, c.q, strided(c.k), c.v, far_pools, c.table + far)
    for x, y in zip(want, got):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))
    for x, y in zip(near_pools, far_pools):
        assert torch.equal(x.view(torch.uint8), y[far:].view(torch.uint8))
    again = [torch.zeros_like(p) for p in near_pools]
    got = run(c.shape, strided(c.q), c.k, c.v, again, c.table)
    assert torch.equal(want[1], got[1])
    run(c.shape, c.q, c.k, strided(c.v), again, c.table)
    for x, y in zip(near_pools, again):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
