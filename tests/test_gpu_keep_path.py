"""kv_keep_path against the plain implementation: rows and bounds are equal bit by bit."""
import numpy as np
import pytest
import torch

from paged_kv_cache_minmax_gb300 import kvmm
from tests import tree_plain

pytestmark = pytest.mark.gpu


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


class Case:
    def __init__(self, lens, paths, n, L=2, Hkv=2, D=64, T=16, Pmax=None, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.lens, self.paths, self.n = list(lens), [list(x) for x in paths], n
        B = len(lens)
        self.B, self.L, self.Hkv, self.D, self.T = B, L, Hkv, D, T
        P = max(lens) // T + n // T + 3 if Pmax is None else Pmax
        self.P = P
        n_phys = B * L * Hkv * P + 2
        self.table = torch.randperm(n_phys, generator=g, device="cuda")[:B * L * Hkv * P].to(torch.int32).view(B, L, Hkv, P)
        self.table = self.table.contiguous()
        self.k_pool = torch.randn(n_phys, T, D, generator=g, device="cuda").to(torch.bfloat16)
        self.k_pool[:, ::3, ::5] = -0.0
        self.v_pool = torch.randn(n_phys, D, T, generator=g, device="cuda").to(torch.bfloat16)
        self.meta = torch.full((B, L, Hkv, P, 2, D), 3.0, dtype=torch.bfloat16, device="cuda")
        self.shape = kvmm.make_shape(B, L, Hkv, Hkv, D, T, P, 1, n_phys)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.seq = torch.tensor(lens, **i32)
        self.path = torch.tensor([x + [-1] * (n - len(x)) for x in self.paths], **i32).view(B, n)
        self.len = torch.tensor([len(x) for x in self.paths], **i32)
        self.err = torch.zeros(1, **i32)
        self.before = self.k_pool.clone(), self.v_pool.clone()

    def call(self, layer=-1, **kw):
        a = dict(meta=self.meta, err=self.err)
        a.update(kw)
        kvmm.kv_keep_path(self.shape, layer, self.path, self.len, self.seq, self.k_pool, self.v_pool, self.table, **a)

    def check(self, layer=-1, err=0, skip=(), still=()):
        """skip: (page) whose entries lead nowhere; still: sequences that nothing is done to."""
        torch.cuda.synchronize()
        assert int(self.err) == err
        T, D, P = self.T, self.D, self.P
        k0, v0 = (bits(x) for x in self.before)
        k1, v1 = k0.copy(), v0.copy()
        meta = bits(torch.full_like(self.meta, 3.0))
        table = self.table.cpu().numpy()
        for b in range(self.B):
            if b in still:
                continue
            seq, path = self.lens[b], self.paths[b]
            for l in range(self.L):
                if layer not in (-1, l):
                    continue
                for h in range(self.Hkv):
                    t = table[b, l, h]
                    for j, i in enumerate(path):
                        come, go = seq + i, seq + j
                        if come >= P * T or come // T in skip or go // T in skip:
                            continue
                        k1[t[go // T], go % T] = k0[t[come // T], come % T]
                        v1[t[go // T], :, go % T] = v0[t[come // T], :, come % T]
                    end = min(seq + len(path), P * T)
                    for p in range(seq // T, -(-end // T)):
                        if p in skip:
                            continue
                        rows = k1[t[p], :end - p * T].astype(np.int32)
                        key = np.where(rows >= 0x8000, 0xFFFF - rows, rows + 0x8000)
                        lo, hi = key.min(0), key.max(0)
                        for x, y in ((0, lo), (1, hi)):
                            meta[b, l, h, p, x] = np.where(y >= 0x8000, y - 0x8000, 0xFFFF - y)
        assert np.array_equal(bits(self.k_pool), k1)
        assert np.array_equal(bits(self.v_pool), v1)
        assert np.array_equal(bits(self.meta), meta)


def random_paths(r, B, n):
    return [[0] + sorted(r.choice(np.arange(1, n), r.randint(0, n), replace=False).tolist()) if n > 1 else [0] for _ in range(B)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [16, 32])
@pytest.mark.parametrize("n", [1, 2, 8, 33, 64])
@pytest.mark.parametrize("seed", [0, 1])
def test_rows_and_bounds(D, T, n, seed):
    r = np.random.RandomState(seed + n)
    c = Case([0, 5, 16, 31, 100], random_paths(r, 5, n), n, D=D, T=T, seed=seed)
    c.call()
    c.check()


@pytest.mark.parametrize("at", list(range(0, 33)))
def test_every_start_in_a_page(at):
    c = Case([at], [[0, 2, 3, 7, 20, 21]], 22, seed=at, Hkv=3)
    c.call()
    c.check()


def test_one_layer_alone():
    c = Case([40, 3], [[0, 3], [1, 2]], 5, L=3, seed=3)
    c.call(layer=1)
    c.check(layer=1)


def test_nothing_to_move():
    """The path is a prefix, or nothing: rows stay, bounds are taken again; a whole number of pages and no node: nothing."""
    c = Case([40, 3, 32], [[0, 1, 2], [], []], 5, seed=4)
    c.call()
    c.check()


def test_long_paths_of_many_sequences():
    r = np.random.RandomState(5)
    c = Case([(11 * b) % 70 for b in range(40)], random_paths(r, 40, 16), 16, L=5, Hkv=4, D=128, seed=5)
    c.call()
    c.check()


def test_no_bounds_no_error_word():
    c = Case([40], [[0, 3, 4]], 5, seed=6)
    c.call(meta=None, err=None)
    c.meta.fill_(3.0)
    k, v = c.k_pool.clone(), c.v_pool.clone()
    c.k_pool.copy_(c.before[0])
    c.v_pool.copy_(c.before[1])
    c.call()
    c.check()
    assert torch.equal(k, c.k_pool) and torch.equal(v, c.v_pool)


def test_to_the_last_slot():
    c = Case([58], [[0, 3, 5]], 6, Pmax=4, seed=7)
    c.call()
    c.check()
    c = Case([60], [[0, 2, 3, 4, 9]], 10, Pmax=4, seed=7)  # nodes 4 and 9 have no place
    c.call()
    c.check(err=kvmm.ERR_OUT_OF_RANGE)


@pytest.mark.parametrize("path,m", [([0, 2, 2], 3), ([0, 3, 1], 3), ([-1, 1, 2], 3), ([0, 1, 8], 3), ([0, 1, 2], 9), ([0, 1, 2], -1)])
def test_impossible_paths(path, m):
    """The sequence is left as it was; the others are not."""
    c = Case([40, 41], [[0, 2, 5], [0, 1, 2]], 8, seed=8)
    c.path[1, :3] = torch.tensor(path, dtype=torch.int32)
    c.len[1] = m
    c.call()
    c.check(err=kvmm.ERR_OUT_OF_RANGE, still=(1,))


@pytest.mark.parametrize("seq", [-1, 10 ** 6, 2 ** 31 - 1])
def test_impossible_lengths(seq):
    c = Case([40, 41], [[0, 2, 5], [0, 1, 2]], 8, seed=8)
    c.seq[1] = seq
    c.call()
    c.check(err=kvmm.ERR_OUT_OF_RANGE, still=(1,))


@pytest.mark.parametrize("entry", [-1, 1 << 30])
@pytest.mark.parametrize("page", [2, 3])
def test_pages_without_a_place(entry, page):
    c = Case([40], [[0, 3, 9, 12]], 14, L=1, seed=9)
    c.table[0, 0, :, page] = entry
    c.call()
    c.check(err=kvmm.ERR_NULL_BLOCK if entry < 0 else kvmm.ERR_OUT_OF_RANGE, skip=(page,))


def test_stream_and_graph():
    c = Case([40, 7], [[0, 3], [0, 1, 4]], 5, seed=10)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.call(stream=side)
    side.synchronize()
    c.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call()
    c.k_pool.copy_(c.before[0])
    c.v_pool.copy_(c.before[1])
    g.replay()
    c.check()


def test_refusals():
    c = Case([40], [[0, 3]], 5, seed=1)
    with pytest.raises(kvmm.KvmmError, match="invalid"):
        c.call(layer=2)
    with pytest.raises(ValueError, match="path"):
        kvmm.kv_keep_path(c.shape, -1, c.path[0], c.len, c.seq, c.k_pool, c.v_pool, c.table)
    with pytest.raises(ValueError, match="meta"):
        c.call(meta=c.meta.float())
