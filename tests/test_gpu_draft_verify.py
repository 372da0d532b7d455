"""draft_verify against the plain implementation: whole numbers, so every path and token is equal."""
import numpy as np
import pytest
import torch

from paged_kv_cache_minmax_gb300 import kvmm
from tests import tree_plain

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, B, n, V, kind="rows", width=1, sharp=2.0, seed=0, pad=0, near=0.4, nodes=None):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        r = np.random.RandomState(seed)
        self.B, self.n, self.V, self.kind = B, n, V, kind
        z = torch.randn(B, n, V, generator=g, device="cuda") * sharp
        wide = torch.full((B, n, V + pad), float("nan"), device="cuda")
        wide[..., :V] = torch.softmax(z, -1)
        self.target = wide[..., :V]
        z = z + near * torch.randn(B, n, V, generator=g, device="cuda")
        self.draft = None
        if kind != "certain":
            wide = torch.full((B, n, V + 2 * pad), float("nan"), device="cuda")
            wide[..., :V] = torch.softmax(z, -1)
            self.draft = wide[..., :V]
        parent = np.full((B, n), -1, dtype=np.int32)
        tokens = r.randint(0, V, (B, n)).astype(np.int32)
        zc = z.cpu().numpy()
        noise = r.gumbel(size=z.shape)
        for b in range(B):
            for i in range(1, n):
                parent[b, i] = r.randint(max(0, i - width), i)
                at = parent[b, i]
                k = int((parent[b, 1:i] == at).sum())
                if kind == "rows":
                    tokens[b, i] = (zc[b, at] + r.gumbel(size=V)).argmax()
                else:
                    order = np.argsort(-(zc[b, at] + (noise[b, at] if kind == "distinct" else 0)))
                    tokens[b, i] = order[min(k, V - 1)]
        i32 = dict(dtype=torch.int32, device="cuda")
        self.parent, self.tokens = torch.from_numpy(parent).cuda(), torch.from_numpy(tokens).cuda()
        self.u = torch.rand(B, n, generator=g, device="cuda")
        self.u_next = torch.rand(B, generator=g, device="cuda")
        self.nodes = None if nodes is None else torch.tensor(nodes, **i32)
        self.path, self.said = torch.full((B, n), 77, **i32), torch.full((B, n), 77, **i32)
        self.len, self.err = torch.full((B,), 77, **i32), torch.zeros(1, **i32)

    def call(self, **kw):
        a = dict(draft_probs=self.draft, n_nodes=self.nodes, distinct=self.kind == "distinct", err=self.err)
        a.update(kw)
        kvmm.draft_verify(self.target, self.tokens, self.parent, self.u, self.u_next, self.path, self.len, self.said, **a)

    def check(self, err=0):
        torch.cuda.synchronize()
        assert int(self.err) == err
        total = 0
        for b in range(self.B):
            m = self.n if self.nodes is None else int(self.nodes[b].clamp(0, self.n))
            path, said = tree_plain.verify(self.target[b].cpu().numpy(), None if self.draft is None else self.draft[b].cpu().numpy(),
                                           self.tokens[b].tolist(), self.parent[b].tolist(), self.u[b].tolist(),
                                           float(self.u_next[b]), self.kind == "distinct", m)
            pad = [-1] * (self.n - len(path))
            assert int(self.len[b]) == len(path), b
            assert self.path[b].tolist() == path + pad, b
            assert self.said[b].tolist() == said + pad, b
            total += len(path)
        return total


@pytest.mark.parametrize("kind", ["rows", "distinct", "certain"])
@pytest.mark.parametrize("V", [1, 2, 31, 33, 1000, 4099, 32000])
@pytest.mark.parametrize("B,n,width", [(3, 1, 1), (5, 6, 1), (4, 12, 4), (2, 64, 3)])
def test_paths_and_tokens(kind, V, B, n, width):
    c = Case(B, n, V, kind, width, seed=V + n)
    c.call()
    assert c.check() >= B


@pytest.mark.parametrize("kind", ["rows", "distinct", "certain"])
def test_large_vocabularies_and_padded_rows(kind):
    c = Case(3, 7, 131072 + 13, kind, 3, sharp=4.0, seed=5, pad=19)
    c.call()
    c.check()
    c = Case(1, 3, 600001, kind, 2, sharp=4.0, seed=6)
    c.call()
    c.check()


@pytest.mark.parametrize("kind", ["rows", "distinct", "certain"])
def test_wide_trees_reject_many(kind):
    """Every node hangs from the root and the draft is far from the target: many rejections at one node."""
    c = Case(6, 40, 500, kind, 40, sharp=2.0, near=3.0, seed=9)
    c.parent[:, 1:] = 0
    if kind != "rows":
        z = torch.rand(6, 500, device="cuda").argsort(-1)[:, :39]
        c.tokens[:, 1:] = z.to(torch.int32)
    c.u.fill_(0.999)
    c.call()
    c.check()


def test_the_same_token_twice():
    for kind in ("rows", "distinct", "certain"):
        c = Case(4, 10, 50, kind, 10, seed=10)
        c.parent[:, 1:] = 0
        c.tokens[:, 1:] = c.tokens[:, 1:2]
        c.u.fill_(0.97)
        c.call()
        c.check()


def test_equal_distributions_accept_everything():
    c = Case(8, 9, 3000, "rows", 1, near=0.0, seed=11)
    c.call()
    assert c.check() == 72


def test_ends_of_the_random_numbers():
    for u in (0.0, 1.0 - 2.0 ** -24):
        for kind in ("rows", "distinct", "certain"):
            c = Case(4, 6, 777, kind, 2, seed=12)
            c.u.fill_(u)
            c.u_next.fill_(u)
            c.call()
            c.check()


def test_one_hot_rows():
    """Greedy: rows with a single 1, and a draft that is certain of another token."""
    c = Case(5, 6, 40, "rows", 1, seed=13)
    best = torch.randint(0, 40, (5, 6), device="cuda")
    c.target = torch.nn.functional.one_hot(best, 40).float()
    c.tokens[:, 1:] = best[:, :-1].to(torch.int32)
    c.tokens[2, 3] = (c.tokens[2, 3] + 1) % 40
    c.call()
    assert c.check() == 4 * 6 + 3
    assert c.said[2, 2] == best[2, 2]
    c.call(draft_probs=None)
    c.draft = None
    c.check()


def test_rows_without_weight():
    """A target row of zeros gives token 0; a residual of nothing the row itself."""
    c = Case(2, 1, 300, "certain", seed=14)
    c.target = c.target.contiguous()
    c.target[0] = 0
    c.call()
    c.check()
    assert int(c.said[0, 0]) == 0
    c = Case(1, 2, 4, "certain", seed=14)  # the only token with weight is rejected
    c.target = torch.tensor([[[0, 0.5, 0, 0], [1, 0, 0, 0]]], device="cuda")
    c.tokens[0, 1] = 1
    c.u.fill_(0.75)
    c.call()
    c.check()
    assert c.said.tolist() == [[1, -1]]


def test_nodes_that_do_not_exist():
    c = Case(5, 8, 200, "rows", 2, seed=15, nodes=[8, 0, 3, 1, 5])
    c.tokens[2, 3:] = -9
    c.parent[4, 5:] = 99
    c.call()
    c.check()
    assert int(c.len[1]) == 0
    c = Case(2, 8, 200, "rows", 2, seed=15, nodes=[9, -1])
    c.call()
    c.check(err=kvmm.ERR_OUT_OF_RANGE)


@pytest.mark.parametrize("what,value", [("tokens", -1), ("tokens", 200), ("tokens", 1 << 30), ("parent", -1), ("parent", 4),
                                        ("parent", 1 << 30)])
def test_impossible_nodes(what, value):
    for kind in ("rows", "certain"):
        c = Case(3, 8, 200, kind, 1, near=0.0, seed=16)
        getattr(c, what)[1, 4] = value
        c.call()
        c.check(err=kvmm.ERR_OUT_OF_RANGE)
        assert int(c.len[1]) <= 4


def test_odd_probabilities_do_no_harm():
    """NaN, infinite and negative entries: no promise but that the call ends and names a token."""
    c = Case(4, 6, 1000, "rows", 2, seed=17)
    for t in (c.target, c.draft):
        t[0, :, ::3] = float("nan")
        t[1, :, ::5] = float("inf")
        t[2] = -1.0
    c.call()
    torch.cuda.synchronize()
    last = c.said.gather(1, (c.len.long() - 1).unsqueeze(1))
    assert (c.len >= 1).all() and (last >= 0).all() and (last < 1000).all()


def test_more_sequences_than_run_at_once():
    c = Case(700, 4, 300, "distinct", 2, seed=19)
    c.call()
    c.check()


def test_stream_and_graph():
    c = Case(6, 8, 5000, "distinct", 3, seed=18)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.call(stream=side)
    side.synchronize()
    c.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call()
    c.u.copy_(torch.rand_like(c.u))
    c.u_next.copy_(torch.rand_like(c.u_next))
    g.replay()
    c.check()
    g.replay()
    c.check()


def test_refusals():
    c = Case(2, 4, 100, seed=1)
    with pytest.raises(ValueError, match="target_probs"):
        kvmm.draft_verify(c.target.half(), c.tokens, c.parent, c.u, c.u_next, c.path, c.len, c.said)
    with pytest.raises(ValueError, match="target_probs"):
        kvmm.draft_verify(c.target[0], c.tokens, c.parent, c.u, c.u_next, c.path, c.len, c.said)
    with pytest.raises(ValueError, match="draft_probs"):
        c.call(draft_probs=c.draft[:, :3])
    with pytest.raises(ValueError, match="draft_probs"):
        c.call(draft_probs=c.draft.transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(ValueError, match="tokens"):
        kvmm.draft_verify(c.target, c.tokens[:, :3], c.parent, c.u, c.u_next, c.path, c.len, c.said)
    with pytest.raises(ValueError, match="u_accept"):
        kvmm.draft_verify(c.target, c.tokens, c.parent, c.u[:, :3], c.u_next, c.path, c.len, c.said)
    with pytest.raises(kvmm.KvmmError, match="unsupported"):
        big = Case(1, 64, 10, seed=1)
        z = torch.zeros(1, 65, 10, device="cuda")
        i = torch.zeros(1, 65, dtype=torch.int32, device="cuda")
        kvmm.draft_verify(z, i, i, z[..., 0].contiguous(), big.u_next, i, big.len, i.clone())
