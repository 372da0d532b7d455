"""TreeDecode on the GPU: what its steps do beyond the calls they are made of."""
import pytest
import torch

from paged_kv_cache_minmax_gb300 import kvmm
from paged_kv_cache_minmax_gb300.runtime import TreeDecode
from tests.test_gpu_tree_step import build, rows

pytestmark = pytest.mark.gpu

B, L, HQ, HKV, D, V, N = 2, 2, 8, 2, 64, 200, 5


def test_replaced_trees_reach_a_captured_step():
    """A graph of a step replays with the trees set after its capture, as an eager step with them does."""
    (st, rope, g), (ref, _, _) = build(B=B), build(B=B)
    trees = [TreeDecode(s, torch.tensor([[-1, 0, 1, 2, 3]] * B, dtype=torch.int32, device="cuda"), rope) for s in (st, ref)]
    q, k, v = (rows(g, B, N, H, D) for H in (HQ, HKV, HKV))
    target = torch.softmax(torch.randn(B, N, V, generator=g, device="cuda") * 4, -1)
    tokens = target.argmax(-1)[:, [0, 0, 0, 1, 2]].to(torch.int32)
    u, un = torch.rand(B, N, generator=g, device="cuda"), torch.rand(B, generator=g, device="cuda")

    def step(t):
        t.begin()
        for l in range(L):
            t.layer_step(l, q, k, v)
        t.verify(target, tokens, u, un)
        t.keep()

    for t in trees:
        step(t)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(trees[0])
    keep = []
    for parent in ([[-1, 0, 0, 1, 2], [-1, 0, 0, 0, 0]], [[-1, 0, 1, 0, 3], [-1, 0, 0, 1, 1]]):
        for t in trees:
            t.set_trees(torch.tensor(parent, dtype=torch.int32, device="cuda"))
        keep += [torch.full((B, N), 1 << 40, device="cuda") for _ in range(64)]  # (what was freed is written over)
        graph.replay()
        step(trees[1])
        torch.cuda.synchronize()
        for a in ("out", "lse", "path", "path_len", "out_tokens", "positions"):
            assert torch.equal(getattr(trees[0], a), getattr(trees[1], a)), a
        assert torch.equal(st.seq_len, ref.seq_len) and torch.equal(st.meta, ref.meta)
    assert st.read_err() == 0 and ref.read_err() == 0


def test_a_table_that_is_full():
    """Accepted nodes beyond the table's end are told, and the settled tokens stop at its end."""
    st, rope, g = build(B=B)
    cap = 24 * 16
    tree = TreeDecode(st, torch.tensor([[-1, 0, 1, 2, 3]] * B, dtype=torch.int32, device="cuda"))
    st.seq_len.copy_(torch.tensor([cap - 2, 100], dtype=torch.int32))
    target = torch.zeros(B, N, V, device="cuda")
    target[:, :, 3] = 1  # every node's token is the target's
    one = torch.full((B, N), 3, dtype=torch.int32, device="cuda")
    for want in ([cap, 105], [cap, 110]):
        tree.begin()
        for l in range(L):
            tree.layer_step(l, rows(g, B, N, HQ, D), rows(g, B, N, HKV, D), rows(g, B, N, HKV, D), every_page=True)
        tree.verify(target, one, torch.zeros(B, N, device="cuda"), torch.zeros(B, device="cuda"))
        tree.keep()
        assert tree.path_len.tolist() == [N, N] and st.seq_len.tolist() == want
    assert st.read_err() == kvmm.ERR_OUT_OF_RANGE
