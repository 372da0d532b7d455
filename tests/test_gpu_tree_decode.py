"""TreeDecode on the GPU: what its steps do beyond the calls they are made of."""
import numpy as np
import pytest
import torch

from paged_kv_cache_minmax_gb300 import kvmm
from paged_kv_cache_minmax_gb300.runtime import TreeDecode
from tests import tree_plain
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


@pytest.mark.parametrize("mask", [None, [[1, 0], [0, 1]], [[0, 0], [0, 0]]])
def test_pages_are_selected_by_the_roots_queries(mask):
    """A step over selected pages: rescored units hold the root's own best pages, the others those of the step before; every
    node attends over exactly these and over its ancestors."""
    K, T, n = 6, 16, N
    st, rope, g = build(B=B, K=K)
    parent = [[-1, 0, 0, 1, 2], [-1, 0, 1, 1, 0]]
    tree = TreeDecode(st, torch.tensor(parent, dtype=torch.int32, device="cuda"), rope)
    end = torch.tensor([250, 170], dtype=torch.int32, device="cuda")
    for l in range(L):
        k, v = rows(g, B, 250, HKV, D), rows(g, B, 250, HKV, D)
        kvmm.kv_append_rope(st.shape, l, None, k, v, torch.zeros_like(end), end, st.k_pool, st.v_pool, st.block_table, st.meta,
                            rope=rope, err=st.err)
    st.seq_len.copy_(end)
    rescore = None if mask is None else torch.tensor(mask, dtype=torch.uint8, device="cuda")
    for step in range(2):
        tree.begin()
        was = st.sel_idx.clone()
        for l in range(L):
            tree.layer_step(l, rows(g, B, n, HQ, D), rows(g, B, n, HKV, D), rows(g, B, n, HKV, D),
                            rescore_mask=rescore if step else None)
        torch.cuda.synchronize()
        meta, sel, cnt = st.meta.double().cpu().numpy(), st.sel_idx.cpu().numpy(), st.sel_cnt.cpu().numpy()
        k_pool, v_pool = st.k_pool.double().cpu().numpy(), st.v_pool.double().cpu().numpy()
        table, bits, G = st.block_table.cpu().numpy(), tree_plain.masks(parent), HQ // HKV
        for b in range(B):
            seq = int(end[b])
            pages = -(-seq // T)
            for l in range(L):
                q = tree.q_turned[l, b].double().cpu().numpy()
                for h in range(HKV):
                    got = sel[b, l, h, :cnt[b, l, h]]
                    assert cnt[b, l, h] == K and len(set(got)) == K and got.max() < pages
                    if step and mask is not None and not mask[l][h]:
                        assert (got == was[b, l, h].cpu().numpy()).all()
                    else:
                        lo, hi = meta[b, l, h, :pages, 0], meta[b, l, h, :pages, 1]
                        score = sum(np.maximum(q[0, h * G + i] * lo, q[0, h * G + i] * hi).sum(-1) for i in range(G))
                        rest = np.setdiff1d(np.arange(pages), got)
                        # scores of G * D products in fp32
                        slack = G * D * 2.0 ** -23 * np.abs(score).max()
                        assert score[got].min() >= score[rest].max() - slack
                    tok = np.arange(seq + n)
                    old = (tok < seq) & np.isin(tok // T, got)
                    shown = np.stack([old | ((tok >= seq) & ((int(bits[b, i]) >> np.maximum(tok - seq, 0)) & 1 == 1)) for i in range(n)])
                    at = table[b, l, h, tok // T]
                    rows_q = q[:, h * G:(h + 1) * G].reshape(n * G, D)
                    o, lse, weighted, size = tree_plain.attend(rows_q, k_pool[at, tok % T], v_pool[at, :, tok % T],
                                                               shown.repeat(G, 0), D ** -0.5)
                    out = tree.out[l, b, :, h * G:(h + 1) * G].double().cpu().numpy().reshape(n * G, D)
                    assert (np.abs(out - o) <= tree_plain.out_bound(o, weighted, size, D, seq + n)).all()
                    off = np.abs(tree.lse[l, b, :, h * G:(h + 1) * G].double().cpu().numpy().reshape(-1) - lse)
                    assert (off <= tree_plain.lse_bound(lse, size, D, seq + n)).all()
    assert st.read_err() == 0


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
