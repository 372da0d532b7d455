"""A step of speculative decoding as a program takes it: rotate and append the nodes, select, attend, verify, keep."""
import numpy as np
import pytest
import torch

from paged_kv_cache_minmax_gb300 import kvmm
from paged_kv_cache_minmax_gb300.runtime import DecodeState, TreeDecode

pytestmark = pytest.mark.gpu


def build(B=3, L=2, Hq=8, Hkv=2, D=64, T=16, Pmax=24, K=6, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n_phys = B * L * Hkv * Pmax
    k = torch.zeros(n_phys, T, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros(n_phys, D, T, dtype=torch.bfloat16, device="cuda")
    table = torch.randperm(n_phys, generator=g, device="cuda").to(torch.int32).view(B, L, Hkv, Pmax).contiguous()
    seq = torch.zeros(B, dtype=torch.int32, device="cuda")
    st = DecodeState(B, L, Hq, Hkv, D, T, Pmax, K, k, v, table, seq)
    i = torch.arange(D // 2, dtype=torch.float64, device="cuda")
    a = torch.arange(Pmax * T, dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (-2.0 * i / D)
    rope = kvmm.Rope(torch.stack([a.cos(), a.sin()], 1).float().contiguous(), D)
    return st, rope, g


def rows(g, B, n, H, D):
    return torch.randn(B, n, H, D, generator=g, device="cuda").to(torch.bfloat16)


@pytest.mark.parametrize("every_page", [True, False])
def test_steps_leave_what_appending_the_accepted_tokens_leaves(every_page):
    """After each step the settled tokens' pages and bounds equal those of a state that appended the accepted rows alone,
    and a path's attention equals decode attention token by token, within the bf16 rounding of its weights and result."""
    B, L, Hq, Hkv, D, V, n = 3, 2, 8, 2, 64, 300, 7
    st, rope, g = build()
    ref, rope2, _ = build()
    lens = [37, 0, 130]
    for l in range(L):
        k, v = rows(g, B, 130, Hkv, D), rows(g, B, 130, Hkv, D)
        begin, end = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.tensor(lens, dtype=torch.int32, device="cuda")
        for s in (st, ref):
            kvmm.kv_append_rope(s.shape, l, None, k, v, begin, end, s.k_pool, s.v_pool, s.block_table, s.meta, rope=rope, err=s.err)
    st.seq_len.copy_(end)
    ref.seq_len.copy_(end)
    parent = torch.tensor([[-1, 0, 0, 1, 1, 2, 3], [-1, 0, 1, 2, 3, 4, 5], [-1, 0, 0, 0, 3, 3, 4]], dtype=torch.int32, device="cuda")
    tree = TreeDecode(st, parent, rope)
    depth = [[0, 1, 1, 2, 2, 2, 3], [0, 1, 2, 3, 4, 5, 6], [0, 1, 1, 1, 2, 2, 3]]
    assert tree.depth.tolist() == depth
    for step in range(4):
        nodes = torch.tensor([n, n - step % 2, n - step], dtype=torch.int32, device="cuda")
        tree.begin(nodes)
        q, k, v = ([rows(g, B, n, H, D) for _ in range(L)] for H in (Hq, Hkv, Hkv))
        for l in range(L):
            tree.layer_step(l, q[l], k[l], v[l], every_page=every_page)
        target = torch.softmax(torch.randn(B, n, V, generator=g, device="cuda") * 3, -1)
        draft = torch.softmax(target.log() + 0.3 * torch.randn(B, n, V, generator=g, device="cuda"), -1)
        par = parent.long().clamp(min=0)
        tokens = torch.multinomial(draft[torch.arange(B, device="cuda")[:, None], par].flatten(0, 1), 1, generator=g).view(B, n)
        tree.verify(target, tokens.to(torch.int32), torch.rand(B, n, generator=g, device="cuda"),
                    torch.rand(B, generator=g, device="cuda"), draft_probs=draft)
        torch.cuda.synchronize()
        path, count = tree.path.cpu().numpy(), tree.path_len.tolist()
        outs = tree.out.clone()
        tree.keep()
        # the same tokens one at a time
        for j in range(max(count)):
            at = torch.tensor([path[b][min(j, count[b] - 1)] for b in range(B)], device="cuda")
            ok = torch.tensor([j < c for c in count], device="cuda")
            begin = ref.seq_len.clone()
            ref.seq_len.add_(ok.to(torch.int32))
            b = torch.arange(B, device="cuda")
            for l in range(L):
                one = [t[b, at].unsqueeze(1).contiguous() for t in (q[l], k[l], v[l])]
                kvmm.kv_append_rope(ref.shape, l, *one, begin, ref.seq_len, ref.k_pool, ref.v_pool, ref.block_table, ref.meta,
                                    rope=rope2, q_out=ref.q_turned[l], err=ref.err)
                if every_page:
                    ref.sel_idx.copy_(torch.arange(ref.K, device="cuda").expand_as(ref.sel_idx))
                    full = kvmm.make_shape(B, L, Hq, Hkv, D, 16, 24, 24, ref.shape.n_phys)
                    sel = torch.arange(24, dtype=torch.int32, device="cuda").expand(B, L, Hkv, 24).contiguous()
                    cnt = ((ref.seq_len + 15) // 16).view(B, 1, 1).expand(B, L, Hkv).to(torch.int32).contiguous()
                    kvmm.sparse_paged_decode_attn(full, l, ref.q_turned[l], ref.k_pool, ref.v_pool, ref.block_table, ref.seq_len, sel,
                                                  cnt, ref.out[l], ref.workspace, err=ref.err)
                    d = (outs[l][b, at].float() - ref.out[l])[ok].abs().max().item()
                    # weights and outputs to bf16 on one side, weights on the other: 3 half steps of values up to 4.5
                    assert d <= 3 * 2.0 ** -8 * 4.5, d
        assert torch.equal(st.seq_len, ref.seq_len)
        for bb in range(B):
            N = int(st.seq_len[bb])
            t = torch.arange(N, device="cuda")
            for l in range(L):
                for h in range(Hkv):
                    x, y = (s.block_table[bb, l, h].long()[t // 16] for s in (st, ref))
                    assert torch.equal(st.k_pool[x, t % 16], ref.k_pool[y, t % 16])
                    assert torch.equal(st.v_pool[x, :, t % 16], ref.v_pool[y, :, t % 16])
            pages = -(-N // 16)
            assert torch.equal(st.meta[bb, :, :, :pages], ref.meta[bb, :, :, :pages])
    assert st.read_err() == 0 and ref.read_err() == 0


def test_a_captured_step():
    """The whole step replays from a graph, with new rows and random numbers each time."""
    B, L, Hq, Hkv, D, V, n = 2, 2, 8, 2, 64, 200, 5
    st, rope, g = build(B=B)
    ref, _, _ = build(B=B)
    parent = torch.tensor([[-1, 0, 0, 1, 2]] * B, dtype=torch.int32, device="cuda")
    trees = [TreeDecode(s, parent, rope) for s in (st, ref)]
    q, k, v = (rows(g, B, n, H, D) for H in (Hq, Hkv, Hkv))
    target = torch.softmax(torch.randn(B, n, V, generator=g, device="cuda") * 4, -1)
    tokens = target.argmax(-1)[:, [0, 0, 0, 1, 2]].to(torch.int32)
    u, un = torch.rand(B, n, device="cuda"), torch.rand(B, device="cuda")

    def step(t):
        t.begin()
        for l in range(L):
            t.layer_step(l, q, k, v)
        t.verify(target, tokens, u, un)
        t.keep()

    for s in (st, ref):
        s.seq_len.fill_(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(trees[0])
    torch.cuda.current_stream().wait_stream(side)
    step(trees[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(trees[0])
    for _ in range(5):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        u.copy_(torch.rand(u.shape, generator=g, device="cuda"))
        un.copy_(torch.rand(un.shape, generator=g, device="cuda"))
        graph.replay()
        step(trees[1])
        torch.cuda.synchronize()
        for a, b in ((trees[0].out, trees[1].out), (trees[0].path, trees[1].path), (trees[0].out_tokens, trees[1].out_tokens),
                     (st.seq_len, ref.seq_len), (st.meta, ref.meta)):
            assert torch.equal(a, b)
    assert st.read_err() == 0
    assert np.all(st.seq_len.cpu().numpy() >= 6)
