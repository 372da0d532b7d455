"""What a step of speculative decoding over the paged cache costs, case by case.

Three operators.  A step hands each sequence a tree of n nodes: node 0 is the token sampled last, the others are drafted;
their keys and values stand in the cache behind the seq_len tokens that are settled.

``sparse_paged_tree_attn``: attention of every node over the settled tokens (of the selected pages, or all pages) and over
the nodes that a bit mask shows it.  ``draft_verify``: which path of the tree the target's probabilities accept, from given
random numbers, and the token that follows it.  ``kv_keep_path``: the accepted nodes' rows moved to the end of the
sequence, in every layer, and the pages' key bounds taken again.

Verification counts in whole numbers: a probability is floor(p * 2^53), so that sums are exact in any order.

``run`` computes them with elementary torch operations in fp32, or, with ``own``, calls the framework.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False


# ------------------------------------------------------------------------------------------------------------------
# the cases
def _attend_case(name, **kw):
    c = dict(name=name, kind="attend", B=1, Hq=32, Hkv=8, D=128, T=16, tokens=0, n=8, K=0, ragged=False, chain=False)
    c.update(kw)
    return c


def _verify_case(name, **kw):
    c = dict(name=name, kind="verify", B=1, V=32000, n=5, width=1, draft="rows", sharp=2.5)
    c.update(kw)
    return c


def _keep_case(name, **kw):
    c = dict(name=name, kind="keep", B=1, L=32, Hkv=8, D=128, T=16, tokens=40, n=8)
    c.update(kw)
    return c


def listed():
    return [
        # the smallest: four drafted tokens in a row, one KV head of 1,024 tokens
        _attend_case("tree_tiny", Hq=4, Hkv=1, D=64, tokens=1021, n=4, chain=True),
        # one user's 4K chat, a tree of eight
        _attend_case("tree_4k_b1", tokens=4090),
        # 32K context, batch 8, 128 selected pages a head, trees of 16
        _attend_case("tree_32k_k128", B=8, tokens=32768, n=16, K=128),
        # every page of a ragged batch of up to 16K tokens, five query heads a KV head, pages of 32 tokens, 13 nodes
        _attend_case("tree_all_gqa5_b16", B=16, Hq=40, T=32, tokens=16381, n=13, ragged=True),
        # every page of one 128K sequence, the widest tree: 256 query rows a KV head
        _attend_case("tree_all_128k_n64", tokens=131072, n=64),
        # one user's chain of four drafted tokens, a vocabulary of 32,000
        _verify_case("verify_chain_b1"),
        # trees of 16 drawn without replacement for a batch of 8, a vocabulary of odd size
        _verify_case("verify_tree_b8", B=8, V=100003, n=16, width=3, draft="distinct"),
        # candidates that a head proposes with certainty, 24 a tree
        _verify_case("verify_certain_b16", B=16, V=131072, n=24, width=4, draft="certain", sharp=6.0),
        # chains of seven for a batch of 64
        _verify_case("verify_chain_b64", B=64, V=131072, n=8),
        # one sequence's accepted nodes in 32 layers
        _keep_case("keep_b1"),
        # other heads and pages, odd sizes
        _keep_case("keep_odd", B=5, L=7, Hkv=3, D=64, T=32, tokens=77, n=31),
        # a batch of 32 in 32 layers, trees of 16
        _keep_case("keep_b32_l32", B=32, tokens=50, n=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    kind = rng.choice(["attend", "attend", "attend", "verify", "verify", "keep"])
    if kind == "verify":
        n, V = _log(rng, 1, 64), _log(rng, 50, 160000)
        return dict(kind=kind, n=n, V=V, B=_log(rng, 1, max(1, min(64, (1 << 26) // (n * V)))), width=rng.choice([1, 1, 2, 3, 5]),
                    draft=rng.choice(["rows", "rows", "distinct", "certain"]), sharp=rng.choice([1.0, 2.5, 4.0, 6.0]))
    D, T = rng.choice([64, 128, 128]), rng.choice([16, 32])
    Hkv, n = rng.choice([1, 2, 3, 4, 5, 8, 8]), _log(rng, 1, 64)
    if kind == "keep":
        L, tokens = _log(rng, 1, 40), _log(rng, 1, 200)
        most = (1 << 26) // (L * Hkv * D * (tokens + n + 2 * T))
        return dict(kind=kind, L=L, Hkv=Hkv, D=D, T=T, tokens=tokens, n=n, B=_log(rng, 1, max(1, min(64, most))))
    G, B = rng.choice([1, 2, 3, 4, 4, 5, 7, 8]), _log(rng, 1, 48)
    most = min(131072, 2500000 // (B * Hkv), 250000000 // (B * Hkv * G * n))
    return dict(kind=kind, B=B, Hq=Hkv * G, Hkv=Hkv, D=D, T=T, tokens=_log(rng, 1, max(1, most)), n=n,
                K=0 if rng.random() < 0.5 else _log(rng, 1, 300), ragged=rng.random() < 0.6, chain=rng.random() < 0.3)


def _lens(c):
    """Settled tokens of each sequence."""
    n, B = c["tokens"], c["B"]
    if c["kind"] == "keep":
        return [max(0, n - 3 * b) for b in range(B)]
    if not c["ragged"]:
        return [n] * B
    got = [max(0, n - b * n // (2 * B) - (b * 7) % c["T"]) for b in range(B)]
    if B >= 3:
        got[B - 2] = 0  # a slot of the batch with no sequence
    return got


def _nodes(c):
    n, B = c["n"], c["B"]
    if not c.get("ragged"):
        return [n] * B
    got = [max(1, n - b % 3 * (n // 4)) for b in range(B)]
    if B >= 3:
        got[B - 2] = 0
    return got


def _kept(c):
    """Accepted nodes of each sequence."""
    return [1 + (5 * b + c["n"] // 2) % c["n"] for b in range(c["B"])]


def _picked(c):
    pages = [-(-s // c["T"]) for s in _lens(c)]
    return [min(c["K"], p) for p in pages] if c["K"] else pages


def work(c):
    B, n = c["B"], c["n"]
    if c["kind"] == "verify":
        # the row that the next token is drawn from, and the draft's where it is subtracted; each node's numbers
        row = 4 * c["V"] * (1 if c["draft"] == "certain" else 2)
        return {"bytes": B * (row + n * (4 * 6 + 8)), "flops": B * c["V"] * 3}
    Hkv, D, T = c["Hkv"], c["D"], c["T"]
    if c["kind"] == "keep":
        moved = sum(k - 1 for k in _kept(c))
        begun = sum(s // T * T for s in _lens(c))
        held = sum(s + k for s, k in zip(_lens(c), _kept(c))) - begun  # keys that the bounds are taken over
        pages = sum(-(-(s + k) // T) - s // T for s, k in zip(_lens(c), _kept(c)))
        units = c["L"] * Hkv
        return {"bytes": units * (moved * 2 * 4 * D + held * 2 * D + pages * (4 * D + 4)), "flops": units * held * D * 2}
    # a sequence's partial last page counts whole when only some pages are read, as any other
    toks = [(p * T if c["K"] else s) + m for s, p, m in zip(_lens(c), _picked(c), _nodes(c))]
    rows = [m * c["Hq"] for m in _nodes(c)]
    by = sum(toks) * Hkv * 4 * D + sum(rows) * (4 * D + 4) + sum(_picked(c)) * Hkv * (8 if c["K"] else 4)
    return {"bytes": by, "flops": sum(t * r for t, r in zip(toks, rows)) * 4 * D}


# ------------------------------------------------------------------------------------------------------------------
def _parents(c, seed):
    """Each sequence's tree: a node hangs from one of the last `width` before it."""
    r = np.random.RandomState(seed % (1 << 31))
    width = 1 if c.get("chain") else c.get("width", 3)
    par = np.full((c["B"], c["n"]), -1, dtype=np.int64)
    for i in range(1, c["n"]):
        par[:, i] = r.randint(max(0, i - width), i, c["B"])
    return par


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"attend": _prepare_attend, "verify": _prepare_verify, "keep": _prepare_keep}[c["kind"]](c, seed, gen)
    s["c"], s["err"] = c, torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _table(gen, B, L, Hkv, P):
    return torch.randperm(B * L * Hkv * P, generator=gen, device="cuda").to(torch.int32).view(B, L, Hkv, P)


def _prepare_attend(c, seed, gen):
    B, Hq, Hkv, D, T, n = c["B"], c["Hq"], c["Hkv"], c["D"], c["T"], c["n"]
    lens, nodes = _lens(c), _nodes(c)
    P = max(1, -(-max(a + b for a, b in zip(lens, nodes)) // T))
    n_phys = B * Hkv * P
    s = dict(P=P, n_phys=n_phys, table=_table(gen, B, 1, Hkv, P), seq_len=_ints(lens), n_nodes=_ints(nodes))
    # a few channels of the keys are far larger than the rest
    loud = torch.ones(D, device="cuda")
    loud[torch.randperm(D, generator=gen, device="cuda")[:4]] = 6.0
    s["k_pool"] = torch.empty(n_phys, T, D, dtype=torch.bfloat16, device="cuda")
    s["v_pool"] = torch.empty(n_phys, D, T, dtype=torch.bfloat16, device="cuda")
    step = max(1, (1 << 26) // (T * D))
    for i in range(0, n_phys, step):
        m = min(step, n_phys - i)
        s["k_pool"][i:i + m] = _normal(gen, m, T, D) * loud
        s["v_pool"][i:i + m] = _normal(gen, m, D, T)
    s["q"] = _normal(gen, B, n, Hq, D).to(torch.bfloat16)
    s["out"] = torch.zeros(B, n, Hq, D, dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.zeros(B, n, Hq, device="cuda")
    par = _parents(c, seed)
    bits = np.zeros((B, n), dtype=np.uint64)
    for i in range(n):
        bits[:, i] = (bits[np.arange(B), par[:, i]] if i else 0) | np.uint64(1 << i)
    s["mask"] = None if c["chain"] else torch.from_numpy(bits.view(np.int64)).cuda()
    s["sel"] = s["cnt"] = None
    if c["K"]:
        key = torch.rand(B, Hkv, P, generator=gen, device="cuda")
        past = torch.arange(P, device="cuda") >= _ints([-(-x // T) for x in lens]).view(B, 1, 1)
        at = key.masked_fill(past, 2.0).argsort(-1)[..., :c["K"]]
        at = at.masked_fill(torch.arange(at.shape[-1], device="cuda") >= _ints(_picked(c)).view(B, 1, 1), P)
        sel = torch.full((B, Hkv, c["K"]), P, dtype=torch.int64, device="cuda")
        sel[..., :at.shape[-1]] = at
        sel = sel.sort(-1).values
        s["sel"] = sel.masked_fill(sel == P, 0).to(torch.int32).view(B, 1, Hkv, -1)
        s["cnt"] = _ints(_picked(c)).view(B, 1, 1).expand(B, 1, Hkv).contiguous()
    return s


def _gumbel(gen, *shape):
    return -torch.log(-torch.log(torch.rand(*shape, generator=gen, device="cuda").clamp(1e-9, 1 - 1e-7)))


def _prepare_verify(c, seed, gen):
    B, V, n = c["B"], c["V"], c["n"]
    par = _parents(c, seed)
    z = _normal(gen, B, n, V) * c["sharp"]
    s = dict(target=torch.softmax(z, -1), draft=None)
    z += 0.5 * _normal(gen, B, n, V)  # what the draft model takes the target for
    tokens = torch.randint(0, V, (B, n), generator=gen, device="cuda")
    rank = np.zeros((B, n), dtype=np.int64)  # which child of its parent a node is
    for i in range(1, n):
        rank[:, i] = (par[:, 1:i] == par[:, i:i + 1]).sum(1)
    if c["draft"] == "rows":
        s["draft"] = torch.softmax(z, -1)
        for i in range(1, n):
            row = z[torch.arange(B, device="cuda"), _ints(par[:, i], torch.int64)]
            tokens[:, i] = (row + _gumbel(gen, B, V)).argmax(-1)
    else:
        if c["draft"] == "distinct":
            s["draft"] = torch.softmax(z, -1)
            z += _gumbel(gen, B, n, V)
        top = z.topk(min(V, int(rank.max()) + 1), -1).indices  # [B, n, most children]
        if n > 1:
            b = torch.arange(B, device="cuda").unsqueeze(1)
            tokens[:, 1:] = top[b, _ints(par[:, 1:], torch.int64), _ints(rank[:, 1:], torch.int64).clamp(max=top.shape[-1] - 1)]
    s["tokens"], s["parent"] = tokens.to(torch.int32), _ints(par)
    s["u"] = torch.rand(B, n, generator=gen, device="cuda")
    s["u_next"] = torch.rand(B, generator=gen, device="cuda")
    s["path"] = torch.zeros(B, n, dtype=torch.int32, device="cuda")
    s["path_len"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    s["out_tokens"] = torch.zeros(B, n, dtype=torch.int32, device="cuda")
    return s


def _prepare_keep(c, seed, gen):
    B, L, Hkv, D, T, n = c["B"], c["L"], c["Hkv"], c["D"], c["T"], c["n"]
    P = -(-(c["tokens"] + n) // T)
    s = dict(P=P, n_phys=B * L * Hkv * P, table=_table(gen, B, L, Hkv, P), seq_len=_ints(_lens(c)))
    s["k_pool"] = _normal(gen, s["n_phys"], T, D).to(torch.bfloat16)
    s["v_pool"] = _normal(gen, s["n_phys"], D, T).to(torch.bfloat16)
    s["meta"] = torch.zeros(B, L, Hkv, P, 2, D, dtype=torch.bfloat16, device="cuda")
    r = np.random.RandomState(seed % (1 << 31))
    path = np.full((B, n), -1, dtype=np.int64)
    for b, k in enumerate(_kept(c)):
        path[b, 1:k] = 1 + np.sort(r.permutation(n - 1)[:k - 1])
        path[b, 0] = 0
    s["path"], s["path_len"] = _ints(path), _ints(_kept(c))
    return s


def run(s):
    if own:
        return _run_own(s)
    return {"attend": _attend, "verify": _verify, "keep": _keep}[s["c"]["kind"]](s)


def _run_own(s):
    from paged_kv_cache_minmax_gb300 import kvmm

    c = s["c"]
    if c["kind"] == "verify":
        kvmm.draft_verify(s["target"], s["tokens"], s["parent"], s["u"], s["u_next"], s["path"], s["path_len"],
                          s["out_tokens"], draft_probs=s["draft"], distinct=c["draft"] == "distinct", err=s["err"])
        return {n: s[n] for n in ("path", "path_len", "out_tokens", "err")}
    if "shape" not in s:
        s["shape"] = kvmm.make_shape(c["B"], c.get("L", 1), c.get("Hq", c["Hkv"]), c["Hkv"], c["D"], c["T"], s["P"],
                                     max(1, c.get("K", 1)), s["n_phys"])
        s["ws"] = kvmm.alloc_tree_workspace(s["shape"], c["n"]) if c["kind"] == "attend" else None
    if c["kind"] == "keep":
        kvmm.kv_keep_path(s["shape"], -1, s["path"], s["path_len"], s["seq_len"], s["k_pool"], s["v_pool"], s["table"],
                          s["meta"], err=s["err"])
        return {n: s[n] for n in ("k_pool", "v_pool", "meta", "err")}
    kvmm.sparse_paged_tree_attn(s["shape"], 0, s["q"], s["k_pool"], s["v_pool"], s["table"], s["seq_len"], s["out"],
                                s["ws"], n_nodes=s["n_nodes"], tree_mask=s["mask"], sel_idx=s["sel"], sel_cnt=s["cnt"],
                                lse=s["lse"], err=s["err"])
    return {n: s[n] for n in ("out", "lse", "err")}


# ------------------------------------------------------------------------------------------------------------------
# the plain forms
def _attend(s):
    c = s["c"]
    B, Hq, Hkv, D, T, P, n = c["B"], c["Hq"], c["Hkv"], c["D"], c["T"], s["P"], c["n"]
    G = Hq // Hkv
    dev = s["q"].device
    seq, nodes = s["seq_len"].view(B, 1, 1).long(), s["n_nodes"].view(B, 1, 1).long()
    slots = torch.arange(T, device=dev)
    if c["K"]:
        # the selected pages' settled tokens, then the pages that hold nodes
        sel = s["sel"][:, 0].long()
        last = seq // T + torch.arange((n + T - 2) // T + 1, device=dev)
        page = torch.cat([sel, last.expand(B, Hkv, -1)], -1)
        picked = torch.arange(page.shape[-1], device=dev) < sel.shape[-1]
        here = torch.arange(page.shape[-1], device=dev) < s["cnt"][:, 0].unsqueeze(-1)
        tok = page.unsqueeze(-1) * T + slots
        old = ((tok < seq.unsqueeze(-1)) & (here & picked).unsqueeze(-1)).flatten(2)
        new = ~picked.unsqueeze(-1).expand(B, Hkv, -1, T).flatten(2)
        page = page.clamp(max=P - 1)
    else:
        page = torch.arange(P, device=dev).expand(B, Hkv, P)
        tok = page.unsqueeze(-1) * T + slots
        old = (tok < seq.unsqueeze(-1)).flatten(2)
        new = ~old
    j = tok.flatten(2) - seq
    new = new & (j >= 0) & (j < nodes)
    phys = s["table"][:, 0].long().gather(2, page)
    k = s["k_pool"][phys].float().flatten(2, 3)  # [B, Hkv, tokens, D]
    q = s["q"].float().view(B, n, Hkv, G, D).transpose(1, 2).flatten(2, 3)  # rows: node, then head of the group
    z = (q @ k.transpose(2, 3)) / math.sqrt(D)
    del k
    i = torch.arange(n, device=dev)
    bits = s["mask"] if s["mask"] is not None else (torch.ones_like(i) << i) * 2 - 1
    shown = (bits.expand(B, n).view(B, 1, n, 1) >> j.clamp(0, 63).unsqueeze(2)) & 1 > 0  # [B, Hkv, n, tokens]
    live = old.unsqueeze(2) | (new.unsqueeze(2) & shown)
    z = z.unflatten(2, (n, G)).masked_fill_(~live.unsqueeze(3), -math.inf)
    m = z.amax(-1, keepdim=True).clamp(min=-3e38)
    e = (z - m).exp_().flatten(2, 3)
    l = e.sum(-1, keepdim=True)
    v = s["v_pool"][phys].transpose(3, 4).float().flatten(2, 3)
    out = (e @ v) / l.clamp(min=1e-38)
    lse = torch.where(l > 0, m.flatten(2, 3) + l.log(), torch.full_like(l, -math.inf))
    there = i < s["n_nodes"].view(B, 1)  # rows behind a sequence's last node are left as they were
    s["out"][there] = out.view(B, Hkv, n, G, D).transpose(1, 2).reshape(B, n, Hq, D).to(torch.bfloat16)[there]
    s["lse"][there] = lse.view(B, Hkv, n, G).transpose(1, 2).reshape(B, n, Hq)[there]
    return {x: s[x] for x in ("out", "lse", "err")}


def _weights(p):
    """Probabilities (fp32) as whole multiples of 2^-53, rounded down."""
    return (p.double().clamp(0, 512) * 2.0 ** 53).long()


def _verify(s):
    c = s["c"]
    B, V, n = c["B"], c["V"], c["n"]
    dev = s["tokens"].device
    b, one = torch.arange(B, device=dev), 1 << 53
    tokens, cur = s["tokens"].long(), torch.zeros(B, dtype=torch.int64, device=dev)
    w, total, left = _weights(s["target"][:, 0]), torch.full((B,), one, device=dev), torch.ones(B, dtype=torch.float64, device=dev)
    took = torch.zeros(B, n, dtype=torch.bool, device=dev)
    took[:, 0] = True
    for i in range(1, n):  # a node's parent and elder siblings come before it: one walk visits the path in order
        x = tokens[:, i:i + 1]
        asked = s["parent"][:, i] == cur
        if s["draft"] is None:
            minus, at = None, total
        else:
            f = torch.where((total > 0) & (left > 0), total.double() * 2.0 ** -53 / left, torch.zeros_like(left)).float()
            minus = _weights(s["draft"][b, cur] * f.unsqueeze(1))
            at = minus.gather(1, x).squeeze(1)
        held = w.gather(1, x).squeeze(1)
        yes = asked & (s["u"][:, i].double() * at.double() < held.double())
        no = asked & ~yes
        if minus is None:
            less = w.scatter(1, x, 0)
            total = torch.where(no, (total - held).clamp(min=0), total)
        else:
            less = (w - minus).clamp(min=0)
            total = torch.where(no, less.sum(1), total)
            if c["draft"] == "distinct":
                left = torch.where(no, left - s["draft"][b, cur].gather(1, x).squeeze(1).double(), left)
        w = torch.where(no.unsqueeze(1), less, w)
        cur = torch.where(yes, torch.full_like(cur, i), cur)
        w = torch.where(yes.unsqueeze(1), _weights(s["target"][:, i]), w)
        total = torch.where(yes, torch.full_like(total, one), total)
        left = torch.where(yes, torch.ones_like(left), left)
        took[:, i] = yes
    w = torch.where((w.sum(1) == 0).unsqueeze(1), _weights(s["target"][b, cur]), w)
    total = w.sum(1)
    goal = torch.minimum((s["u_next"].double() * total.double()).long(), total - 1)
    following = (w.cumsum(1) <= goal.unsqueeze(1)).sum(1).clamp(max=V - 1)
    place = torch.arange(n, device=dev).expand(B, n)
    path = torch.where(took, place, torch.full_like(place, n)).sort(1).values
    length = took.sum(1)
    s["path"].copy_(torch.where(path < n, path, torch.full_like(path, -1)))
    s["path_len"].copy_(length)
    said = torch.cat([path[:, 1:], torch.full((B, 1), n, device=dev)], 1)
    said = torch.where(said < n, tokens.gather(1, said.clamp(max=n - 1)), torch.full_like(said, -1))
    s["out_tokens"].copy_(said.scatter(1, (length - 1).unsqueeze(1), following.unsqueeze(1)))
    return {x: s[x] for x in ("path", "path_len", "out_tokens", "err")}


def _keep(s):
    c = s["c"]
    B, T, P, n = c["B"], c["T"], s["P"], c["n"]
    dev = s["path"].device
    seq, kept = s["seq_len"].long(), s["path_len"].long()
    b, j = (torch.arange(n, device=dev) < kept.unsqueeze(1)).nonzero(as_tuple=True)
    come, go = seq[b] + s["path"][b, j].long(), seq[b] + j
    was, now = (s["table"][b, :, :, t // T].long() for t in (come, go))  # [rows, L, Hkv]
    k = s["k_pool"][was, (come % T).view(-1, 1, 1)]
    v = s["v_pool"][was, :, (come % T).view(-1, 1, 1)]
    s["k_pool"][now, (go % T).view(-1, 1, 1)] = k
    s["v_pool"][now, :, (go % T).view(-1, 1, 1)] = v
    end = seq + kept
    page = torch.arange(P, device=dev)
    b, p = ((page >= (seq // T).unsqueeze(1)) & (page * T < end.unsqueeze(1))).nonzero(as_tuple=True)
    keys = s["k_pool"][s["table"][b, :, :, p].long()].float()  # [pages, L, Hkv, T, D]
    past = (p.unsqueeze(1) * T + torch.arange(T, device=dev) >= end[b].unsqueeze(1)).view(-1, 1, 1, T, 1)
    s["meta"][b, :, :, p, 0] = keys.masked_fill(past, math.inf).amin(3).to(torch.bfloat16)
    s["meta"][b, :, :, p, 1] = keys.masked_fill(past, -math.inf).amax(3).to(torch.bfloat16)
    return {x: s[x] for x in ("k_pool", "v_pool", "meta", "err")}


# ------------------------------------------------------------------------------------------------------------------
# the same in 64 bits, from the definitions
def exact(c, seed):
    s = prepare(c, seed)
    return {"attend": _exact_attend, "verify": _exact_verify, "keep": _exact_keep}[c["kind"]](s)


def _exact_attend(s):
    c = s["c"]
    Hkv, D, T, n = c["Hkv"], c["D"], c["T"], c["n"]
    G = c["Hq"] // Hkv
    out, lse = s["out"].double(), s["lse"].double()
    bits = None if s["mask"] is None else s["mask"].cpu().numpy().view(np.uint64)
    for b, (seq, m) in enumerate(zip(_lens(c), _nodes(c))):
        if not m:
            continue
        see = np.tril(np.ones((n, n), dtype=bool)) if bits is None else (bits[b][:, None] >> np.arange(n, dtype=np.uint64)) & np.uint64(1) > 0
        see = torch.from_numpy(see[:m, :m]).cuda().repeat_interleave(G, 0)  # node rows x nodes
        for h in range(Hkv):
            table = s["table"][b, 0, h].long()

            def rows(tok):
                return s["k_pool"][table[tok // T], tok % T].double(), s["v_pool"][table[tok // T], :, tok % T].double()

            tok = torch.arange(seq, device="cuda")
            if c["K"]:
                tok = tok[torch.isin(tok // T, s["sel"][b, 0, h, :_picked(c)[b]].long())]
            k, v = rows(tok)
            kn, vn = rows(torch.arange(seq, seq + m, device="cuda"))
            q = s["q"][b, :m, h * G:(h + 1) * G].reshape(m * G, D).double()
            z = torch.cat([q @ k.T, (q @ kn.T).masked_fill(~see, -math.inf)], 1) / math.sqrt(D)
            lse[b, :m, h * G:(h + 1) * G] = torch.logsumexp(z, -1).view(m, G)
            out[b, :m, h * G:(h + 1) * G] = (torch.softmax(z, -1) @ torch.cat([v, vn])).view(m, G, D)
    return {"out": out, "lse": lse, "err": None}


def _exact_verify(s):
    c = s["c"]
    n = c["n"]
    tokens, parent, u, u_next = (s[x].cpu().numpy() for x in ("tokens", "parent", "u", "u_next"))
    path, length, said = np.full((c["B"], n), -1), np.zeros(c["B"], dtype=np.int64), np.full((c["B"], n), -1)

    def whole(row):
        return np.floor(np.ldexp(np.clip(row.astype(np.float64), 0.0, 512.0), 53)).astype(np.int64)

    for b in range(c["B"]):
        walk = [0]
        while True:
            at = walk[-1]
            w = full = whole(s["target"][b, at].cpu().numpy())
            q = None if s["draft"] is None else s["draft"][b, at].cpu().numpy()
            weight, mass, found = 1 << 53, 1.0, None
            for i in np.flatnonzero(parent[b] == at):
                x = tokens[b, i]
                if q is None:
                    take = weight
                else:
                    f = np.float32(weight / 2.0 ** 53 / mass) if weight > 0 and mass > 0 else np.float32(0)
                    taken = whole(q * f)
                    take = int(taken[x])
                if float(u[b, i]) * float(take) < float(w[x]):
                    found = i
                    break
                if q is None:
                    weight = max(0, weight - int(w[x]))
                    w = w.copy()
                    w[x] = 0
                else:
                    w = np.maximum(w - taken, 0)
                    weight = int(w.sum())
                    mass -= float(q[x]) if c["draft"] == "distinct" else 0.0
            if found is None:
                break
            walk.append(int(found))
        w = full if w.sum() == 0 else w
        total = int(w.sum())
        goal = min(int(float(u_next[b]) * float(total)), total - 1)
        path[b, :len(walk)], length[b] = walk, len(walk)
        said[b, :len(walk)] = [tokens[b, i] for i in walk[1:]] + [min(c["V"] - 1, int(np.searchsorted(np.cumsum(w), goal, side="right")))]
    return {"path": path.astype(np.int32), "path_len": length.astype(np.int32), "out_tokens": said.astype(np.int32), "err": None}


def _exact_keep(s):
    c = s["c"]
    T, path = c["T"], s["path"].tolist()
    k_pool, v_pool, meta = (s[x].double() for x in ("k_pool", "v_pool", "meta"))
    k_old, v_old = k_pool.clone(), v_pool.clone()
    for b, (seq, kept) in enumerate(zip(_lens(c), _kept(c))):
        table = s["table"][b].long()  # [L, Hkv, P]
        for j in range(kept):
            come, go = seq + path[b][j], seq + j
            k_pool[table[..., go // T], go % T] = k_old[table[..., come // T], come % T]
            v_pool[table[..., go // T], :, go % T] = v_old[table[..., come // T], :, come % T]
        for p in range(seq // T, -(-(seq + kept) // T)):
            held = k_pool[table[..., p], :seq + kept - p * T]
            meta[b, :, :, p, 0], meta[b, :, :, p, 1] = held.amin(2), held.amax(2)
    return {"k_pool": k_pool, "v_pool": v_pool, "meta": meta, "err": None}
