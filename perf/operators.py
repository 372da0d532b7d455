"""What the cache-writing and 4-bit cache operators cost, case by case.

Four operators of the paged KV cache: ``kv_append_rope`` (new queries, keys and values rotated by position; keys and
values written to their pages, the pages' key MinMax refreshed), ``kv4_append_rope`` (the same into a cache held in
4 bits), ``kv4_gather`` (tokens of the 4-bit cache back as bf16 rows) and ``sparse_paged_decode_attn_kv4`` (decode
attention over selected pages, or all pages, of the 4-bit cache).

A 4-bit value is an e2m1 code (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) times the e4m3 scale of its 16
channels times one factor for the call's keys or values.  A page holds its keys' codes [T][D/2] (channel 2i in the low
nibble of byte i), their scales [T][D/16], then the values' codes and scales the same way.

``run`` computes them with elementary torch operations in fp32, or, with ``own``, calls the framework.
"""
from __future__ import annotations

import math

import torch

own = False

STEPS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)  # borders between neighbouring e2m1 magnitudes
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------------------------------------
# the cases
def _case(name, kind, **kw):
    c = dict(name=name, kind=kind, B=1, Hq=32, Hkv=8, D=128, T=16, tokens=0, n=1, ragged=False, rope="half", rot=128,
             fused=True, K=0, k_scale=1.0, v_scale=1.0)
    c.update(kw)
    return c


def listed():
    return [
        # one sequence's next token, its rows cut from one projection's output: latency
        _case("append_token_b1", "append", tokens=4095, n=1),
        # the next token of a full decode batch of ragged sequences
        _case("append_token_b32", "append", B=32, tokens=4099, n=1, ragged=True),
        # prompts of odd lengths that start inside a page, other heads, head size and page size, half of the
        # channels rotated in neighbouring pairs, rows head by head
        _case("append_prompts_odd", "append", B=5, Hq=15, Hkv=3, D=64, T=32, tokens=45, n=1031, ragged=True,
              rope="pairs", rot=32, fused=False),
        # a whole 32K prompt, queries included
        _case("append_prompt_32k", "append", tokens=0, n=32768),
        # the next token of eight long sequences into the 4-bit cache, and its rows back
        _case("append4_token_b8", "append4", B=8, tokens=32767, n=1, k_scale=2.0, v_scale=0.5),
        # 8K chunks of two prompts into the 4-bit cache, and the chunk back as bf16 for its own attention
        _case("append4_chunk_8k", "append4", B=2, tokens=8192, n=8192, k_scale=1.5, v_scale=0.37),
        # the cached prefixes of a ragged batch as bf16 rows, other heads and page size
        _case("gather4_prefixes", "gather4", B=8, Hq=40, Hkv=8, T=32, tokens=9001, ragged=True, k_scale=1.25),
        # the smallest decode attention: one KV head, 8 of 64 pages
        _case("attend4_tiny", "attend4", Hq=4, Hkv=1, D=64, tokens=1024, K=8),
        # a decode step's attention at 32K context, batch 8, 128 selected pages a head
        _case("attend4_32k_k128", "attend4", B=8, tokens=32768, K=128, v_scale=0.5),
        # 64K context, five query heads a KV head, pages of 32 tokens, ragged batch
        _case("attend4_64k_gqa5", "attend4", B=16, Hq=40, Hkv=8, T=32, tokens=65536, K=64, ragged=True),
        # every page of one 128K sequence: few rows, one long axis
        _case("attend4_all_128k", "attend4", tokens=131072, k_scale=0.75),
        # every page of a ragged decode batch of up to 16K tokens
        _case("attend4_all_b32", "attend4", B=32, tokens=16381, ragged=True, k_scale=1.5, v_scale=0.25),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    kind = rng.choice(["append", "append", "append4", "gather4", "attend4", "attend4", "attend4"])
    D, T = rng.choice([64, 128, 128]), rng.choice([16, 32])
    Hkv, G = rng.choice([1, 2, 3, 4, 5, 8, 8]), rng.choice([1, 2, 3, 4, 4, 5, 7, 8])
    rope = rng.choice(["half", "half", "pairs", "none"])
    c = dict(kind=kind, Hq=Hkv * G, Hkv=Hkv, D=D, T=T, ragged=rng.random() < 0.6, rope=rope,
             rot=rng.choice(list(range(32, D + 1, 32))) if rope != "none" else 0, fused=rng.random() < 0.5,
             k_scale=rng.choice([1.0, 0.5, 1.3]), v_scale=rng.choice([1.0, 2.0, 0.7]), n=1, K=0)
    if kind in ("append", "append4"):
        c["B"] = _log(rng, 1, 48)
        c["n"] = 1 if rng.random() < 0.4 else _log(rng, 2, max(2, 120000 // (c["B"] * (Hkv + Hkv * G) // 4 + 8)))
        c["tokens"] = _log(rng, 1, 6000)
    elif kind == "gather4":
        c["B"] = _log(rng, 1, 16)
        c["tokens"] = _log(rng, 1, 60000 // c["B"])
    else:
        c["B"] = _log(rng, 1, 64)
        most = min(131072, 3000000 // (c["B"] * Hkv))
        c["tokens"] = _log(rng, 1, most)
        c["K"] = 0 if rng.random() < 0.5 else _log(rng, 1, 300)
    return c


def _cached(c):
    """Tokens of each sequence before the call."""
    n, B = c["tokens"], c["B"]
    if not c["ragged"]:
        return [n] * B
    got = [max(0, n - b * n // (2 * B) - (b * 7) % c["T"]) for b in range(B)]
    if B >= 3 and c["kind"] != "append":
        got[B - 2] = 0  # a slot of the batch with no sequence
    return got


def _added(c):
    n, B = c["n"], c["B"]
    return [n] * B if not c["ragged"] or n == 1 else [max(1, n - b * n // (2 * B) - b) for b in range(B)]


def _picked(c):
    """Selected pages of each sequence (all of them with K = 0)."""
    pages = [-(-s // c["T"]) for s in _cached(c)]
    return [min(c["K"], p) for p in pages] if c["K"] else pages


def work(c):
    B, Hq, Hkv, D, T = c["B"], c["Hq"], c["Hkv"], c["D"], c["T"]
    row4 = D // 2 + D // 16
    if c["kind"] == "gather4":
        rows = sum(_cached(c)) * Hkv
        return {"bytes": rows * 2 * (row4 + 2 * D), "flops": rows * 4 * D}
    if c["kind"] == "attend4":
        # a sequence's partial last page counts whole when all its pages are read, as any other when some are
        toks = sum(_cached(c)) if not c["K"] else sum(p * T for p in _picked(c))
        by = toks * Hkv * 2 * row4 + B * Hq * D * (2 + 4) + sum(_picked(c)) * Hkv * (8 if c["K"] else 4)
        return {"bytes": by, "flops": toks * Hq * D * 4}
    new = sum(_added(c))
    begun = sum(s % T for s in _cached(c)) * Hkv  # keys of a begun page, read again for its MinMax
    pages = sum(-(-(s + a) // T) - s // T for s, a in zip(_cached(c), _added(c))) * Hkv
    by = new * 2 * D * (2 * Hq + 2 * Hkv) + pages * 4 * D + new * c["rot"] * 4
    if c["kind"] == "append":
        by += new * Hkv * 4 * D + begun * 2 * D
    else:
        by += new * Hkv * (4 * row4 + 4 * D) + begun * row4
    return {"bytes": by, "flops": new * (Hq + Hkv) * c["rot"] * 3}


# ------------------------------------------------------------------------------------------------------------------
# the 4-bit format, plainly
def _quantise(x):
    """fp32 [..., D] -> packed codes [..., D/2] and e4m3 scales [..., D/16] (bytes)."""
    g = x.unflatten(-1, (-1, 16))
    six = torch.full((1,), 6.0, device=x.device)  # a tensor: dividing by a number multiplies by its reciprocal
    s = (g.abs().amax(-1) / six).clamp(max=448.0).to(torch.float8_e4m3fn)
    sf = s.float().unsqueeze(-1)
    a = g.abs()
    # a tie goes to the even code: borders 0.25, 1.25, 2.5 and 5 belong to the code below, the others to the one above
    code = ((a > STEPS[0] * sf).to(torch.uint8) + (a >= STEPS[1] * sf) + (a > STEPS[2] * sf) + (a >= STEPS[3] * sf)
            + (a > STEPS[4] * sf) + (a >= STEPS[5] * sf) + (a > STEPS[6] * sf))
    code = torch.where(sf > 0, code + 8 * (g < 0).to(torch.uint8), torch.zeros_like(code)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.view(torch.uint8)


def _inverse(scale):
    """The fp32 reciprocal of a factor."""
    return float(torch.ones(1) / torch.full((1,), scale))


def _values(codes, scales):
    """Packed codes [..., D/2] and scales [..., D/16] -> fp32 [..., D], without the call's factor."""
    level = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=codes.device)
    v = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    v = level[v.int()]
    return (v.unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2)


def _parts(pool, T, D):
    """Views of a [n_phys, bytes] pool: key codes and scales, value codes and scales, each [n_phys, T, ...]."""
    a, b = T * D // 2, T * D // 16
    at = [0, a, a + b, 2 * a + b, 2 * a + 2 * b]
    return [pool[:, at[i]:at[i + 1]].unflatten(1, (T, -1)) for i in range(4)]


# ------------------------------------------------------------------------------------------------------------------
def prepare(c, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    B, Hq, Hkv, D, T = c["B"], c["Hq"], c["Hkv"], c["D"], c["T"]
    cached, added = _cached(c), _added(c) if c["kind"].startswith("append") else [0] * c["B"]
    after = [s + a for s, a in zip(cached, added)]
    P = max(1, -(-max(after) // T))
    n_phys = B * Hkv * P

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    s = dict(c=c, P=P, n_phys=n_phys)
    s["table"] = torch.randperm(n_phys, generator=gen, device=dev).to(torch.int32).view(B, 1, Hkv, P)
    s["err"] = torch.zeros(1, dtype=torch.int32, device=dev)
    # keys have a few channels far larger than the rest
    loud = torch.ones(Hkv, D, device=dev)
    loud.scatter_(1, torch.rand(Hkv, D, generator=gen, device=dev).argsort(1)[:, :4], 8.0)
    if c["kind"] == "append":
        s["k_pool"] = normal(n_phys, T, D).to(torch.bfloat16)
        s["v_pool"] = normal(n_phys, D, T).to(torch.bfloat16)
    else:
        pool = torch.empty(n_phys, T * (D + D // 8), dtype=torch.uint8, device=dev)
        kc, ks, vc, vs = _parts(pool, T, D)
        head = torch.empty(n_phys, dtype=torch.int64, device=dev)
        head[s["table"].view(-1).long()] = torch.arange(Hkv, device=dev).view(1, Hkv, 1).expand(B, Hkv, P).reshape(-1)
        step = max(1, (1 << 25) // (T * D))
        for i in range(0, n_phys, step):
            m = min(step, n_phys - i)
            kc[i:i + m], ks[i:i + m] = _quantise(normal(m, T, D) * loud[head[i:i + m]].unsqueeze(1))
            vc[i:i + m], vs[i:i + m] = _quantise(normal(m, T, D))
        s["pool"] = pool
    s["tok_begin"], s["tok_end"] = ints(cached), ints(after)
    if c["kind"] == "attend4":
        s["q"] = normal(B, Hq, D).to(torch.bfloat16)
        s["out"] = torch.zeros(B, Hq, D, device=dev)
        s["lse"] = torch.zeros(B, Hq, device=dev)
        s["sel"] = s["cnt"] = None
        if c["K"]:
            key = torch.rand(B, Hkv, P, generator=gen, device=dev)
            past = torch.arange(P, device=dev) >= ints([-(-x // T) for x in cached]).view(B, 1, 1)
            at = key.masked_fill(past, 2.0).argsort(-1)[..., :c["K"]]
            at = at.masked_fill(torch.arange(at.shape[-1], device=dev) >= ints(_picked(c)).view(B, 1, 1), P)
            sel = torch.full((B, Hkv, c["K"]), P, dtype=torch.int64, device=dev)
            sel[..., :at.shape[-1]] = at
            sel = sel.sort(-1).values
            s["sel"] = sel.masked_fill(sel == P, 0).to(torch.int32).view(B, 1, Hkv, -1)
            s["cnt"] = ints(_picked(c)).view(B, 1, 1).expand(B, 1, Hkv).contiguous()
        return s
    rows = max(cached) if c["kind"] == "gather4" else c["n"]
    if c["kind"] != "append":
        s["k_out"] = torch.zeros(B, max(1, rows), Hkv, D, dtype=torch.bfloat16, device=dev)
        s["v_out"] = torch.zeros_like(s["k_out"])
    if c["kind"] == "gather4":
        s["tok_begin"], s["tok_end"] = ints([0] * B), ints(cached)
        s["rows"] = _rows([0] * B, cached, dev)
        return s
    # new rows: cut from one projection's output, or each head's rows together
    n = c["n"]
    if c["fused"]:
        x = normal(B, n, Hq + 2 * Hkv, D)
        x[:, :, Hq:Hq + Hkv] *= loud
        x = x.to(torch.bfloat16)
        s["q"], s["k"], s["v"] = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    else:
        s["q"] = normal(B, Hq, n, D).to(torch.bfloat16).transpose(1, 2)
        s["k"] = (normal(B, Hkv, n, D) * loud.unsqueeze(1)).to(torch.bfloat16).transpose(1, 2)
        s["v"] = normal(B, Hkv, n, D).to(torch.bfloat16).transpose(1, 2)
    s["q_out"] = torch.zeros(B, n, Hq, D, dtype=torch.bfloat16, device=dev)
    s["meta"] = torch.zeros(B, 1, Hkv, P, 2, D, dtype=torch.bfloat16, device=dev)
    if c["rot"]:
        i = torch.arange(c["rot"] // 2, dtype=torch.float64, device=dev)
        angle = torch.arange(max(after), dtype=torch.float64, device=dev)[:, None] * 500000.0 ** (-2.0 * i / c["rot"])
        s["angles"] = torch.stack([angle.cos(), angle.sin()], 1).float()
    # which new rows exist and which pages they reach: a program knows its own lengths
    s["rows"] = _rows(cached, after, dev)
    touched = [(b, p) for b in range(B) for p in range(cached[b] // T, -(-after[b] // T))]
    s["pages"] = torch.tensor(touched, dtype=torch.int64, device=dev).T
    s["filled"] = torch.tensor([min(T, after[b] - p * T) for b, p in touched], device=dev)
    return s


def _rows(begin, end, dev):
    """(batch, row, token) of every new row."""
    b = torch.tensor([x for x, (p, q) in enumerate(zip(begin, end)) for _ in range(q - p)], dtype=torch.int64)
    j = torch.tensor([x for p, q in zip(begin, end) for x in range(q - p)], dtype=torch.int64)
    return b.to(dev), j.to(dev), (j + torch.tensor(begin, dtype=torch.int64)[b]).to(dev)


def run(s):
    if own:
        return _run_own(s)
    c = s["c"]
    if c["kind"] == "attend4":
        return _attend(s)
    if c["kind"] == "gather4":
        return _gather(s)
    return _append(s)


def _run_own(s):
    from paged_kv_cache_minmax_gb300 import kvmm

    c = s["c"]
    if "shape" not in s:
        s["shape"] = kvmm.make_shape(c["B"], 1, c["Hq"], c["Hkv"], c["D"], c["T"], s["P"], max(1, c["K"]), s["n_phys"])
        s["turn"] = kvmm.Rope(s["angles"], c["rot"], interleaved=c["rope"] == "pairs") if "angles" in s else None
        s["ws"] = kvmm.alloc_kv4_workspace(s["shape"]) if c["kind"] == "attend4" else None
    shape, scales = s["shape"], dict(k_scale=c["k_scale"], v_scale=c["v_scale"])
    if c["kind"] == "append":
        kvmm.kv_append_rope(shape, 0, s["q"], s["k"], s["v"], s["tok_begin"], s["tok_end"], s["k_pool"], s["v_pool"],
                            s["table"], s["meta"], rope=s["turn"], q_out=s["q_out"], err=s["err"])
        return {n: s[n] for n in ("q_out", "k_pool", "v_pool", "meta", "err")}
    if c["kind"] == "attend4":
        kvmm.sparse_paged_decode_attn_kv4(shape, 0, s["q"], s["pool"], s["table"], s["tok_end"], s["sel"], s["cnt"],
                                          s["out"], s["ws"], lse=s["lse"], err=s["err"], **scales)
        return {n: s[n] for n in ("out", "lse", "err")}
    if c["kind"] == "append4":
        kvmm.kv4_append_rope(shape, 0, s["q"], s["k"], s["v"], s["tok_begin"], s["tok_end"], s["pool"], s["table"],
                             s["meta"], rope=s["turn"], q_out=s["q_out"], err=s["err"], **scales)
    kvmm.kv4_gather(shape, 0, s["pool"], s["table"], s["tok_begin"], s["tok_end"], s["k_out"], s["v_out"],
                    err=s["err"], **scales)
    return {n: s[n] for n in ("q_out", "k_out", "v_out", "meta", "err") if n in s}


# ------------------------------------------------------------------------------------------------------------------
# the plain forms
def _turned(s, x):
    """bf16 rows [N, H, D] of the new tokens, rotated in fp32: every product and their sum rounded."""
    c, x = s["c"], x.float()
    if not c["rot"]:
        return x
    cos, sin = (s["angles"][s["rows"][2], i].unsqueeze(1) for i in (0, 1))
    h, r = c["rot"] // 2, c["rot"]
    if c["rope"] == "half":
        a, b = x[..., :h], x[..., h:r]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., r:]], -1)
    a, b = x[..., 0:r:2], x[..., 1:r:2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), x[..., r:]], -1)


def _append(s):
    c, (b, j, t) = s["c"], s["rows"]
    T, D = c["T"], c["D"]
    s["q_out"][b, j] = _turned(s, s["q"][b, j]).to(torch.bfloat16)
    k, v = _turned(s, s["k"][b, j]), s["v"][b, j].float()
    phys = s["table"][b, 0, :, t // T].long()  # [N, Hkv]
    slot = (t % T).unsqueeze(1)
    pb, pp = s["pages"]
    where = s["table"][pb, 0, :, pp].long()
    if c["kind"] == "append":
        s["k_pool"][phys, slot] = k.to(torch.bfloat16)
        s["v_pool"][phys, :, slot] = v.to(torch.bfloat16)
        keys = s["k_pool"][where].float()  # [pages, Hkv, T, D]
    else:
        kc, ks, vc, vs = _parts(s["pool"], T, D)
        kc[phys, slot], ks[phys, slot] = _quantise(k * _inverse(c["k_scale"]))
        vc[phys, slot], vs[phys, slot] = _quantise(v * _inverse(c["v_scale"]))
        keys = _values(kc[where], ks[where])
    past = (torch.arange(T, device=k.device) >= s["filled"].unsqueeze(1)).view(-1, 1, T, 1)
    s["meta"][pb, 0, :, pp, 0] = keys.masked_fill(past, math.inf).amin(2).to(torch.bfloat16)
    s["meta"][pb, 0, :, pp, 1] = keys.masked_fill(past, -math.inf).amax(2).to(torch.bfloat16)
    if c["kind"] == "append":
        return {n: s[n] for n in ("q_out", "k_pool", "v_pool", "meta", "err")}
    return {**{n: s[n] for n in ("q_out", "meta")}, **_gather(s)}


def _gather(s):
    c, (b, j, t) = s["c"], s["rows"]
    kc, ks, vc, vs = _parts(s["pool"], c["T"], c["D"])
    phys, slot = s["table"][b, 0, :, t // c["T"]].long(), (t % c["T"]).unsqueeze(1)
    s["k_out"][b, j] = (_values(kc[phys, slot], ks[phys, slot]) * c["k_scale"]).to(torch.bfloat16)
    s["v_out"][b, j] = (_values(vc[phys, slot], vs[phys, slot]) * c["v_scale"]).to(torch.bfloat16)
    return {n: s[n] for n in ("k_out", "v_out", "err")}


def _attend(s):
    c = s["c"]
    B, Hq, Hkv, D, T, P = c["B"], c["Hq"], c["Hkv"], c["D"], c["T"], s["P"]
    table, seq = s["table"][:, 0].long(), s["tok_end"].view(B, 1, 1, 1)
    if c["K"]:
        page = s["sel"][:, 0].long()
        here = torch.arange(page.shape[-1], device=page.device) < s["cnt"][:, 0].unsqueeze(-1)
    else:
        page = torch.arange(P, device=table.device).expand(B, Hkv, P)
        here = page >= 0
    phys = table.gather(2, page)
    kc, ks, vc, vs = _parts(s["pool"], T, D)
    k = _values(kc[phys], ks[phys]).flatten(2, 3)  # [B, Hkv, tokens, D]
    tok = page.unsqueeze(-1) * T + torch.arange(T, device=page.device)
    live = ((tok < seq) & here.unsqueeze(-1)).flatten(2).unsqueeze(2)  # [B, Hkv, 1, tokens]
    q = s["q"].float().view(B, Hkv, Hq // Hkv, D)
    z = (q @ k.transpose(2, 3)) * (c["k_scale"] / math.sqrt(D))
    del k
    z = z.masked_fill(~live, -math.inf)
    m = z.amax(-1, keepdim=True).clamp(min=-3e38)
    e = (z - m).exp()
    l = e.sum(-1, keepdim=True)
    v = _values(vc[phys], vs[phys]).flatten(2, 3)
    out = (e @ v) * (c["v_scale"] / l.clamp(min=1e-38))
    lse = torch.where(l > 0, m + l.log(), torch.full_like(l, -math.inf))
    return {"out": out.view(B, Hq, D), "lse": lse.view(B, Hq), "err": s["err"]}


# ------------------------------------------------------------------------------------------------------------------
# the same in 64 bits, from the definitions
def exact(c, seed):
    s = prepare(c, seed)
    return {"attend4": _exact_attend, "gather4": _exact_gather}.get(c["kind"], _exact_append)(s)


def _f64_two_to(e):
    """Powers of two, exact (a library's pow need not be)."""
    return torch.tensor([2.0 ** i for i in range(-16, 17)], dtype=torch.float64, device=e.device)[(e + 16).long()]


def _f64_code(n):
    """e2m1 nibbles (uint8) -> float64."""
    n = n.double()
    sign = 1 - 2 * torch.floor(n / 8)
    low = n % 8
    e, m = torch.floor(low / 2), low % 2
    return sign * torch.where(e == 0, m * 0.5, (1 + m / 2) * _f64_two_to(e - 1))


def _f64_scale(n):
    """e4m3 bytes (sign bit clear) -> float64."""
    n = n.double()
    e, m = torch.floor(n / 8), n % 8
    return torch.where(e == 0, m / 512, (1 + m / 8) * _f64_two_to(e - 7))


def _f64_rows(pool, T, D, values):
    """Key (or value) rows [pages, T, D] of whole pages, in stored units."""
    a, b = T * D // 2, T * D // 16
    o = (a + b) if values else 0
    codes, scales = pool[:, o:o + a].reshape(-1, T, D // 2), pool[:, o + a:o + a + b].reshape(-1, T, D // 16)
    x = torch.empty(codes.shape[0], T, D, dtype=torch.float64, device=pool.device)
    x[..., 0::2], x[..., 1::2] = _f64_code(codes % 16), _f64_code(codes // 16)
    return x * _f64_scale(scales).repeat_interleave(16, -1)


def _exact_attend(s):
    c = s["c"]
    B, Hq, Hkv, D, T = c["B"], c["Hq"], c["Hkv"], c["D"], c["T"]
    G = Hq // Hkv
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    lens, picked = _cached(c), _picked(c)
    for b in range(B):
        for h in range(Hkv):
            if not lens[b]:
                continue
            page = s["sel"][b, 0, h, :picked[b]].long() if c["K"] else torch.arange(picked[b], device="cuda")
            pool = s["pool"][s["table"][b, 0, h, page].long()]
            tok = (page[:, None] * T + torch.arange(T, device="cuda")).reshape(-1)
            keep = tok < lens[b]
            k = _f64_rows(pool, T, D, False).reshape(-1, D)[keep] * c["k_scale"]
            v = _f64_rows(pool, T, D, True).reshape(-1, D)[keep] * c["v_scale"]
            z = s["q"][b, h * G:(h + 1) * G].double() @ k.T / math.sqrt(D)
            lse[b, h * G:(h + 1) * G] = torch.logsumexp(z, -1)
            out[b, h * G:(h + 1) * G] = torch.softmax(z, -1) @ v
    return {"out": out, "lse": lse, "err": None}


def _exact_gather(s):
    c = s["c"]
    T, D = c["T"], c["D"]
    k, v = (s[n].double() for n in ("k_out", "v_out"))
    for b, n in enumerate(_cached(c)):
        for h in range(c["Hkv"]):
            pool = s["pool"][s["table"][b, 0, h, :-(-n // T)].long()]
            k[b, :n, h] = _f64_rows(pool, T, D, False).reshape(-1, D)[:n] * c["k_scale"]
            v[b, :n, h] = _f64_rows(pool, T, D, True).reshape(-1, D)[:n] * c["v_scale"]
    return {"k_out": k, "v_out": v, "err": None}


def _f64_turn(s, x, begin, to32=False):
    """Rows [n, H, D] of one sequence from token `begin` on, rotated.  `to32`: as the 4-bit cache defines it, with
    every product and their sum rounded to fp32 (each is exact, or all but, in 64 bits first)."""
    c, x = s["c"], x.double()
    if not c["rot"]:
        return x
    near = (lambda y: y.float().double()) if to32 else (lambda y: y)
    n, r = x.shape[0], c["rot"]
    first = torch.arange(0, r // 2, device=x.device)
    i, k = (first, first + r // 2) if c["rope"] == "half" else (2 * first, 2 * first + 1)
    cos, sin = s["angles"][begin:begin + n].double().unbind(1)
    cos, sin = cos[:, None], sin[:, None]
    y = x.clone()
    y[..., i] = near(near(x[..., i] * cos) - near(x[..., k] * sin))
    y[..., k] = near(near(x[..., k] * cos) + near(x[..., i] * sin))
    return y


def _f64_four(x):
    """The values float64 [..., D] is held as in 4 bits: the nearest e4m3 to a sixth of the largest of 16 channels,
    times the nearest e2m1 to each quotient; ties to the even code."""
    g = x.reshape(*x.shape[:-1], -1, 16)
    s = (g.abs().amax(-1) / torch.full((1,), 6.0, dtype=torch.float64, device=g.device)).float().double().clamp(max=448)
    unit = _f64_two_to(torch.frexp(s.clamp(min=2.0 ** -6)).exponent - 4)  # the step of e4m3 there
    s = torch.round(s / unit) * unit  # torch.round: ties to even
    q = g.abs() / s.clamp(min=1e-30).unsqueeze(-1)
    unit = 0.5 + 0.5 * (q >= 2) + (q >= 4)  # the step of e2m1
    q = (torch.round(q / unit) * unit).clamp(max=6.0)
    return (q * g.sign() * s.unsqueeze(-1)).reshape(x.shape)


def _exact_append(s):
    c = s["c"]
    T, D, Hkv, four = c["T"], c["D"], c["Hkv"], c["kind"] == "append4"
    if c["n"] * c["B"] * c["Hq"] * D > 1 << 28:
        return None
    q, meta = s["q_out"].double(), s["meta"].double()
    if four:
        k_out, v_out = s["k_out"].double(), s["v_out"].double()
    else:
        k_pool, v_pool = s["k_pool"].double(), s["v_pool"].double()
    ik, iv = (float(torch.tensor(1.0 / x, dtype=torch.float32)) for x in (c["k_scale"], c["v_scale"]))
    for b, (begin, n) in enumerate(zip(_cached(c), _added(c))):
        q[b, :n] = _f64_turn(s, s["q"][b, :n], begin)
        k, v = _f64_turn(s, s["k"][b, :n], begin, four), s["v"][b, :n].double()
        if four:
            k, v = _f64_four((k * ik).float().double()), _f64_four((v * iv).float().double())
            k_out[b, :n], v_out[b, :n] = k * c["k_scale"], v * c["v_scale"]
        first, end = begin // T, -(-(begin + n) // T)
        for h in range(Hkv):
            phys = s["table"][b, 0, h, first:end].long()
            rows = _f64_rows(s["pool"][phys], T, D, False) if four else k_pool[phys]
            rows = rows.reshape(-1, D)
            o = begin - first * T
            rows[o:o + n] = k[:, h]
            if not four:
                k_pool[phys] = rows.reshape(-1, T, D)
                cols = v_pool[phys].transpose(1, 2).reshape(-1, D)
                cols[o:o + n] = v[:, h]
                v_pool[phys] = cols.reshape(-1, T, D).transpose(1, 2)
            pad = torch.full((rows.shape[0] - o - n, D), math.nan, dtype=torch.float64, device=rows.device)
            whole = torch.cat([rows[:o + n], pad]).reshape(-1, T, D)
            meta[b, 0, h, first:end, 0] = whole.nan_to_num(nan=math.inf).amin(1)
            meta[b, 0, h, first:end, 1] = whole.nan_to_num(nan=-math.inf).amax(1)
    if four:
        return {"q_out": q, "k_out": k_out, "v_out": v_out, "meta": meta, "err": None}
    return {"q_out": q, "k_pool": k_pool, "v_pool": v_pool, "meta": meta, "err": None}
