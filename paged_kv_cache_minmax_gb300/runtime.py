"""Decode-step driver over the four C-ABI calls.

:class:`DecodeState` owns the device buffers one long-context decode needs
beside the caller's pools (MinMax metadata, selections, the committed previous
selections, promotion lists, outputs, workspace, error word) and issues, per
layer and step, the calls in the method's order:

  1. ``kv_minmax_update``          append the new token, refresh its page's MinMax
  2. ``page_score_topk``           rescored units only (stable heads keep their top-K)
  3. ``topk_promotion_diff``       promoted = cur \\ prev (commit cur as prev)
  4. ``sparse_paged_decode_attn``  attention over the selected pages

or, with steps 2 and 4 in one launch, ``page_score_topk_attn`` then the diff.
From a projection's unrotated rows, step 1 is ``kv_append_rope``.
:class:`TreeDecode` takes steps of several drafted tokens a sequence (speculative decoding) over such a state.
:class:`Kv4DecodeState` is the same over a cache held in 4 bits.

(FlexiCache, "Core method", sections 1-3.)  Everything runs on one CUDA
stream; nothing here synchronises.
"""
from __future__ import annotations

import torch

from . import kvmm


class _StepState:
    """The buffers and calls that do not depend on how the pages hold their keys and values."""

    def __init__(self, B, L, Hq, Hkv, D, T, Pmax, K, n_phys, block_table, seq_len, num_splits, group_reduce, device):
        self.shape = kvmm.make_shape(B, L, Hq, Hkv, D, T, Pmax, K, n_phys)
        self.K = K
        self.num_splits = num_splits
        self.group_reduce = group_reduce
        self.block_table, self.seq_len = block_table, seq_len
        i32 = dict(dtype=torch.int32, device=device)
        self.meta = torch.zeros(B, L, Hkv, Pmax, 2, D, dtype=torch.bfloat16, device=device)
        self.sel_idx = torch.zeros(B, L, Hkv, K, **i32)
        self.sel_cnt = torch.zeros(B, L, Hkv, **i32)
        self.prev_idx = torch.zeros(B, L, Hkv, K, **i32)
        self.prev_cnt = torch.zeros(B, L, Hkv, **i32)
        self.promoted = torch.zeros(B, L, Hkv, K, **i32)
        self.promoted_cnt = torch.zeros(B, L, Hkv, **i32)
        self.evicted = torch.zeros(B, L, Hkv, K, **i32)
        self.evicted_cnt = torch.zeros(B, L, Hkv, **i32)
        self.total_promoted = torch.zeros(1, **i32)
        self.out = torch.zeros(L, B, Hq, D, dtype=torch.float32, device=device)
        self.lse = torch.zeros(L, B, Hq, dtype=torch.float32, device=device)
        self.q_turned = torch.zeros(L, B, Hq, D, dtype=torch.bfloat16, device=device)
        self.err = torch.zeros(1, **i32)
        self.tok_begin = torch.zeros(B, **i32)
        self.tok_end = torch.zeros(B, **i32)
        self.workspace = kvmm.alloc_workspace(self.shape, num_splits, device=device)

    def _step_rows(self, q, new_k, new_v):
        """One token's rows [B, 1, H, D] from [B, H, D] or [B, 1, H, D] views; the token is at seq_len - 1 (a slot of
        the batch with no sequence appends nothing)."""
        torch.sub(self.seq_len, 1, out=self.tok_begin).clamp_(min=0)
        return [t if t.dim() == 4 else t.unsqueeze(1) for t in (q, new_k, new_v)]

    def select(self, layer, q, rescore_mask=None, scores_out=None) -> None:
        kvmm.page_score_topk(self.shape, layer, q, self.meta, self.seq_len, rescore_mask, self.K, self.sel_idx,
                             self.sel_cnt, self.workspace, self.err, scores_out=scores_out,
                             group_reduce=self.group_reduce)

    def diff(self, layer, rescore_mask=None, commit=True) -> None:
        kvmm.topk_promotion_diff(self.shape, layer, rescore_mask, self.prev_idx, self.prev_cnt, self.sel_idx,
                                 self.sel_cnt, self.promoted, self.promoted_cnt, self.evicted, self.evicted_cnt,
                                 self.total_promoted, commit=commit, err=self.err)

    def read_err(self) -> int:
        return int(self.err.item())


class DecodeState(_StepState):
    def __init__(self, B, L, Hq, Hkv, D, T, Pmax, K, k_pool, v_pool, block_table, seq_len, num_splits=0,
                 group_reduce=0, device="cuda"):
        super().__init__(B, L, Hq, Hkv, D, T, Pmax, K, k_pool.shape[0], block_table, seq_len, num_splits, group_reduce,
                         device)
        self.k_pool, self.v_pool = k_pool, v_pool

    @classmethod
    def for_workload(cls, wl, K=None, **kw):
        c = wl.cfg
        return cls(c.B, c.L_alloc, c.Hq, c.Hkv, c.D, c.T, c.Pmax, K or c.K, wl.k_pool, wl.v_pool,
                   wl.block_table, wl.seq_len, **kw)

    # ------------------------------------------------------------------ #
    def build_metadata(self, layers=None) -> None:
        """Rebuild the MinMax of every page below seq_len (after a prefill)."""
        s = self.shape
        self.tok_begin.zero_()
        for l in (range(s.L) if layers is None else layers):
            kvmm.kv_minmax_update(s, l, None, None, 0, self.tok_begin, self.seq_len, self.k_pool, self.v_pool,
                                  self.block_table, self.meta, self.err)

    def append(self, layer, new_k, new_v) -> None:
        """Write one new token per batch entry at position seq_len-1 of ``layer``.

        new_k / new_v: ``[B, Hkv, 1, D]`` bf16; ``seq_len`` already counts the token.
        """
        torch.sub(self.seq_len, 1, out=self.tok_begin)
        kvmm.kv_minmax_update(self.shape, layer, new_k, new_v, 1, self.tok_begin, self.seq_len, self.k_pool,
                              self.v_pool, self.block_table, self.meta, self.err)

    def attend(self, layer, q, sm_scale=0.0) -> None:
        kvmm.sparse_paged_decode_attn(self.shape, layer, q, self.k_pool, self.v_pool, self.block_table,
                                      self.seq_len, self.sel_idx, self.sel_cnt, self.out[layer], self.workspace,
                                      lse=self.lse[layer], err=self.err, sm_scale=sm_scale,
                                      num_splits=self.num_splits)

    def select_attend(self, layer, q, rescore_mask=None, scores_out=None, sm_scale=0.0) -> None:
        """select + attend in one launch (page_score_topk_attn)."""
        kvmm.page_score_topk_attn(self.shape, layer, q, self.meta, self.k_pool, self.v_pool, self.block_table,
                                  self.seq_len, rescore_mask, self.K, self.sel_idx, self.sel_cnt, self.out[layer],
                                  self.workspace, lse=self.lse[layer], err=self.err, scores_out=scores_out,
                                  group_reduce=self.group_reduce, sm_scale=sm_scale)

    def decode(self, layer, q, new_k=None, new_v=None, rescore_mask=None, scores_out=None, sm_scale=0.0) -> None:
        """decode_layer: append (new_k/new_v [B, Hkv, 1, D] at seq_len - 1), score, select, attend."""
        if new_k is not None:
            torch.sub(self.seq_len, 1, out=self.tok_begin)
        kvmm.decode_layer(self.shape, layer, q, new_k, new_v, 1, self.tok_begin, self.seq_len, self.k_pool,
                          self.v_pool, self.block_table, self.meta, self.seq_len, rescore_mask, self.K, self.sel_idx,
                          self.sel_cnt, self.out[layer], lse=self.lse[layer], err=self.err, scores_out=scores_out,
                          group_reduce=self.group_reduce, sm_scale=sm_scale, workspace=self.workspace)

    def layer_step(self, layer, q, new_k=None, new_v=None, rescore_mask=None, fused=True) -> None:
        """One layer of one decode step: append, select + attend, diff."""
        if new_k is not None:
            self.append(layer, new_k, new_v)
        if fused:
            self.select_attend(layer, q, rescore_mask)
            self.diff(layer, rescore_mask)
        else:
            self.select(layer, q, rescore_mask)
            self.diff(layer, rescore_mask)
            self.attend(layer, q)

    def append_rope(self, layer, q, new_k, new_v, rope=None) -> None:
        """One new token per batch entry at position seq_len - 1, its query and key rotated (``kvmm.Rope``):
        q [B, Hq, D], new_k and new_v [B, Hkv, D] bf16 views; the turned query goes to ``q_turned[layer]``."""
        q, new_k, new_v = self._step_rows(q, new_k, new_v)
        kvmm.kv_append_rope(self.shape, layer, q, new_k, new_v, self.tok_begin, self.seq_len, self.k_pool, self.v_pool,
                            self.block_table, self.meta, rope=rope, q_out=self.q_turned[layer], err=self.err)

    def layer_step_rope(self, layer, q, new_k, new_v, rope=None, rescore_mask=None) -> None:
        """One layer of one decode step from a projection's rows: rotate and append, select + attend, diff."""
        self.append_rope(layer, q, new_k, new_v, rope)
        self.select_attend(layer, self.q_turned[layer], rescore_mask)
        self.diff(layer, rescore_mask)


class TreeDecode:
    """Speculative decoding over a :class:`DecodeState`: each step hands every sequence a tree of up to ``n_max`` nodes,
    node 0 the token sampled last and the others drafted.  Between steps ``state.seq_len`` counts the settled tokens,
    which do not include node 0.  A step is ``begin``, ``layer_step`` for every layer, ``verify`` with the target's
    probabilities, ``keep``; ``out_tokens[:, path_len - 1]`` are the next roots.

    ``parent`` [B, n_max] int32 gives the trees (see ``kvmm.draft_verify``); they may be replaced with ``set_trees``, which
    steps that are captured in a graph follow."""

    def __init__(self, state: DecodeState, parent: torch.Tensor, rope: kvmm.Rope | None = None):
        s = state.shape
        if parent.dim() != 2 or parent.shape[0] != s.B:
            raise ValueError(f"parent must be [{s.B}, n], got {list(parent.shape)}")
        n = parent.shape[1]
        dev = state.seq_len.device
        i32 = dict(dtype=torch.int32, device=dev)
        self.state, self.n_max = state, n
        self.q_turned = torch.zeros(s.L, s.B, n, s.Hq, s.D, dtype=torch.bfloat16, device=dev)
        self.root_q = torch.zeros(s.B, s.Hq, s.D, dtype=torch.bfloat16, device=dev)
        self.out = torch.zeros(s.L, s.B, n, s.Hq, s.D, dtype=torch.bfloat16, device=dev)
        self.lse = torch.zeros(s.L, s.B, n, s.Hq, dtype=torch.float32, device=dev)
        self.path, self.out_tokens = torch.zeros(s.B, n, **i32), torch.zeros(s.B, n, **i32)
        self.path_len = torch.zeros(s.B, **i32)
        self.n_nodes, self.tok_end = torch.full((s.B,), n, **i32), torch.zeros(s.B, **i32)
        self.positions = torch.zeros(s.B, n, **i32)
        self.parent, self.depth = torch.zeros(s.B, n, **i32), torch.zeros(s.B, n, **i32)
        self.mask = torch.zeros(s.B, n, dtype=torch.int64, device=dev)
        self.workspace = kvmm.alloc_tree_workspace(s, n, device=dev)
        self.rope = None if rope is None else kvmm.Rope(rope.table, rope.dim, bool(rope.c.interleaved), self.positions)
        self.set_trees(parent)

    def set_trees(self, parent: torch.Tensor) -> None:
        """The trees of the following steps, ``parent`` [B, n_max] copied.  What a captured step reads stays in its place:
        its replays take the trees set last."""
        if parent.shape != self.parent.shape:
            raise ValueError(f"parent must be {list(self.parent.shape)}, got {list(parent.shape)}")
        self.parent.copy_(parent)
        self.mask.copy_(kvmm.tree_masks(self.parent))
        j = torch.arange(self.n_max, device=self.mask.device)
        self.depth.copy_(((self.mask.unsqueeze(-1) >> j) & 1).sum(-1).sub_(1))

    def begin(self, n_nodes: torch.Tensor | None = None) -> None:
        """Start a step; ``n_nodes`` [B] int32: the nodes of each tree that exist (default: all)."""
        if n_nodes is None:
            self.n_nodes.fill_(self.n_max)
        else:
            self.n_nodes.copy_(n_nodes)
        torch.add(self.state.seq_len, self.n_nodes, out=self.tok_end)
        torch.add(self.state.seq_len.unsqueeze(1), self.depth, out=self.positions)

    def layer_step(self, layer, q, new_k, new_v, rescore_mask=None, every_page=False, sm_scale=0.0) -> None:
        """One layer: the nodes' rows q [B, n_max, Hq, D], new_k and new_v [B, n_max, Hkv, D] (bf16 views) rotated and
        appended, pages selected by the roots' queries, every node attended."""
        st, qt = self.state, self.q_turned[layer]
        kvmm.kv_append_rope(st.shape, layer, q, new_k, new_v, st.seq_len, self.tok_end, st.k_pool, st.v_pool,
                            st.block_table, None, rope=self.rope, q_out=qt, err=st.err)
        if not every_page:
            self.root_q.copy_(qt[:, 0])
            st.select(layer, self.root_q, rescore_mask)
            st.diff(layer, rescore_mask)
        kvmm.sparse_paged_tree_attn(st.shape, layer, qt, st.k_pool, st.v_pool, st.block_table, st.seq_len,
                                    self.out[layer], self.workspace, n_nodes=self.n_nodes, tree_mask=self.mask,
                                    sel_idx=None if every_page else st.sel_idx,
                                    sel_cnt=None if every_page else st.sel_cnt, lse=self.lse[layer], err=st.err,
                                    sm_scale=sm_scale)

    def verify(self, target_probs, tokens, u_accept, u_next, draft_probs=None, distinct=False) -> None:
        """Accept a path and draw the token behind it (``path``, ``path_len``, ``out_tokens``)."""
        kvmm.draft_verify(target_probs, tokens, self.parent, u_accept, u_next, self.path, self.path_len,
                          self.out_tokens, draft_probs=draft_probs, n_nodes=self.n_nodes, distinct=distinct,
                          err=self.state.err)

    def keep(self) -> None:
        """Settle the accepted nodes in every layer (those with a place in the table: the others are told)."""
        st = self.state
        kvmm.kv_keep_path(st.shape, -1, self.path, self.path_len, st.seq_len, st.k_pool, st.v_pool, st.block_table,
                          st.meta, err=st.err)
        st.seq_len.add_(self.path_len).clamp_(max=st.shape.Pmax * st.shape.T)


class Kv4DecodeState(_StepState):
    """DecodeState over the 4-bit cache: ``kv4_pool`` [n_phys, page bytes] (``kvmm.alloc_kv4_pool``), one factor for
    its keys and one for its values.  Prompts are appended with :meth:`append_prompt`, which also keeps the MinMax."""

    def __init__(self, B, L, Hq, Hkv, D, T, Pmax, K, kv4_pool, block_table, seq_len, k_scale=1.0, v_scale=1.0,
                 group_reduce=0, device="cuda"):
        super().__init__(B, L, Hq, Hkv, D, T, Pmax, K, kv4_pool.shape[0], block_table, seq_len, 0, group_reduce, device)
        self.kv4_pool, self.k_scale, self.v_scale = kv4_pool, k_scale, v_scale
        self.kv4_workspace = kvmm.alloc_kv4_workspace(self.shape, device=device)

    def append_prompt(self, layer, new_k, new_v, tok_begin, tok_end, rope=None, q=None, q_out=None) -> None:
        """Tokens [tok_begin, tok_end) of every sequence from rows [B, n, H, D]."""
        kvmm.kv4_append_rope(self.shape, layer, q, new_k, new_v, tok_begin, tok_end, self.kv4_pool, self.block_table,
                             self.meta, rope=rope, q_out=q_out, k_scale=self.k_scale, v_scale=self.v_scale,
                             err=self.err)

    def gather(self, layer, k_out, v_out, tok_begin=None, tok_end=None) -> None:
        """Tokens [tok_begin, tok_end) (default: the whole sequences) as bf16 rows [B, n_rows, Hkv, D]."""
        kvmm.kv4_gather(self.shape, layer, self.kv4_pool, self.block_table, tok_begin,
                        self.seq_len if tok_end is None else tok_end, k_out, v_out, k_scale=self.k_scale,
                        v_scale=self.v_scale, err=self.err)

    def append_rope(self, layer, q, new_k, new_v, rope=None) -> None:
        """As DecodeState.append_rope."""
        q, new_k, new_v = self._step_rows(q, new_k, new_v)
        self.append_prompt(layer, new_k, new_v, self.tok_begin, self.seq_len, rope, q, self.q_turned[layer])

    def attend(self, layer, q, sm_scale=0.0, every_page=False) -> None:
        """Attention over the kept selections, or over every page."""
        kvmm.sparse_paged_decode_attn_kv4(self.shape, layer, q, self.kv4_pool, self.block_table, self.seq_len,
                                          None if every_page else self.sel_idx, None if every_page else self.sel_cnt,
                                          self.out[layer], self.kv4_workspace, lse=self.lse[layer], err=self.err,
                                          k_scale=self.k_scale, v_scale=self.v_scale, sm_scale=sm_scale)

    def layer_step_rope(self, layer, q, new_k, new_v, rope=None, rescore_mask=None) -> None:
        """One layer of one decode step: rotate and append, select, diff, attend."""
        self.append_rope(layer, q, new_k, new_v, rope)
        self.select(layer, self.q_turned[layer], rescore_mask)
        self.diff(layer, rescore_mask)
        self.attend(layer, self.q_turned[layer])


class StabilityProfiler:
    """Offline profiling of head stability: a ring of the last W steps' selections of every (batch, layer,
    KV head) and the Random-Corrected Overlap classification (FlexiCache, "Core insight: attention heads
    differ in temporal stability").  ``record(state)`` stores one decode step of every layer; ``classify``
    returns (rco per unit [B, L, Hkv], stability [L, Hkv], unstable mask [L, Hkv])."""

    def __init__(self, shape, W: int, device="cuda"):
        s = shape
        i32 = dict(dtype=torch.int32, device=device)
        self.shape, self.W = s, W
        self.hist_idx = torch.zeros(W, s.B, s.L, s.Hkv, s.Kmax, **i32)
        self.hist_cnt = torch.zeros(W, s.B, s.L, s.Hkv, **i32)
        self.hist_pages = torch.zeros(W, s.B, **i32)
        self.rco_unit = torch.zeros(s.B, s.L, s.Hkv, dtype=torch.float32, device=device)
        self.stability = torch.zeros(s.L, s.Hkv, dtype=torch.float32, device=device)
        self.unstable = torch.zeros(s.L, s.Hkv, dtype=torch.uint8, device=device)
        self.err = torch.zeros(1, **i32)
        self.steps = 0

    def record(self, state, layers=None) -> None:
        """Store this step's selections of ``layers`` (default: all) in slot steps mod W, then advance."""
        slot = self.steps % self.W
        for l in [-1] if layers is None else layers:  # -1: every layer in one launch
            kvmm.topk_history_record(self.shape, l, state.sel_idx, state.sel_cnt, state.seq_len, slot,
                                     self.hist_idx, self.hist_cnt, self.hist_pages, err=self.err)
        self.steps += 1

    def classify(self, lag: int = 1, unstable_frac: float = 0.25, n: int | None = None):
        n = min(self.steps, self.W) if n is None else n
        kvmm.topk_stability_rco(self.shape, self.hist_idx, self.hist_cnt, self.hist_pages, n,
                                (self.steps - 1) % self.W, lag, self.rco_unit, self.stability, self.unstable,
                                unstable_frac, err=self.err)
        return self.rco_unit, self.stability, self.unstable
