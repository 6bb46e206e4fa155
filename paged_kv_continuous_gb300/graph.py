"""A whole decode step over L layers captured as one CUDA graph.

koas-w, "errors and solutions", section "CUDA Graph": the engine allocates
fixed-shape static buffers once (input ids, slot_mapping, position ids,
block_table, context_lens), updates their values in place every step, and
replays one captured graph per step, so the step's hundreds of launches are
submitted at once.

``DecodeStepGraph`` captures, for every layer, the two library calls of a
decode step -- ``pa_rope_store_kv`` (or ``pa_store_kv`` when no rotary
tables are given) and then ``pa_decode`` -- both launched with
``PA_LAUNCH_PDL``, so each kernel's start-up overlaps the tail of the one
before.  With ``fused=True`` a layer is one call, ``pa_store_decode`` (or
``pa_rope_store_decode`` with rotary tables, which leaves q as it is), which
also requests its first K/V pages early (``PA_LAUNCH_EARLY_KV``) whenever
the call before it is another layer's, on other pools.  This module only records calls into the graph; every step of
the computation runs in the library's kernels.

Static state (fixed at capture): the batch size, the block-table width, the
per-layer tensors (their addresses are baked into the graph), the split
count and the decode workspace.  Values the caller changes between replays,
in place: the index buffers, through :meth:`DecodeStepGraph.update`, and
each layer's new q / k / v rows (written into the layer tensors given at
construction; with rotary tables and two calls per layer q is rotated in
place, so it must be refilled before every replay; the fused call leaves q
as it is).  The decode kernel partitions its work from
``context_lens`` on the device, so a replay follows new lengths without a
new capture.

``TreeStepGraph`` is a speculative step in two graphs: the stores and the
``pa_decode_tree`` calls of all layers, and ``pa_verify_tree`` with
``pa_commit_tree``.
"""
from __future__ import annotations

import torch

from . import ops


class DecodeStepGraph:
    """One decode step of ``len(layers)`` layers as a single CUDA graph.

    layers: list of dicts with bf16 CUDA tensors ``q`` [B, Hq, D] (contiguous),
    ``k``, ``v`` [B, Hkv, D] (the step's new token rows), ``k_cache``,
    ``v_cache`` (the layer's pools) and ``out`` [B, Hq, D].
    block_tables int32 [B, max_blocks], context_lens int32 [B], slot_mapping
    int32 [B]: the initial values of the static index buffers (copied).
    positions int32 [B] with cos_table / sin_table float32 [max_position,
    D/2]: rotary embedding of q and k fused into the store.
    fused: one pa_store_decode (pa_rope_store_decode with rotary tables)
    per layer instead of a store and a decode; slot_mapping[b] must then be
    the slot of position context_lens[b] - 1 under the block table.
    """

    def __init__(self, layers, block_tables, context_lens, slot_mapping, scale,
                 positions=None, cos_table=None, sin_table=None, num_splits=0, device=None,
                 fused=False):
        if not layers:
            raise ops.PagedAttentionError("DecodeStepGraph needs at least one layer")
        if (cos_table is None) != (positions is None) or (cos_table is None) != (sin_table is None):
            raise ops.PagedAttentionError("positions, cos_table and sin_table go together")
        self.fused = bool(fused)
        dev = layers[0]["q"].device if device is None else torch.device(device)
        self.layers = layers
        self.scale = float(scale)
        self.rope = cos_table is not None
        # static index buffers: one copy, shared by every layer
        self.block_tables = block_tables.to(dev, torch.int32).clone()
        self.context_lens = context_lens.to(dev, torch.int32).clone()
        self.slot_mapping = slot_mapping.to(dev, torch.int32).clone()
        self.positions = positions.to(dev, torch.int32).clone() if self.rope else None
        self.cos_table = cos_table.to(dev, torch.float32).contiguous() if self.rope else None
        self.sin_table = sin_table.to(dev, torch.float32).contiguous() if self.rope else None
        B, Hq, D = layers[0]["q"].shape
        Hkv = layers[0]["k"].shape[1]
        idx = dev.index if dev.index is not None else torch.cuda.current_device()
        self.num_splits = num_splits or ops.default_splits(Hq, Hkv, idx)
        self.workspace = ops.decode_workspace(Hq, Hkv, self.num_splits, D, dev)
        self.error_word = torch.zeros(1, dtype=torch.int32, device=dev)
        self.stream = torch.cuda.Stream(device=dev)
        self.graph = torch.cuda.CUDAGraph()
        self._capture()

    def _layer_calls(self, x, prev):
        if self.fused:
            # early K/V requests only behind another layer's call on other pools
            early = prev is not None and prev["k_cache"].data_ptr() != x["k_cache"].data_ptr() \
                and prev["v_cache"].data_ptr() != x["v_cache"].data_ptr()
            if self.rope:
                ops.rope_store_decode(x["q"], x["k"], x["v"], x["k_cache"], x["v_cache"],
                                      self.slot_mapping, self.block_tables, self.context_lens,
                                      self.scale, self.positions, self.cos_table, self.sin_table,
                                      out=x["out"], num_splits=self.num_splits,
                                      workspace=self.workspace, pdl=True, early_kv=early)
            else:
                ops.store_decode(x["q"], x["k"], x["v"], x["k_cache"], x["v_cache"],
                                 self.slot_mapping, self.block_tables, self.context_lens,
                                 self.scale, out=x["out"], num_splits=self.num_splits,
                                 workspace=self.workspace, pdl=True, early_kv=early)
            return
        if self.rope:
            ops.rope_store_kv(x["q"], x["k"], x["v"], self.positions, self.cos_table,
                              self.sin_table, x["k_cache"], x["v_cache"], self.slot_mapping,
                              q_out=x["q"], error_flags=self.error_word, pdl=True)
        else:
            ops.store_kv(x["k"], x["v"], x["k_cache"], x["v_cache"], self.slot_mapping,
                         error_flags=self.error_word, pdl=True)
        ops.decode(x["q"], x["k_cache"], x["v_cache"], self.block_tables, self.context_lens,
                   self.scale, out=x["out"], num_splits=self.num_splits,
                   workspace=self.workspace, pdl=True)

    def _capture(self):
        # One eager decode call first: kernel attributes (the large dynamic
        # shared memory) are set on a kernel's first launch, which must not
        # happen during capture.  It writes only layer 0's `out`, which every
        # replay rewrites.  The capture itself records the calls without
        # running them, so the pools and q / k / v are left as they are.
        x = self.layers[0]
        ops.decode(x["q"], x["k_cache"], x["v_cache"], self.block_tables, self.context_lens,
                   self.scale, out=x["out"], num_splits=self.num_splits,
                   workspace=self.workspace)
        torch.cuda.synchronize()
        self.stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(self.graph, stream=self.stream):
            prev = None
            for x in self.layers:
                self._layer_calls(x, prev)
                prev = x
        torch.cuda.current_stream().wait_stream(self.stream)

    def launches_per_replay(self) -> int:
        return (1 if self.fused else 2) * len(self.layers)

    def update(self, block_tables=None, context_lens=None, slot_mapping=None, positions=None):
        """Write new values into the static index buffers (same shapes), in
        stream order before the next replay."""
        for src, dst, name in ((block_tables, self.block_tables, "block_tables"),
                               (context_lens, self.context_lens, "context_lens"),
                               (slot_mapping, self.slot_mapping, "slot_mapping"),
                               (positions, self.positions, "positions")):
            if src is None:
                continue
            if dst is None:
                raise ops.PagedAttentionError(f"{name}: this graph has no such buffer")
            if tuple(src.shape) != tuple(dst.shape):
                raise ops.PagedAttentionError(
                    f"{name} has shape {tuple(src.shape)}; the graph was captured with "
                    f"{tuple(dst.shape)}")
            dst.copy_(src.to(torch.int32), non_blocking=True)

    def replay(self):
        """Run the captured step on the current stream (after any update)."""
        self.graph.replay()

    def read_error_word(self) -> int:
        """Device error bits of the store calls (and the decode workspace's)."""
        return int(self.error_word.item()) | ops.read_error_word(self.workspace)


class TreeStepGraph:
    """One speculative step over ``len(layers)`` layers: :meth:`replay` stores
    the drafted nodes' K/V rows and attends to every sequence's tree in all
    layers (one CUDA graph), and, once the target's probabilities of the nodes
    are there, :meth:`verify` accepts a walk down each tree, draws the token
    after it and commits the accepted rows in all pools (another).

    layers: list of dicts with bf16 CUDA tensors ``q`` [T, Hq, D] (contiguous),
    ``k``, ``v`` [T, Hkv, D] (the nodes' rows, packed by cu_seqlens), ``k_cache``,
    ``v_cache`` (the layer's pools) and ``out`` [T, Hq, D].
    cu_seqlens int32 [N + 1], parents, tokens, slot_mapping int32 [T],
    block_tables int32 [N, max_blocks], context_lens int32 [N] (the nodes
    included): the initial values of the static index buffers (copied).
    target_probs (and draft_probs, if there are) float32 [T, V], uniforms
    float32 [T] and sample_uniforms float32 [N]: read where they are.
    ref_counts int32 [num_blocks]: the pages' counts, changed where they are.

    After :meth:`verify`, ``context_lens`` holds the committed lengths, the
    accepted nodes included: the next step's are those plus its trees' nodes.
    """

    def __init__(self, layers, cu_seqlens, parents, tokens, block_tables, context_lens,
                 slot_mapping, scale, max_q_len, target_probs, uniforms, sample_uniforms,
                 draft_probs=None, with_replacement=False, ref_counts=None, num_splits=0,
                 device=None):
        if not layers:
            raise ops.PagedAttentionError("TreeStepGraph needs at least one layer")
        dev = layers[0]["q"].device if device is None else torch.device(device)
        self.layers = layers
        i32 = lambda t: t.to(dev, torch.int32).clone()
        # static index buffers: one copy, shared by every layer
        self.cu_seqlens, self.parents, self.tokens = map(i32, (cu_seqlens, parents, tokens))
        self.block_tables, self.context_lens = i32(block_tables), i32(context_lens)
        self.slot_mapping = i32(slot_mapping)
        self.error_word = torch.zeros(1, dtype=torch.int32, device=dev)
        self.workspace = ops.tree_workspace(num_splits, dev)
        self._store = [(x["k"], x["v"], x["k_cache"], x["v_cache"]) for x in layers]
        self._attend = [
            ops.DecodeTreeCall(x["q"], self.cu_seqlens, self.parents, x["k_cache"], x["v_cache"],
                               self.block_tables, self.context_lens, scale, max_q_len, x["out"],
                               num_splits, self.workspace, pdl=True) for x in layers]
        B = self.cu_seqlens.shape[0] - 1
        self.accepted = torch.zeros(B, dtype=torch.int32, device=dev)
        self.path, self.out_tokens = (torch.full((B, int(max_q_len)), -1, dtype=torch.int32,
                                                 device=dev) for _ in range(2))
        self._verify = ops.VerifyTreeCall(
            self.tokens, self.parents, self.cu_seqlens, target_probs, uniforms, sample_uniforms,
            max_q_len, draft_probs, with_replacement, self.accepted, self.path, self.out_tokens,
            self.error_word, pdl=True)
        pools = ops.PagePools([x[name] for x in layers for name in ("k_cache", "v_cache")])
        self._commit = ops.CommitTreeCall(pools, self.cu_seqlens, self.block_tables,
                                          self.context_lens, self.path, self.accepted, ref_counts,
                                          self.error_word, pdl=True)
        self.stream = torch.cuda.Stream(device=dev)
        self._graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
        self._capture(dev)

    def _capture(self, dev):
        # Eager calls first, so that no kernel's first launch falls into a capture.  They write
        # what every replay rewrites; the commit's is one of a sequence without nodes.
        self._attend[0]()
        self._verify()
        none = torch.zeros(2, dtype=torch.int32, device=dev)
        page = torch.zeros((1, 16, 16), dtype=torch.uint8, device=dev)
        ops.commit_tree(ops.PagePools([page]), none, none[:1].view(1, 1), none[:1],
                        none[:1].view(1, 1), none[:1])
        torch.cuda.synchronize()
        self.error_word.zero_()  # (the tensors may hold anything yet)
        self.workspace[:4].zero_()
        self.stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(self._graphs[0], stream=self.stream):
            for rows, attend in zip(self._store, self._attend):
                ops.store_kv(*rows, self.slot_mapping, error_flags=self.error_word, pdl=True)
                attend()
        with torch.cuda.graph(self._graphs[1], stream=self.stream):
            self._verify()
            self._commit()
        torch.cuda.current_stream().wait_stream(self.stream)

    def update(self, cu_seqlens=None, parents=None, tokens=None, block_tables=None,
               context_lens=None, slot_mapping=None):
        """Write new values into the static index buffers (same shapes), in
        stream order before the next replay.  Trees may have other sizes as long
        as they fit the rows and max_q_len."""
        for src, dst, name in ((cu_seqlens, self.cu_seqlens, "cu_seqlens"),
                               (parents, self.parents, "parents"),
                               (tokens, self.tokens, "tokens"),
                               (block_tables, self.block_tables, "block_tables"),
                               (context_lens, self.context_lens, "context_lens"),
                               (slot_mapping, self.slot_mapping, "slot_mapping")):
            if src is None:
                continue
            if tuple(src.shape) != tuple(dst.shape):
                raise ops.PagedAttentionError(
                    f"{name} has shape {tuple(src.shape)}; the graph was captured with "
                    f"{tuple(dst.shape)}")
            dst.copy_(src.to(torch.int32), non_blocking=True)

    def replay(self):
        """Run the layers' stores and attention on the current stream."""
        self._graphs[0].replay()

    def verify(self):
        """Verify and commit on the current stream (once a step, after
        :meth:`replay` and the target's probabilities).  Returns the static
        (accepted [N], path [N, max_q_len], out_tokens [N, max_q_len])."""
        self._graphs[1].replay()
        return self.accepted, self.path, self.out_tokens

    def read_error_word(self) -> int:
        """Device error bits of the calls so far."""
        return int(self.error_word.item()) | ops.read_error_word(self.workspace)
