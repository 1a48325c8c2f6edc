"""Whole decode steps captured in CUDA graphs.

The pages' system part (gist.science explainer, Methodology 3, "Fused Kernel
and System Optimization": the entire decoding step is captured in a CUDA graph
to remove CPU launch overhead at small batch) applied to the FFD step:

* :class:`DecodeStep` -- one layer's FFD decode with host-side inputs and
  outputs, as the library's native step graph (``ffd_step_graph_*``): the H2D
  copy of the step's query and new K/V rows from pinned memory, optionally the
  length increment, and the fused append + re-quantisation + decode launch
  (``ffd_decode_append``), whose kernel writes the output rows and the mask
  straight into pinned host memory (or, with ``results_to_host`` off, one D2H
  copy does).  A step is one call into the library, which launches the graph
  and waits.
* :class:`StandInAttentionLayer` -- a decode-step attention layer with random
  weights (there is no checkpoint): q, k and v projections of the hidden
  state, the FFD step, the output projection, captured whole.  The
  projections are plain library GEMMs (torch.matmul); every attention step
  runs in the FFD kernel, with rotary positions before it where asked for.
* :class:`TreeStep` -- verification of a tree of drafted tokens a sequence:
  rotary positions and the cache write of all nodes (``ffd_append_tokens``),
  their attention over the cache (``ffd_decode_tree``), captured whole, and the
  accepted nodes' rows moved to where an accepted sequence has them.

PyTorch provides the memory, streams and graphs; the compute of the attention
step is the CUDA library's.
"""
from __future__ import annotations

import math
from typing import Optional

from . import ffd


def _require_torch():
    import torch
    if not torch.cuda.is_available():
        raise RuntimeError("the FFD decode step needs a CUDA device")
    return torch


class DecodeStep:
    """One attention layer's decode step, captured in a CUDA graph.

    k_cache, v_cache: bf16 [B, Hkv, cap, 128] device tensors, prefilled;
    lengths: int32 [B] device tensor, the lengths BEFORE the first step when
    ``advance`` is set (each step adds one token), else the lengths including
    the new token.  fmt: "int4" (int4 scan copy + bf16 K/V) or "tr" (2-bit
    thumbnails + 8-bit residuals).  The key copies are built here from the
    cache for the current lengths.

    Per step the caller writes the query [B, Hq, 128] and the new token's K/V
    rows [B, Hkv, 128] into ``host_q``, ``host_k_new``, ``host_v_new``
    (pinned), calls :meth:`step`, and reads ``host_out`` [B, Hq, 128] and
    ``host_mask`` [B, Hkv, words].  A sequence whose length would pass the
    capacity is reported by the device flag (see :meth:`check`) and yields a
    zero row.
    """

    def __init__(self, shape: ffd.Shape, k_cache, v_cache, lengths, delta: float,
                 reference: int = ffd.FFD_REFERENCE_RUNNING_MAX, fmt: str = "int4",
                 advance: bool = False, results_to_host: bool = True):
        torch = _require_torch()
        if fmt not in ("int4", "tr"):
            raise ValueError("fmt must be 'int4' or 'tr'")
        self.torch, self.shape, self.fmt = torch, shape, fmt
        # the graph's kernel writes output and mask straight into pinned host
        # memory (no D2H copy) unless results_to_host is off
        self.results_to_host = bool(results_to_host)
        self.delta, self.reference, self.advance = float(delta), int(reference), bool(advance)
        self.k, self.v, self.lengths = k_cache, v_cache, lengths
        dev = k_cache.device
        B, Hq, Hkv, D = shape.batch, shape.num_q_heads, shape.num_kv_heads, shape.head_dim
        self.bufs = (ffd.ThumbResidBuffers(shape, device=dev) if fmt == "tr"
                     else ffd.DecodeBuffers(shape, device=dev))
        b = self.bufs
        if fmt == "tr":
            ffd.quantize_keys_tr(shape, k_cache, lengths, 0, b.k_thumb, b.k_resid, b.k_scales)
        else:
            ffd.quantize_keys(shape, k_cache, lengths, 0, b.k_packed, b.k_scales)
        nq, nk = B * Hq * D, B * Hkv * D
        self._host_in = torch.empty(nq + 2 * nk, dtype=torch.bfloat16).pin_memory()
        self._dev_in = torch.empty(nq + 2 * nk, dtype=torch.bfloat16, device=dev)
        self.host_q = self._host_in[:nq].view(B, Hq, D)
        self.host_k_new = self._host_in[nq:nq + nk].view(B, Hkv, D)
        self.host_v_new = self._host_in[nq + nk:].view(B, Hkv, D)
        self._q = self._dev_in[:nq].view(B, Hq, D)
        self._k_new = self._dev_in[nq:nq + nk].view(B, Hkv, D)
        self._v_new = self._dev_in[nq + nk:].view(B, Hkv, D)
        # output rows and mask share one device buffer, so one D2H copy returns both
        mask_shape = tuple(b.mask.shape)
        out_bytes = B * Hq * D * 2
        mask_off = (out_bytes + 15) // 16 * 16
        total = mask_off + (mask_shape[0] * mask_shape[1] * mask_shape[2]) * 4
        self._mask_off = mask_off
        self._dev_res = torch.empty(total, dtype=torch.uint8, device=dev)
        self._host_res = torch.empty(total, dtype=torch.uint8).pin_memory()
        b.out = self._dev_res[:out_bytes].view(torch.bfloat16).view(B, Hq, D)
        b.mask = self._dev_res[mask_off:].view(torch.int32).view(mask_shape)
        self.host_out = self._host_res[:out_bytes].view(torch.bfloat16).view(B, Hq, D)
        self.host_mask = self._host_res[mask_off:].view(torch.int32).view(mask_shape)
        self.h2d_bytes = self._host_in.numel() * 2
        self.d2h_bytes = total
        self._stream = torch.cuda.Stream(dev)
        self._graph: Optional[object] = None

    def _launch(self):
        b = self.bufs
        if self.advance:
            self.lengths.add_(1)
        if self.fmt == "tr":
            ffd.decode_append_tr(self.shape, self._q, self._k_new, self._v_new, self.k, self.v,
                                 b.k_thumb, b.k_resid, b.k_scales, self.lengths, self.delta, b.out,
                                 b.mask, b.workspace, reference=self.reference)
        else:
            ffd.decode_append(self.shape, self._q, self._k_new, self._v_new, self.k, self.v,
                              b.k_packed, b.k_scales, self.lengths, self.delta, b.out, b.mask,
                              b.workspace, reference=self.reference)

    def _body(self):
        self._dev_in.copy_(self._host_in, non_blocking=True)
        self._launch()
        self._host_res.copy_(self._dev_res, non_blocking=True)

    def capture(self):
        """Build the native step graph (done by the first :meth:`step`).
        Nothing runs at capture; earlier device work on the caches is ordered
        first by a device synchronisation."""
        self.torch.cuda.synchronize(self.k.device)
        b = self.bufs
        tr = self.fmt == "tr"
        self._graph = ffd.StepGraph(
            self.shape, 1 if tr else 0, self.reference, self.delta, self.advance, self._host_in,
            self._dev_in, self.k, self.v, b.k_thumb if tr else b.k_packed, b.k_resid if tr else None,
            b.k_scales, self.lengths, None if self.results_to_host else self._dev_res,
            self._host_res, self._mask_off, b.workspace)
        return self._graph

    def step(self):
        """One decode step: host inputs -> host outputs (one library call)."""
        if self._graph is None:
            self.capture()
        self._graph.run()

    def check(self) -> int:
        """Device flags (ffd.FFD_DEVICE_FLAG_*) raised since the last check."""
        return ffd.check_device_status(self.bufs.workspace)


class StandInAttentionLayer:
    """A decode-step attention layer with random weights around the FFD step.

    hidden: model width; weights drawn N(0, 1/hidden) from ``seed`` (bf16):
    w_q [hidden, Hq*128], w_k and w_v [hidden, Hkv*128], w_o [Hq*128, hidden].
    A step takes x [B, hidden] (pinned host ``host_x``), appends the new
    token's k/v to the caches, attends with FFD and writes the projected output
    [B, hidden] to ``host_y``.  lengths and ``advance`` as for DecodeStep (with
    advance off every step re-appends at position lengths - 1).  With `rope` (an
    ffd.Rope) q and k are rotated in place by the new token's position, between
    the projections and the step; the keys in the cache are then taken to be
    rotated.  No normalisation: this is a stand-in that exercises the step's data
    flow, not a model.
    """

    def __init__(self, shape: ffd.Shape, hidden: int, k_cache, v_cache, lengths, delta: float,
                 seed: int = 0, reference: int = ffd.FFD_REFERENCE_RUNNING_MAX, fmt: str = "int4",
                 advance: bool = True, rope: Optional[ffd.Rope] = None):
        torch = _require_torch()
        self.torch, self.shape, self.rope = torch, shape, rope
        dev = k_cache.device
        B, Hq, Hkv, D = shape.batch, shape.num_q_heads, shape.num_kv_heads, shape.head_dim
        gen = torch.Generator(device="cpu").manual_seed(int(seed))

        def weight(rows, cols):
            w = torch.randn((rows, cols), generator=gen, dtype=torch.float32) / math.sqrt(rows)
            return w.to(dtype=torch.bfloat16, device=dev)

        self.w_q, self.w_k = weight(hidden, Hq * D), weight(hidden, Hkv * D)
        self.w_v, self.w_o = weight(hidden, Hkv * D), weight(Hq * D, hidden)
        self.core = DecodeStep(shape, k_cache, v_cache, lengths, delta, reference=reference,
                               fmt=fmt, advance=advance)
        self.host_x = torch.empty((B, hidden), dtype=torch.bfloat16).pin_memory()
        self.host_y = torch.empty((B, hidden), dtype=torch.bfloat16).pin_memory()
        self._x = torch.empty((B, hidden), dtype=torch.bfloat16, device=dev)
        self._y = torch.empty((B, hidden), dtype=torch.bfloat16, device=dev)
        self._position = torch.empty(B, dtype=torch.int32, device=dev)
        self._stream = torch.cuda.Stream(dev)
        self._graph = None

    def _body(self):
        torch, c = self.torch, self.core
        B = self.shape.batch
        self._x.copy_(self.host_x, non_blocking=True)
        torch.matmul(self._x, self.w_q, out=c._q.view(B, -1))
        torch.matmul(self._x, self.w_k, out=c._k_new.view(B, -1))
        torch.matmul(self._x, self.w_v, out=c._v_new.view(B, -1))
        if self.rope is not None:  # the new token's slot
            torch.sub(c.lengths, 0 if c.advance else 1, out=self._position)
            ffd.rotate(self.rope, self._position, c._q, c._q, c._k_new, c._k_new)
        c._launch()
        torch.matmul(c.bufs.out.view(B, -1), self.w_o, out=self._y)
        self.host_y.copy_(self._y, non_blocking=True)

    def capture(self):
        """As DecodeStep.capture: one eager run with the current host_x first."""
        torch = self.torch
        saved = self.core.lengths.clone()
        with torch.cuda.stream(self._stream):
            self._body()
        self._stream.synchronize()
        self.core.lengths.copy_(saved)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=self._stream):
            self._body()
        self._graph = g
        torch.cuda.synchronize(self._x.device)
        return g

    def step(self):
        if self._graph is None:
            self.capture()
        self._graph.replay()
        self.torch.cuda.current_stream(self._x.device).synchronize()


class TreeStep:
    """One attention layer's verification of drafted tokens, captured in a CUDA
    graph.

    cache: an ffd.KVCache of either format, whose first ``lengths`` tokens
    (int32 [B], device) are the sequences so far.  A step takes up to num_nodes
    drafted tokens a sequence from static device buffers that the caller fills:
    ``q`` [B, n, Hq, 128], ``k_new``, ``v_new`` [B, n, Hkv, 128] (bf16, before
    rotation), ``tree_mask`` int64 [B, n] and ``depth`` int32 [B, n]
    (ffd.tree_from_parents makes both), ``sizes`` int32 [B].  They start as a
    chain of num_nodes.  :meth:`step` rotates queries and keys by lengths + depth
    (with `rope`), writes the nodes behind the sequences and attends; results are
    in ``out`` [B, n, Hq, 128], on the current stream.  ``lengths`` stays: the
    nodes are drafts until :meth:`accept` keeps some.  A sequence without room for
    its nodes, or with more than num_nodes of them, yields zero rows and
    FFD_DEVICE_FLAG_BAD_LENGTH (:meth:`check`).
    """

    def __init__(self, shape: ffd.Shape, cache: "ffd.KVCache", lengths, num_nodes: int,
                 rope: Optional[ffd.Rope] = None):
        torch = _require_torch()
        self.torch, self.shape, self.cache, self.lengths, self.rope = torch, shape, cache, lengths, rope
        B, Hq, Hkv, n = shape.batch, shape.num_q_heads, shape.num_kv_heads, int(num_nodes)
        dev = lengths.device
        bf16, i32 = torch.bfloat16, torch.int32
        cache._of(shape)
        ffd._tensor(lengths, i32, (B,), "lengths", cache.device)
        self.workspace = ffd.tree_workspace(shape, n, device=dev)
        self._flags = self.workspace[:4].view(i32)  # what ffd_check_device_status reads
        self.q, self.out, self._rotated = (torch.zeros((B, n, Hq, 128), dtype=bf16, device=dev) for _ in range(3))
        self.k_new, self.v_new = (torch.zeros((B, n, Hkv, 128), dtype=bf16, device=dev) for _ in range(2))
        mask, depth = ffd.tree_from_parents([list(range(-1, n - 1))] * B)
        self.tree_mask, self.depth = mask.to(dev), depth.to(dev)
        self.sizes = torch.full((B,), n, dtype=i32, device=dev)
        self._total = torch.empty(B, dtype=i32, device=dev)
        self._positions = torch.empty((B, n), dtype=i32, device=dev)
        self._stream = torch.cuda.Stream(dev)
        self._graph = None

    def _body(self):
        torch = self.torch
        torch.add(self.lengths, self.sizes, out=self._total)
        torch.add(self.lengths[:, None], self.depth, out=self._positions)
        ffd.append_tokens(self.shape, self.cache, self.k_new, self.v_new, self._total, rope=self.rope,
                          positions=self._positions, new_lengths=self.sizes, q=self.q, q_out=self._rotated)
        ffd.decode_tree(self.shape, self.cache, self._rotated, self._total, self.out, self.workspace,
                        tree_mask=self.tree_mask, tree_sizes=self.sizes)

    def capture(self):
        """Capture the step's graph (done by the first :meth:`step`).  Nothing
        runs at capture."""
        torch = self.torch
        torch.cuda.synchronize(self.lengths.device)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=self._stream):
            self._body()
        self._graph = g
        return g

    def step(self):
        """One verification step; returns ``out`` (not waited for)."""
        if self._graph is None:
            self.capture()
        self._graph.replay()
        return self.out

    def accept(self, nodes, counts):
        """Keep counts[b] nodes of each sequence, nodes[b, :counts[b]] in order
        (int64 [B, m] and int32 [B], on the device; the rest of a row is
        ignored): node i of the list becomes token lengths[b] + i, rotated for
        that position, and ``lengths`` grows by counts.  The list is a path of the
        tree from a root, so its keys are the ones already attended to.  (The low-bit
        keys of ffd.decode on the same cache are the caller's: quantize_keys from the
        first block that changed on.)  A sequence
        whose count is outside [0, m], that has no room for it, or whose list names a
        node outside [0, sizes[b]) stays as it is, and FFD_DEVICE_FLAG_BAD_LENGTH is
        raised (:meth:`check`)."""
        torch, B, n = self.torch, self.shape.batch, self.k_new.shape[1]
        dev = self.lengths.get_device()
        if nodes.dim() != 2:
            raise ValueError(f"nodes: want int64 [B, m], got {tuple(nodes.shape)}")
        m = nodes.shape[1]
        ffd._tensor(counts, torch.int32, (B,), "counts", dev)
        if nodes.dtype is not torch.int64 or nodes.shape[0] != B or nodes.get_device() != dev:
            raise ValueError(f"nodes: want int64 [{B}, m] on cuda:{dev}, got {nodes.dtype} {tuple(nodes.shape)} "
                             f"on {nodes.device}")
        if m > self.shape.capacity:
            raise ValueError(f"nodes: {m} a sequence are more than the cache holds")
        listed = torch.arange(m, device=nodes.device) < counts[:, None]
        known = (nodes >= 0) & (nodes < self.sizes[:, None])
        good = ((known | ~listed).all(1) & (counts >= 0) & (counts <= m) & (self.lengths >= 0) &
                (self.lengths <= self.shape.capacity - counts))
        self._flags.bitwise_or_((~good).any().to(torch.int32) * ffd.FFD_DEVICE_FLAG_BAD_LENGTH)
        kept = torch.where(good, counts, 0)
        at = nodes.clamp(0, n - 1)[:, :, None, None].expand(B, m, self.shape.num_kv_heads, 128)
        self.lengths.add_(kept)
        ffd.append_tokens(self.shape, self.cache, self.k_new.gather(1, at), self.v_new.gather(1, at), self.lengths,
                          rope=self.rope, new_lengths=kept)

    def check(self) -> int:
        """Device flags (ffd.FFD_DEVICE_FLAG_*) raised since the last check."""
        return ffd.check_device_status(self.workspace)
