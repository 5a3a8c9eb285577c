"""CUDA-graph decode step over the paged cache: one capture per bucket.

Mirrors vLLM-Omni's SenseNova-U1 DecodeGraphRunner without a model: every
input a step varies (the new rows' q/k/v and the segment table holding the
live lengths) sits in static device tensors, so one captured graph of
`num_layers` append+attend launches serves every length in the bucket.  A
capture is keyed on (bucket, generation); a resize bumps the generation and
the next step captures again.  Warm-up runs three times on a side stream
before capture (it rewrites the same rows to the same slots, so it is
idempotent), and every capture shares one graph memory pool: a private pool
per runner grew device memory without bound in the page's measurement.
"""
from __future__ import annotations

import math
from typing import Dict, List, Optional, Sequence, Tuple, Union

import torch

from . import _lib
from .api import (PagedKVCache, Rope, append, append_attend, attend_varlen, attend_workspace_bytes, fp4_keys,
                  new_err_flags, norm_rope_append)
from .api import advance as advance_lengths

_SHARED_POOL = None


def shared_pool():
    global _SHARED_POOL
    if _SHARED_POOL is None:
        _SHARED_POOL = torch.cuda.graph_pool_handle()
    return _SHARED_POOL


def _carve(spec, device) -> Tuple[torch.Tensor, List[torch.Tensor]]:
    """One zeroed uint8 buffer holding tensors of the given (shape, dtype)
    back to back, each at a 16-byte offset; returns it and the typed views."""
    sizes = [math.prod(shape) * torch.empty((), dtype=dt).element_size() for shape, dt in spec]
    offs, total = [], 0
    for n in sizes:
        offs.append(total)
        total += (n + 15) // 16 * 16
    buf = torch.zeros(max(total, 16), dtype=torch.uint8, device=device)
    views = [buf[o:o + n].view(dt).view(shape) for (shape, dt), o, n in zip(spec, offs, sizes)]
    return buf, views


class DecodeStep:
    """Static buffers and launches of one decode step over all layers.

    Every input a step varies (per layer q, k_new, v_new; then the segment
    table) lives in one device buffer, `inputs`, and every output (per layer
    out, then lse) in another, `outputs`; the per-layer tensors are views of
    them, so a step's host round trip is one copy each way.

    With advance=True the step ends with `kv_end += q_len` for every segment
    on the device (tiny-llm kv_cache.py, SlotKVCache.end_step), so a replay
    leaves the segment table ready for the next step and the host writes it
    only once: per step it copies q, k_new and v_new (`step_inputs`) and
    keeps its own copy of the lengths in step (advance_host).

    rope (a Rope for every layer, or one per layer) makes q and k_new the rows
    as the projections give them: each layer is then norm_rope_append, which
    leaves the turned queries in `q_rot`, and the attention over them, two
    launches (fused does not apply).  The angles are those of the rows'
    positions in the cache, on every axis of a rope that has several: right for a text alone, not
    after an image, whose patches take more places in the cache than the text's position moves on.
    positions=True gives the step `positions`, int32 (rows,) or (rows, axes) as its ropes have
    them, which the host fills like q (they are part of `step_inputs`; advance leaves them).  A cache held in 4 or 8 bits takes two launches a layer
    as well, three where large bounds share the key ranges; its outputs may be
    bf16 (out_dtype).  The workspace of that merge belongs to the step: a
    capture allocates nothing, and captured steps share no memory.

    pdl lets a layer's attention start before the launch in front of it has
    finished, and read the sequences' older pages: fused steps (append_attend, no
    two segments of which may name one column) always do.  With a rope two
    segments may be pieces of one sequence, and the older pages of one are
    then written in the same step: by default (None) only a step of one segment
    starts early; True promises that no segment's rows are older keys of another.
    """

    def __init__(self, cache: PagedKVCache, num_q_heads: int, rows: int = 1, num_segments: int = 1,
                 max_q_len: int = 1, max_kv: Optional[int] = None, scale: Optional[float] = None,
                 causal: bool = False, window: int = 0, fused: bool = True, pdl: Optional[bool] = None,
                 flags: int = 0, num_splits: int = 0, with_lse: bool = False, prefetch_next: bool = True,
                 workspace: bool = False, advance: bool = False,
                 rope: Union[Rope, Sequence[Rope], None] = None, out_dtype: torch.dtype = torch.float32,
                 positions: bool = False):
        dev = cache.k[0].device
        L, Hkv, D = cache.num_layers, cache.kv_heads, cache.head_dim
        self.cache = cache
        self.num_q_heads = num_q_heads
        self.max_q_len = max_q_len
        self.max_kv = int(max_kv if max_kv is not None else cache.bucket)
        self.scale = scale if scale is not None else 1.0 / math.sqrt(D)
        self.causal, self.window = causal, window
        self.fused, self.pdl, self.flags, self.num_splits = fused, pdl is None or pdl, flags, num_splits
        self.rope_pdl = num_segments == 1 if pdl is None else pdl
        self.prefetch_next = prefetch_next
        if out_dtype != torch.float32 and not (out_dtype == torch.bfloat16 and cache._quantised):
            raise ValueError("out_dtype is float32, or bfloat16 over a quantised cache")
        self.rope = None if rope is None else [rope] * L if isinstance(rope, Rope) else list(rope)
        if self.rope is not None and len(self.rope) != L:
            raise ValueError("rope needs one entry per layer")
        axes = sorted({r.num_axes for r in self.rope or []})
        if positions and len(axes) != 1:
            raise ValueError("positions are those of a rope, and every layer's has as many axes")
        row = cache.row_dtype
        spec_in = ([((rows, num_q_heads, D), row)] * L + [((rows, Hkv, D), row)] * (2 * L)
                   + ([((rows,) if axes == [1] else (rows, axes[0]), torch.int32)] if positions else []) + [((num_segments, 4), torch.int32)])
        self.inputs, views = _carve(spec_in, dev)
        self.q, self.k_new, self.v_new = views[:L], views[L:2 * L], views[2 * L:3 * L]
        self.positions = views[3 * L] if positions else None
        self.seq_info = views[-1]
        # the per-step part of `inputs` (q, k_new, v_new of every layer, positions): the
        # segment table sits after it
        self.step_inputs = self.inputs[:self.seq_info.data_ptr() - self.inputs.data_ptr()]
        self.advance = advance
        self.q_rot = None if self.rope is None else [torch.zeros(rows, num_q_heads, D, dtype=row, device=dev) for _ in range(L)]
        spec_out = [((rows, num_q_heads, D), out_dtype)] * L
        if with_lse:
            spec_out += [((rows, num_q_heads), torch.float32)] * L
        self.outputs, views = _carve(spec_out, dev)
        self.out = views[:L]
        self.lse = views[L:] if with_lse else [None] * L
        self.err = new_err_flags(dev)
        self.use_workspace = workspace
        self.ws = None
        self.size_workspace()

    def size_workspace(self) -> None:
        """(Re)allocate the split-merge workspace where the current cache and bounds need another size (None: they need none)."""
        quantised, n = self.cache._quantised, 0
        if self.use_workspace or (quantised and self.num_splits == 0):
            keys = fp4_keys(self.max_kv, self.max_q_len, self.window) if quantised else self.max_kv
            n = attend_workspace_bytes(self.cache, self.num_q_heads, int(self.seq_info.shape[0]), self.max_q_len, keys,
                                       self.num_splits, self.flags)
        if n <= 0:
            self.ws = None
        elif self.ws is None or self.ws.numel() != n:
            make = torch.empty if quantised else torch.zeros  # (a quantised cache's need not be zeroed)
            self.ws = make(n, dtype=torch.uint8, device=self.cache.k[0].device)

    def launch_count(self) -> int:
        """Kernels of one run (a quantised cache's merge launches, which its bounds decide, not counted)."""
        one = self.fused and self.rope is None and not self.cache._quantised
        return self.cache.num_layers * (1 if one else 2) + (1 if self.advance else 0)

    def run(self, stream=None, advance: Optional[bool] = None) -> None:
        """Enqueue every layer's append + attention on the current stream,
        then (advance=True, by default the step's setting) the on-device
        length advance."""
        c = self.cache
        for layer in range(c.num_layers):
            flags = self.flags
            if self.rope_pdl if self.rope is not None else self.pdl and layer > 0 and self.fused:
                flags |= _lib.FLAG_PDL
            if self.prefetch_next and layer + 1 < c.num_layers:
                flags |= _lib.FLAG_PREFETCH_NEXT  # the next call attends layer + 1 over the same segments
            if self.rope is not None:
                norm_rope_append(c, layer, self.rope[layer], self.q[layer], self.k_new[layer], self.v_new[layer],
                                 self.seq_info, self.q_rot[layer], self.err, positions=self.positions, window=self.window, stream=stream)
                attend_varlen(c, layer, self.q_rot[layer], self.seq_info, self.out[layer], self.err, self.max_q_len,
                              self.max_kv, self.scale, self.causal, self.window, lse=self.lse[layer],
                              num_splits=self.num_splits, flags=flags, stream=stream, workspace=self.ws)
            elif self.fused:
                append_attend(c, layer, self.q[layer], self.k_new[layer], self.v_new[layer], self.seq_info,
                              self.out[layer], self.err, self.max_q_len, self.max_kv, self.scale, self.causal,
                              self.window, lse=self.lse[layer], num_splits=self.num_splits, flags=flags,
                              stream=stream, workspace=self.ws)
            else:
                append(c, layer, self.k_new[layer], self.v_new[layer], self.seq_info, self.err,
                       window=self.window, stream=stream)
                attend_varlen(c, layer, self.q[layer], self.seq_info, self.out[layer], self.err, self.max_q_len,
                              self.max_kv, self.scale, self.causal, self.window, lse=self.lse[layer],
                              num_splits=self.num_splits, flags=flags, stream=stream, workspace=self.ws)
        if self.advance if advance is None else advance:
            advance_lengths(self.seq_info, stream=stream)


class DecodeGraphRunner:
    """One captured DecodeStep per (bucket, generation), replayed for every length."""

    def __init__(self, step: DecodeStep):
        self.step_bufs = step
        self._graphs: Dict[Tuple[int, int], torch.cuda.CUDAGraph] = {}
        self.captures = 0

    def _capture(self, key):
        st = self.step_bufs
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            # Warm-up leaves the lengths alone (a warm-up that advanced them
            # would move the step three tokens on); the advance kernel is
            # warmed on a scratch row instead.
            for _ in range(3):
                st.run(advance=False)
            if st.advance:
                advance_lengths(torch.zeros(1, 4, dtype=torch.int32, device=st.seq_info.device))
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=shared_pool()):
            st.run()
        self.captures += 1
        self._graphs[key] = graph
        return graph

    def rebind(self, cache: PagedKVCache) -> None:
        """Point the step at a resized cache; captures of older buffers are dropped."""
        st = self.step_bufs
        st.cache = cache
        st.max_kv = cache.bucket
        ws = st.ws
        st.size_workspace()
        if ws is not None and st.ws is not ws:  # every capture holds the old one
            ws.record_stream(torch.cuda.current_stream(ws.device))  # (a replay of theirs may still run)
            self._graphs = {}
        self._graphs = {k: g for k, g in self._graphs.items() if k == (cache.bucket, cache.generation)}

    def graph_for(self) -> torch.cuda.CUDAGraph:
        c = self.step_bufs.cache
        key = (c.bucket, c.generation)
        return self._graphs.get(key) or self._capture(key)

    def step(self) -> None:
        """Replay the step for whatever lengths the segment table holds now."""
        self.graph_for().replay()
