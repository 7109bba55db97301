"""One MLA layer's decode step as the five C-ABI calls, in the pages' order.

[P5] "MLA · latent KV, decoupled RoPE và matrix absorption", section 2
"Luồng": project the hidden state to the latent, write the cache, then read
it and project the output.  Here that is: append the new latent rows, build
the absorbed queries, run split-KV decode over the paged cache, merge the
splits, and apply W_UV / W_O.  All buffers are allocated once, up front.
"""

from __future__ import annotations

import dataclasses
from typing import Dict, Optional

import torch

from . import abi


class DecodeLayer:
    def __init__(self, cfg: abi.Config, weights: Dict[str, torch.Tensor], cache: abi.Cache,
                 batch: int, n_q: int, max_workers: int = 0, packed_query: bool = True):
        self.cfg, self.W, self.cache = cfg, weights, cache
        self.batch, self.n_q, self.max_workers = batch, n_q, max_workers
        n = batch * n_q
        dev = cache.pool.device
        dt = cfg.torch_dtype
        H = cfg.n_heads
        # An FP8 cache is appended as E4M3 rows; each step expands its visible
        # pages into a bf16 scratch cache (mla_cache_dequant_fp8) that the bf16
        # tensor-core path decodes: `dcfg` / `dcache` are what the queries, the
        # decode and the projections see.
        self.dcfg, self.dcache, self.fp8_scratch = cfg, cache, None
        if cfg.fp8_cache and packed_query:
            self.dcfg = dataclasses.replace(cfg, fp8_cache=False)
            mb = cache.block_table.shape[1]
            self.fp8_scratch = torch.empty(abi.mla_fp8_scratch_bytes(cfg, batch, mb), dtype=torch.uint8, device=dev)
            self.dcache = abi.fp8_scratch_cache(self.dcfg, self.fp8_scratch, batch, mb)
        cfg = self.dcfg
        # bf16: the absorbed query goes from the projection to the decode in the
        # decode's packed bf16 layout (no fp32 round trip); fp32: q_lat / q_rope
        self.packed = packed_query and abi.mla_query_packed_bytes(cfg, n) > 0
        if self.packed:
            rows = (2 if cfg.split_query else 1) * n
            self.q_packed = torch.empty(rows, H, cfg.d_c + cfg.d_r, dtype=torch.bfloat16, device=dev)
        else:
            self.q_lat = torch.empty(n, H, cfg.d_c, dtype=torch.float32, device=dev)
            self.q_rope = torch.empty(n, H, cfg.d_r, dtype=torch.float32, device=dev)
        self.o_lat = torch.empty(n, H, cfg.d_c, dtype=torch.float32, device=dev)
        self.y = torch.empty(n, cfg.hidden, dtype=dt, device=dev)
        # bf16: the split combine runs inside the W_UV projection (mla_combine_out_proj)
        self.fused_out = cfg.dtype == "bf16" and abi.mla_combine_out_proj_workspace_size(cfg, batch, n_q) > 0
        gemm_ws = max(abi.mla_cache_append_workspace_size(cfg, n), abi.mla_absorb_q_workspace_size(cfg, n),
                      abi.mla_out_proj_workspace_size(cfg, n),
                      abi.mla_combine_out_proj_workspace_size(cfg, batch, n_q) if self.fused_out else 0)
        self.ws_gemm = torch.empty(max(gemm_ws, 256), dtype=torch.uint8, device=dev)
        self.ws_decode = torch.empty(abi.mla_decode_workspace_size(cfg, batch, n_q, max_workers),
                                     dtype=torch.uint8, device=dev)
        # The step's append runs on a second stream beside the query projections
        # (fp64 work next to weight streaming), with a workspace of its own.
        self.side = torch.cuda.Stream(device=dev)
        self.ws_append = torch.empty(max(abi.mla_cache_append_workspace_size(cfg, n), 256), dtype=torch.uint8,
                                     device=dev)

    def _gemm_ws(self, n: int) -> torch.Tensor:
        need = max(abi.mla_cache_append_workspace_size(self.cfg, n), abi.mla_absorb_q_workspace_size(self.cfg, n),
                   abi.mla_out_proj_workspace_size(self.cfg, n))
        if need > self.ws_gemm.numel():
            self.ws_gemm = torch.empty(need, dtype=torch.uint8, device=self.ws_gemm.device)
        return self.ws_gemm

    def append(self, x, seq_idx, pos, stream=None):
        self._gemm_ws(x.shape[0])
        abi.mla_cache_append(self.cfg, x, self.W["W_DKV"], self.W["W_KR"], seq_idx, pos, self.cache,
                             self.ws_gemm, stream)

    def queries(self, x, pos, stream=None):
        W_DQ = self.W.get("W_DQ")
        W_UQ = self.W["W_UQ"] if "W_UQ" in self.W else self.W["W_Q"]
        if self.packed:
            abi.mla_absorb_q_packed(self.dcfg, x, W_DQ, W_UQ, self.W["W_UK"], pos, self.q_packed, self.ws_gemm,
                                    stream)
        else:
            abi.mla_absorb_q(self.dcfg, x, W_DQ, W_UQ, self.W["W_UK"], pos, self.q_lat, self.q_rope,
                             self.ws_gemm, stream)

    def queries_fp32(self):
        """(q_lat, q_rope) of the last step as fp32 tensors (for checks): the
        fp32 outputs, or the packed bf16 rows (plus their remainders in
        split-query mode) widened."""
        if not self.packed:
            return self.q_lat, self.q_rope
        n = self.batch * self.n_q
        q = self.q_packed[:n].float()
        if self.dcfg.split_query:
            q = q + self.q_packed[n:].float()
        return q[..., :self.dcfg.d_c], q[..., self.dcfg.d_c:]

    def append_and_queries(self, x, seq_idx, pos, stream=None, seq_lens=None):
        """The append and the query projections of one step, overlapped: the
        projections go first on ``stream`` (so their CTAs are placed first), the
        append on a side stream; ``stream`` waits for both before returning.
        With ``seq_lens`` (packed-query path) the side stream also computes the
        decode's split plan, and the next ``decode(..., planned=True)`` skips it."""
        main = stream or torch.cuda.current_stream()
        ready = torch.cuda.Event()
        ready.record(main)
        self.queries(x, pos, main)
        self.side.wait_event(ready)
        need = abi.mla_cache_append_workspace_size(self.cfg, x.shape[0])
        if need > self.ws_append.numel():
            self.ws_append = torch.empty(need, dtype=torch.uint8, device=self.ws_append.device)
        abi.mla_cache_append(self.cfg, x, self.W["W_DKV"], self.W["W_KR"], seq_idx, pos, self.cache,
                             self.ws_append, self.side)
        keep = [x, seq_idx, pos]
        if seq_lens is not None and self.packed:
            abi.mla_decode_plan(self.dcfg, self.batch, self.n_q, self.dcache, seq_lens, self.ws_decode,
                                self.max_workers, self.side)
            keep.append(seq_lens)
        done = torch.cuda.Event()
        done.record(self.side)
        main.wait_event(done)
        # keep the inputs alive until the side stream has used them
        for t in keep:
            t.record_stream(self.side)

    def decode(self, seq_lens, stream=None, planned=False):
        """Split-KV decode; ``planned``: the plan is already in the workspace
        (``append_and_queries`` with ``seq_lens``, same sequence lengths)."""
        if self.fp8_scratch is not None:   # this step's visible FP8 pages -> the bf16 scratch cache
            abi.mla_cache_dequant_fp8(self.cfg, self.cache, self.batch, seq_lens, self.fp8_scratch, stream)
        if self.packed and planned:
            abi.mla_decode_packed_planned(self.dcfg, self.q_packed, self.batch, self.n_q, self.dcache, seq_lens,
                                          self.ws_decode, self.max_workers, stream)
        elif self.packed:
            abi.mla_decode_packed(self.dcfg, self.q_packed, self.batch, self.n_q, self.dcache, seq_lens,
                                  self.ws_decode, self.max_workers, stream)
        else:
            abi.mla_decode(self.dcfg, self.q_lat, self.q_rope, self.batch, self.n_q, self.dcache, seq_lens,
                           self.ws_decode, self.max_workers, stream)

    def combine(self, stream=None):
        abi.mla_combine(self.dcfg, self.ws_decode, self.batch, self.n_q, self.o_lat, stream)

    def attend(self, seq_lens, stream=None):
        """Decode, then the latent output ``o_lat`` (merged splits, fp32)."""
        self.decode(seq_lens, stream)
        self.combine(stream)

    def project(self, stream=None, y=None):
        """``y`` from this step's decode: on the bf16 path the split merge runs
        inside the W_UV projection (``o_lat`` is not needed); otherwise from
        ``o_lat`` (after ``combine``)."""
        y = self.y if y is None else y
        if self.fused_out:
            abi.mla_combine_out_proj(self.dcfg, self.ws_decode, self.batch, self.n_q, self.W["W_UV"], self.W["W_O"],
                                     y, self.ws_gemm, self.max_workers, stream)
        else:
            abi.mla_out_proj(self.dcfg, self.o_lat, self.W["W_UV"], self.W["W_O"], y, self.ws_gemm, stream)

    def step(self, x, seq_idx, pos, seq_lens, stream=None, want_o_lat: bool = False) -> torch.Tensor:
        """Device-resident step: returns ``y`` ``[batch * n_q, hidden]`` (a reused buffer).
        ``want_o_lat`` also fills ``self.o_lat`` (always filled on the fp32 path)."""
        self.append_and_queries(x, seq_idx, pos, stream, seq_lens=seq_lens)
        self.decode(seq_lens, stream, planned=self.packed)
        if want_o_lat or not self.fused_out:
            self.combine(stream)
        self.project(stream)
        return self.y

    def capture_step(self, x, seq_idx, pos, seq_lens, want_o_lat: bool = False) -> torch.cuda.CUDAGraph:
        """Record one ``step`` on these device buffers as a CUDA graph: the
        launches (and the side-stream fork and join) are replayed by
        ``graph.replay()`` without host work.  Refill ``x``, ``seq_idx``,
        ``pos`` and ``seq_lens`` in place between replays; ``self.y`` holds the
        result.  One eager step runs first (outside the capture) so that every
        kernel's one-time setup is done; it appends the same rows the replays
        append again."""
        self.step(x, seq_idx, pos, seq_lens, want_o_lat=want_o_lat)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step(x, seq_idx, pos, seq_lens, want_o_lat=want_o_lat)
        return graph

    def run_from_host(self, inputs, y_hosts, between=None, stream=None, copy_stream=None):
        """Several steps over host (pinned) inputs, pipelined.

        ``inputs[k]`` is ``(x, seq_idx, pos, seq_lens)`` on the host for step k;
        step k's ``y`` lands in ``y_hosts[k]``.  The host-to-device copy of step
        k + 1's inputs and the device-to-host copy of step k's ``y`` run on
        ``copy_stream`` while step k computes on ``stream`` (double-buffered
        device inputs and outputs), as a serving loop would overlap them.
        ``between(k)``, if given, runs on ``stream`` before step k's compute.
        Returns the host buffers; the caller synchronises."""
        stream = stream or torch.cuda.current_stream()
        copy_stream = copy_stream or self._copy_stream()
        dev = self.cache.pool.device
        n = len(inputs)
        if n == 0:
            return y_hosts
        shapes = tuple((tuple(t.shape), t.dtype) for t in inputs[0])
        if getattr(self, "_pipe_shapes", None) != shapes:   # kept across calls: work may still be in flight
            self._pipe_bufs = ([[torch.empty_like(t, device=dev) for t in inputs[0]] for _ in range(2)],
                               [torch.empty_like(self.y) for _ in range(2)])
            self._pipe_shapes = shapes
        dbuf, ybuf = self._pipe_bufs
        copy_stream.wait_stream(stream)   # nothing of this call starts before work already queued on stream
        loaded = [torch.cuda.Event() for _ in range(n)]
        computed = [torch.cuda.Event() for _ in range(n)]
        drained = [torch.cuda.Event() for _ in range(n)]

        def load(k):
            with torch.cuda.stream(copy_stream):
                if k >= 2:   # the step that last used this input buffer has finished
                    copy_stream.wait_event(computed[k - 2])
                for d, h in zip(dbuf[k % 2], inputs[k]):
                    d.copy_(h, non_blocking=True)
                loaded[k].record(copy_stream)

        load(0)
        for k in range(n):
            if k + 1 < n:
                load(k + 1)
            stream.wait_event(loaded[k])
            if k >= 2:       # the y buffer of step k - 2 has been copied out
                stream.wait_event(drained[k - 2])
            if between is not None:
                between(k)
            x, seq_idx, pos, seq_lens = dbuf[k % 2]
            self.append_and_queries(x, seq_idx, pos, stream, seq_lens=seq_lens)
            self.decode(seq_lens, stream, planned=self.packed)
            if not self.fused_out:
                self.combine(stream)
            self.project(stream, y=ybuf[k % 2])
            computed[k].record(stream)
            with torch.cuda.stream(copy_stream):
                copy_stream.wait_event(computed[k])
                y_hosts[k].copy_(ybuf[k % 2], non_blocking=True)
                drained[k].record(copy_stream)
        stream.wait_event(drained[n - 1])
        return y_hosts

    def _copy_stream(self):
        if getattr(self, "_copies", None) is None:
            self._copies = torch.cuda.Stream(device=self.cache.pool.device)
        return self._copies

    def step_from_host(self, x_host, seq_idx_host, pos_host, seq_lens_host, y_host,
                       stream: Optional[torch.cuda.Stream] = None):
        """Same step with host (pinned) inputs and output; copies are on ``stream``."""
        stream = stream or torch.cuda.current_stream()
        with torch.cuda.stream(stream):
            dev = self.cache.pool.device
            x = x_host.to(dev, non_blocking=True)
            seq_idx = seq_idx_host.to(dev, non_blocking=True)
            pos = pos_host.to(dev, non_blocking=True)
            seq_lens = seq_lens_host.to(dev, non_blocking=True)
            y = self.step(x, seq_idx, pos, seq_lens, stream)
            y_host.copy_(y, non_blocking=True)
        return y_host


def _refuse_without_a_step(cfg: abi.Config):
    """Configurations of which a ragged step's kernels do not take every part: bf16 queries are packed for the
    tensor-core attention's shape only, and the CUDA-core attention takes rows of up to 1024 values."""
    if cfg.dtype == "bf16":
        shape = (cfg.n_heads, cfg.d_c, cfg.d_r, cfg.block_size)
        if shape != (128, 512, 64, 64):
            raise ValueError("RaggedLayer: bf16 takes 128 heads, d_c 512, d_r 64 and pages of 64, got "
                             f"{cfg.n_heads}, {cfg.d_c}, {cfg.d_r} and {cfg.block_size}")
        if abi.mla_out_proj_workspace_size(cfg, 1) == 0:
            raise ValueError("RaggedLayer: no tensor-core projections of this hidden, q_lora, qk_nope or v_head")
    elif cfg.d_c + cfg.d_r > 1024:
        raise ValueError(f"RaggedLayer: rows of up to 1024 values, got {cfg.d_c + cfg.d_r}")


class RaggedLayer:
    """One MLA layer's step for a batch whose requests bring different numbers
    of new tokens: none, one (a decode) or a prompt's chunk.

    All new tokens lie one behind the other in ``x`` ``[n_tok, hidden]``, request
    by request; rows behind the last token are padding (``n_tok`` is the largest
    step's), so that one captured graph can serve every step.  A step builds the
    tables on the device (``mla_batch_tables``: pages for the new tokens come
    from ``free_blocks``), projects the queries, stores the new latent rows
    through their slots, attends (causally, or over a sliding window and a few
    first rows) and projects the output.  ``cache.block_table`` is extended in
    place.  ``window`` = 0: all rows up to the token's own.  bf16 (with a bf16 or
    FP8 cache) in the tensor-core shape: 128 heads, d_c 512, d_r 64, pages of 64;
    fp32 in any shape of up to 1024 values a row.

    A request that cannot be served (its rows are more than its table holds, or
    the free pages or the token rows are used up) and all behind it wait: their
    ``seq_lens`` stays, nothing is stored for them, their rows of ``y`` mean
    nothing, and the device error word says so.  The caller takes it out (a
    ``new_lens`` of 0) and goes on.

    Pages that have left a window may be given to other requests, with any entry
    left in the table; not so with an FP8 cache, whose step expands all pages
    that the lengths cover, in time too (64 requests, window 2048: 145 us over
    4,000 rows, 379 over 16,000).

    The projections and the append take all ``n_tok`` rows, padding included: 64
    decodes cost 0.27 ms in a step of 64 rows and 1.40 in one of 1,024, so a
    server captures a graph for its decode steps beside that for prompts."""

    def __init__(self, cfg: abi.Config, weights: Dict[str, torch.Tensor], cache: abi.Cache, n_tok: int,
                 window: int = 0, n_sinks: int = 0, max_workers: int = 0):
        if window < 0 or n_sinks < 0 or max_workers < 0:
            raise ValueError("window, n_sinks and max_workers must not be negative")
        abi._need_i32(window=window, n_sinks=n_sinks, max_workers=max_workers)
        if cache.block_table.shape[0] > abi.MAX_CHUNK_BATCH:
            raise ValueError(f"at most {abi.MAX_CHUNK_BATCH} requests a step, got {cache.block_table.shape[0]}")
        _refuse_without_a_step(cfg)
        self.cfg, self.W, self.cache, self.n_tok = cfg, weights, cache, n_tok
        self.window, self.n_sinks, self.max_workers = window, n_sinks, max_workers
        dev, H = cache.pool.device, cfg.n_heads
        batch, width = cache.block_table.shape
        self.tcfg = dataclasses.replace(cfg, fixed_rows=True)    # x is laid out by new_lens
        # an FP8 cache is expanded into a bf16 scratch for the step, as in DecodeLayer
        self.dcfg, self.dcache, self.fp8_scratch = cfg, cache, None
        if cfg.fp8_cache:
            self.dcfg = dataclasses.replace(cfg, fp8_cache=False)
            self.fp8_scratch = torch.empty(abi.mla_fp8_scratch_bytes(cfg, batch, width), dtype=torch.uint8, device=dev)
            self.dcache = abi.fp8_scratch_cache(self.dcfg, self.fp8_scratch, batch, width)
        cfg = self.dcfg
        if cfg.dtype == "bf16":
            self.q = torch.empty((2 if cfg.split_query else 1) * n_tok, H, cfg.d_c + cfg.d_r, dtype=torch.bfloat16, device=dev)
        else:
            self.q = (torch.empty(n_tok, H, cfg.d_c, device=dev), torch.empty(n_tok, H, cfg.d_r, device=dev))
        i32 = dict(dtype=torch.int32, device=dev)
        self.cu_q = torch.zeros(batch + 1, **i32)
        self.seq_lens = torch.zeros(batch, **i32)
        self.seq_idx = torch.zeros(n_tok, **i32)
        self.pos = torch.zeros(n_tok, **i32)
        self.slots = torch.zeros(n_tok, dtype=torch.int64, device=dev)
        # padding rows are never written: zeros, so that their projections stay finite
        self.o_lat = torch.zeros(n_tok, H, cfg.d_c, dtype=cfg.torch_dtype, device=dev)
        self.lse = torch.zeros(n_tok, H, device=dev)
        self.y = torch.empty(n_tok, cfg.hidden, dtype=cfg.torch_dtype, device=dev)
        u8 = dict(dtype=torch.uint8, device=dev)
        self.ws_gemm = torch.empty(max(abi.mla_absorb_q_workspace_size(cfg, n_tok), abi.mla_out_proj_workspace_size(cfg, n_tok),
                                       256), **u8)
        self.ws_append = torch.empty(max(abi.mla_cache_append_workspace_size(cfg, n_tok), 256), **u8)
        self.ws_attend = torch.empty(abi.mla_chunk_workspace_size(cfg, n_tok, max_workers), **u8)
        self.side = torch.cuda.Stream(device=dev)

    def tables(self, cached_lens, new_lens, free_blocks, free_head, stream=None):
        """Tables, positions and slots of a step; ``self.seq_lens`` afterwards holds the next step's ``cached_lens``."""
        abi.mla_batch_tables(self.tcfg, cached_lens, new_lens, free_blocks, free_head, self.cache.pool.shape[0],
                             self.cache.block_table, self.cu_q, self.seq_lens, self.seq_idx, self.pos, self.slots,
                             stream=stream)

    def attend(self, stream=None):
        """Attention of the step's tokens: ``self.o_lat`` (storage dtype) and ``self.lse``."""
        if self.fp8_scratch is not None:
            abi.mla_cache_dequant_fp8(self.cfg, self.cache, self.seq_lens.shape[0], self.seq_lens, self.fp8_scratch, stream)
        args = (self.o_lat, self.ws_attend, self.lse, self.max_workers, stream)
        if self.window:
            abi.mla_window_attention(self.dcfg, self.q, self.cu_q, self.dcache, self.seq_lens, self.window, self.n_sinks, *args)
        else:
            abi.mla_chunk_attention(self.dcfg, self.q, self.cu_q, self.dcache, self.seq_lens, *args)

    def step(self, x, cached_lens, new_lens, free_blocks, free_head, stream=None) -> torch.Tensor:
        """One step on device tensors: ``y`` ``[n_tok, hidden]`` (a reused buffer; padding rows mean nothing).
        ``free_head`` moves on in place; pass ``self.seq_lens`` as the next step's ``cached_lens``."""
        W, cfg = self.W, self.dcfg
        W_DQ, W_UQ, W_UK = W.get("W_DQ"), W["W_UQ"] if "W_UQ" in W else W["W_Q"], W["W_UK"]
        W_DKV, W_KR, W_UV, W_O = W["W_DKV"], W["W_KR"], W["W_UV"], W["W_O"]
        # the tables change the caller's state: what the later calls would refuse is refused ahead of them
        abi._need(x, "x", cfg.torch_dtype, shape=(self.n_tok, cfg.hidden))
        abi._need_here(x, self.cache.pool)
        if cfg.dtype == "bf16" and x.data_ptr() % 16:
            raise ValueError("x must start on a 16-byte boundary")
        main = stream or torch.cuda.current_stream()
        self.tables(cached_lens, new_lens, free_blocks, free_head, main)
        ready = torch.cuda.Event()
        ready.record(main)
        if cfg.dtype == "bf16":
            abi.mla_absorb_q_packed(cfg, x, W_DQ, W_UQ, W_UK, self.pos, self.q, self.ws_gemm, main)
        else:
            abi.mla_absorb_q(cfg, x, W_DQ, W_UQ, W_UK, self.pos, *self.q, self.ws_gemm, main)
        # the new rows on a second stream beside the query projections
        self.side.wait_event(ready)
        abi.mla_cache_append_slots(self.cfg, x, W_DKV, W_KR, self.pos, self.slots, self.cache, self.ws_append, self.side)
        done = torch.cuda.Event()
        done.record(self.side)
        main.wait_event(done)
        x.record_stream(self.side)
        self.attend(main)
        abi.mla_out_proj_stored(cfg, self.o_lat, W_UV, W_O, self.y, self.ws_gemm, main)
        return self.y

    def capture_step(self, x, cached_lens, new_lens, free_blocks, free_head) -> torch.cuda.CUDAGraph:
        """Record one ``step`` on these device buffers as a CUDA graph.  Refill ``x``, ``cached_lens`` and
        ``new_lens`` in place between replays (``free_head`` moves on by itself); ``self.y`` holds the result.
        The kernels' one-time setup is done first by a step without new tokens, which changes nothing."""
        none = torch.zeros_like(new_lens)
        self.step(x, cached_lens, none, free_blocks, free_head)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step(x, cached_lens, new_lens, free_blocks, free_head)
        return graph
