"""One verify step on the device: buffers plus the four C-ABI calls.

``VerifyStep`` owns the device buffers for a fixed geometry (torch is used
for allocation and streams only) and issues, on one stream and with no host
synchronisation, the calls of ``include/jsv.h`` in order: tree attention,
LM head + argmax, and the accept walk with the KV compaction (one launch,
``jsv_accept_compact``; the separate ``jsv_accept_path`` and
``jsv_kv_compact`` are kept as methods too).

``run_host`` is the end-to-end form: it copies the step's per-step inputs
from pinned host memory, runs the step, and copies the accepted paths back.
The per-step inputs (tree arrays, tokens, q, hidden) live in one device
arena and the outputs (paths, lengths) in another, each mirrored by one
pinned host buffer, so each direction is a single copy.

``capture`` records the step's calls once into a CUDA graph (the engine the
JetSpec README describes replays CUDA graphs for wall-clock latency); every
kernel is launched with programmatic dependent launch, so the graph keeps
those overlapping edges.  ``replay`` launches the whole step in one call;
``capture_host`` / ``replay_host`` do the same for the end-to-end form,
copies included.
"""
from __future__ import annotations

import numpy as np
import torch

from . import jsv


def _i32(x, device):
    return torch.as_tensor(np.ascontiguousarray(x, dtype=np.int32)).to(device)


def _on(stream):
    """Torch's current stream for a while: a torch stream, a raw handle (0: the
    default stream), or None for the one that is current already."""
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _bf16(bits, device):
    t = torch.from_numpy(np.ascontiguousarray(bits, dtype=np.uint16).view(np.int16))
    return t.view(torch.bfloat16).to(device)


class _Arena:
    """Named arrays packed at 256-byte offsets in one device buffer, with a
    pinned host mirror; ``dev[name]`` / ``host[name]`` are typed views."""

    def __init__(self, fields, device):
        # fields: name -> (shape, torch dtype)
        self.layout, off = {}, 0
        for name, (shape, dtype) in fields.items():
            n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
            self.layout[name] = (off, n, shape, dtype)
            off += (n + 255) // 256 * 256
        self.nbytes = max(off, 256)
        self.dev_buf = torch.zeros(self.nbytes, dtype=torch.uint8, device=device)
        self.host_buf = torch.zeros(self.nbytes, dtype=torch.uint8).pin_memory()
        self.dev = {k: self._view(self.dev_buf, k) for k in self.layout}
        self.host = {k: self._view(self.host_buf, k) for k in self.layout}

    def _view(self, buf, name):
        off, n, shape, dtype = self.layout[name]
        return buf[off:off + n].view(dtype).view(shape)


class VerifyStep:
    """Device state for one verify step of a workload (see ``synth.Workload``)."""

    def __init__(self, wl, tokens, device="cuda", max_path=None):
        dev = torch.device(device)
        self.device = dev
        self.B, self.Hq, self.Hkv, self.D = wl.B, wl.Hq, wl.Hkv, wl.D
        self.T, self.d, self.V = wl.T, wl.d, wl.V
        self.scale = wl.scale
        self.max_path = int(max_path or wl.max_nodes)
        # per-step inputs in one arena (filled once here from the workload)
        inputs = {"page_table": np.ascontiguousarray(wl.page_table, dtype=np.int32),
                  "prefix_len": np.ascontiguousarray(wl.prefix_len, dtype=np.int32),
                  "node_offsets": np.ascontiguousarray(wl.node_offsets, dtype=np.int32),
                  "parent": np.ascontiguousarray(wl.parent, dtype=np.int32),
                  "tokens": np.ascontiguousarray(tokens, dtype=np.int32),
                  "q": np.ascontiguousarray(wl.q, dtype=np.uint16),
                  "hidden": np.ascontiguousarray(wl.hidden, dtype=np.uint16)}
        self._in = _Arena({k: (v.shape, torch.int32 if v.dtype == np.int32 else torch.bfloat16)
                           for k, v in inputs.items()}, dev)
        for k, v in inputs.items():
            hv = self._in.host[k]
            if v.dtype == np.int32:
                hv.copy_(torch.from_numpy(v))
            else:
                hv.view(torch.int16).copy_(torch.from_numpy(v.view(np.int16)))
        self._in.dev_buf.copy_(self._in.host_buf)
        for k, t in self._in.dev.items():
            setattr(self, k, t)
        self.k_cache = _bf16(wl.k_cache, dev)
        self.v_cache = _bf16(wl.v_cache, dev)
        self.w = _bf16(wl.w, dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.out = torch.empty((self.T, self.Hq, self.D), dtype=torch.bfloat16, device=dev)
        self.argmax = torch.empty(self.T, dtype=torch.int32, device=dev)
        self.max_logit = torch.empty(self.T, dtype=torch.float32, device=dev)
        # per-step outputs in one arena
        self._out = _Arena({"path": ((self.B, self.max_path), torch.int32), "accept_len": ((self.B,), torch.int32),
                            "bonus": ((self.B,), torch.int32), "new_len": ((self.B,), torch.int32)}, dev)
        for k, t in self._out.dev.items():
            setattr(self, k, t)
        self.batch = jsv.make_batch(
            B=self.B, Hq=self.Hq, Hkv=self.Hkv, D=self.D,
            max_pages_per_req=wl.page_table.shape[1], num_pages=wl.num_pages,
            total_nodes=self.T, max_nodes=wl.max_nodes, max_prefix=wl.max_prefix,
            page_table=self.page_table, prefix_len=self.prefix_len,
            node_offsets=self.node_offsets, parent=self.parent, dev_status=self.status)
        aws = jsv.jsv_tree_attention_workspace_size(self.batch)
        lws = jsv.jsv_lmhead_argmax_workspace_size(self.T, self.d, self.V)
        self.attn_ws = torch.zeros(max(aws, 256), dtype=torch.uint8, device=dev)   # any contents: every call writes what it reads
        self.lm_ws = torch.zeros(max(lws, 8), dtype=torch.uint8, device=dev)   # zeroed once; each call leaves it zeroed
        self._graph = None
        self._host_graph = None

    # -- the four calls -----------------------------------------------------
    def attention(self, stream=None):
        jsv.jsv_tree_attention(self.batch, self.q, self.k_cache, self.v_cache, self.scale,
                               self.out, self.attn_ws, stream=stream)

    def lmhead(self, stream=None):
        jsv.jsv_lmhead_argmax(self.hidden, self.w, self.T, self.d, self.V, self.argmax,
                              self.max_logit, self.lm_ws, dev_status=self.status, stream=stream)

    def accept(self, stream=None):
        jsv.jsv_accept_path(self.batch, self.tokens, self.argmax, self.max_path, self.path,
                            self.accept_len, self.bonus, stream=stream)

    def compact(self, stream=None):
        jsv.jsv_kv_compact(self.batch, self.k_cache, self.v_cache, self.path, self.max_path,
                           self.accept_len, self.new_len, stream=stream)

    def accept_compact(self, stream=None):
        """The walk and the compaction in one launch (same results as
        ``accept`` followed by ``compact``)."""
        jsv.jsv_accept_compact(self.batch, self.tokens, self.argmax, self.max_path, self.path,
                               self.accept_len, self.bonus, self.k_cache, self.v_cache, self.new_len,
                               stream=stream)

    def run(self, stream=None):
        """One verify step on one stream, no host sync: tree attention, LM head
        + argmax, then the accept walk fused with the KV compaction."""
        self.attention(stream)
        self.lmhead(stream)
        self.accept_compact(stream)

    # -- CUDA graph -----------------------------------------------------------
    def capture(self):
        """Record one verify step into a CUDA graph on a side stream.

        One eager step runs first so that every one-time host set-up (kernel
        attributes, tensor-map entry point) happens outside the capture; it
        executes the step, so callers that need pristine caches restore them
        before replaying."""
        self.run()
        torch.cuda.synchronize(self.device)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.run()
        torch.cuda.synchronize(self.device)
        self._graph = graph
        return graph

    def replay(self):
        """One verify step through the captured graph (same buffers)."""
        self._graph.replay()

    # -- end-to-end form ----------------------------------------------------
    def host_inputs(self):
        """Pinned host views of the per-step inputs (tree arrays, tokens, q,
        hidden); ``run_host`` copies all of them in one transfer."""
        return self._in.host

    def h2d_bytes(self) -> int:
        return self._in.nbytes

    def d2h_bytes(self) -> int:
        return self._out.nbytes

    def run_host(self, stream=None):
        """Copy the input arena host->device, run the step, copy the output
        arena back (one copy each way), all on ``stream``; returns pinned host
        views of path, accept_len, bonus and new_len."""
        with _on(stream):
            self._in.dev_buf.copy_(self._in.host_buf, non_blocking=True)
            self.run(stream)
            self._out.host_buf.copy_(self._out.dev_buf, non_blocking=True)
        return self._out.host

    def capture_host(self):
        """Record the end-to-end step (the input arena's copy up from pinned
        host memory, the step's calls, the output arena's copy back) into one
        CUDA graph, so that ``replay_host`` issues all of it with one launch.
        The graph's copies read and write the pinned buffers when it runs:
        the caller fills ``host_inputs()`` before each replay and reads the
        returned views after synchronising.  One eager ``run_host`` runs
        first (one-time host set-up outside the capture)."""
        self.run_host()
        torch.cuda.synchronize(self.device)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.run_host()
        torch.cuda.synchronize(self.device)
        self._host_graph = graph
        return graph

    def replay_host(self):
        """One end-to-end step through the graph of ``capture_host``; returns
        the pinned host views of path, accept_len, bonus and new_len (filled
        once the current stream has been synchronised)."""
        self._host_graph.replay()
        return self._out.host


class VerifyStepKv8(VerifyStep):
    """The verify step over a prefix held in 8 bits, with its pages managed on
    the device.

    The full pages of every prefix are quantised once at the start and their
    bf16 pages freed; ``run`` (and ``capture`` / ``replay``, ``run_host``) is
    then the base class's step with ``jsv_tree_attention_kv8``.  ``advance``
    follows a step: the pages that the accepted tokens filled are written to
    the 8-bit cache, what the bf16 table no longer needs is freed, and pages
    for the next tree are mapped, all on the stream, so that the caller only
    writes the next tree's K/V and runs again.  A prefix may grow by as much as
    the page table's row holds, or to ``max_prefix`` where that is given (a
    longer one is flagged): the attention shares out a request by that bound,
    and where prefixes stay far below it the splits are too few (64 nodes over
    2048 tokens: 23 us by their own bound, 29 by four times that).

    The caches of this class are the workload's whole bf16 pool and an 8-bit
    pool for full rows beside it.  What the 8-bit prefix saves are the bf16
    pages that it frees in the pool, for other rows to take.

    The page tables, the prefix lengths and the trees' sizes live on the device,
    where ``advance`` turns them over; ``host_inputs`` has the others (parent,
    tokens, q, hidden).  Trees of other sizes (as many nodes in all) are
    announced to ``advance``, which maps their pages.
    """

    def __init__(self, wl, tokens, fmt="e4m3", device="cuda", max_path=None, max_prefix=None):
        width = wl.page_table.shape[1]
        if max_prefix is None:
            max_prefix = width * 16 - 1
        if not wl.max_prefix <= max_prefix < width * 16:
            raise ValueError(f"max_prefix {max_prefix}: not from the longest prefix, {wl.max_prefix}, to below the "
                             f"{width * 16} slots of a row")
        super().__init__(wl, tokens, device, max_path)
        dev, B = self.device, self.B
        self.width = width
        self.batch = jsv.make_batch(
            B=B, Hq=self.Hq, Hkv=self.Hkv, D=self.D, max_pages_per_req=width, num_pages=wl.num_pages,
            total_nodes=self.T, max_nodes=wl.max_nodes, max_prefix=max_prefix, page_table=self.page_table,
            prefix_len=self.prefix_len, node_offsets=self.node_offsets, parent=self.parent, dev_status=self.status)
        pages8 = B * width
        self.k8, self.v8 = (torch.zeros((pages8, self.Hkv, 16, self.D), dtype=torch.uint8, device=dev) for _ in range(2))
        self.k_scale, self.v_scale = (torch.zeros((pages8, self.Hkv), device=dev) for _ in range(2))
        self.page_table8 = torch.full((B, width), -1, dtype=torch.int32, device=dev)
        self.cache8 = jsv.make_kv8(format=fmt, num_pages=pages8, max_pages_per_req=width, k=self.k8, v=self.v8,
                                   k_scale=self.k_scale, v_scale=self.v_scale, page_table=self.page_table8)
        held = wl.page_table[wl.page_table >= 0]
        self.refcount = _i32(np.bincount(held, minlength=wl.num_pages), dev)
        self.refcount8 = torch.zeros(pages8, dtype=torch.int32, device=dev)
        self.pool = jsv.make_page_pool(num_pages=wl.num_pages, refcount=self.refcount, dev_status=self.status)
        self.pool8 = jsv.make_page_pool(num_pages=pages8, refcount=self.refcount8, dev_status=self.status)
        self.nodes = self.node_offsets[1:] - self.node_offsets[:-1]
        self.tree_end = torch.empty_like(self.prefix_len)
        self.pages_ws = torch.empty(max(jsv.jsv_pages_workspace_size(n, B) for n in (wl.num_pages, pages8)),
                                    dtype=torch.uint8, device=dev)
        self.attn_ws = torch.empty(max(jsv.jsv_tree_attention_kv8_workspace_size(self.batch, self.cache8), 256),
                                   dtype=torch.uint8, device=dev)
        torch.add(self.prefix_len, self.nodes, out=self.tree_end)
        self._write_full_pages(None, self.prefix_len, None)
        jsv.jsv_pages_trim(self.pool, self.page_table, B, width, self.prefix_len, self.tree_end)

    def _write_full_pages(self, from_len, to_len, stream):
        jsv.jsv_pages_alloc(self.pool8, self.page_table8, self.B, self.width, None, to_len, True, self.pages_ws,
                            stream=stream)
        jsv.jsv_kv8_quantize(self.batch, self.cache8, self.k_cache, self.v_cache, from_len, to_len, stream=stream)

    def attention(self, stream=None):
        jsv.jsv_tree_attention_kv8(self.batch, self.cache8, self.q, self.k_cache, self.v_cache, self.scale, self.out,
                                   self.attn_ws, stream=stream)

    def advance(self, stream=None, node_offsets=None):
        """The turn to the next step: ``prefix_len`` becomes ``new_len``.
        ``stream``: the one the step ran on, or None for the current one.
        ``node_offsets``: where the next trees' sizes differ, their [B + 1]
        offsets, on the host (checked here) or on the device (checked by the
        next step's kernels)."""
        if node_offsets is not None:
            node_offsets = self._checked_offsets(node_offsets)
        with _on(stream):
            self._write_full_pages(self.prefix_len, self.new_len, stream)
            if node_offsets is not None:
                self.node_offsets.copy_(node_offsets, non_blocking=True)
                torch.sub(self.node_offsets[1:], self.node_offsets[:-1], out=self.nodes)
            jsv.jsv_pages_trim(self.pool, self.page_table, self.B, self.width, self.new_len, self.new_len,
                               stream=stream)
            self.prefix_len.copy_(self.new_len)
            torch.add(self.new_len, self.nodes, out=self.tree_end)
            jsv.jsv_pages_alloc(self.pool, self.page_table, self.B, self.width, self.new_len, self.tree_end, False,
                                self.pages_ws, stream=stream)

    def _checked_offsets(self, offs):
        if isinstance(offs, torch.Tensor) and offs.is_cuda:
            if offs.shape != (self.B + 1,):
                raise ValueError(f"node_offsets: shape {tuple(offs.shape)}, not ({self.B + 1},)")
            return offs
        offs = np.ascontiguousarray(offs, dtype=np.int32)
        if offs.shape != (self.B + 1,):
            raise ValueError(f"node_offsets: shape {offs.shape}, not ({self.B + 1},)")
        n = np.diff(offs)
        if offs[0] != 0 or offs[-1] != self.T or n.min() < 1 or n.max() > self.batch.max_nodes:
            raise ValueError(f"node_offsets: not {self.B} trees of 1 to {self.batch.max_nodes} nodes, {self.T} in all")
        return torch.from_numpy(offs)

    # -- end-to-end form: what follows the tables, lengths and sizes is copied --
    def _copied(self) -> int:
        return self._in.layout["parent"][0]

    def host_inputs(self):
        at = self._copied()
        return {k: v for k, v in self._in.host.items() if self._in.layout[k][0] >= at}

    def run_host(self, stream=None):
        """As the base class's; copies what ``host_inputs`` has."""
        at = self._copied()
        with _on(stream):
            self._in.dev_buf[at:].copy_(self._in.host_buf[at:], non_blocking=True)
            self.run(stream)
            self._out.host_buf.copy_(self._out.dev_buf, non_blocking=True)
        return self._out.host

    def h2d_bytes(self) -> int:
        return self._in.nbytes - self._copied()
