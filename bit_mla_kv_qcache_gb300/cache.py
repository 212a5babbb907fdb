"""Device buffers of one layer's low-bit dual-path MLA cache and the calls that use them.

PyTorch only allocates device memory and provides the stream; the writer and the decode
attention run in libmla_qcache.so.
"""
from __future__ import annotations

import torch

from . import binding


class QuantizedMLACache:
    """Page pool, BF16 sink/recent buffers, page table and lengths for B sequences.

    The page table is the caller's (a paged allocator maps positions to physical pages);
    by default sequence b owns pages [b*max_pages, (b+1)*max_pages).
    """

    def __init__(self, cfg: binding.Config, batch: int, max_pages: int, n_pages: int | None = None,
                 page_table: torch.Tensor | None = None, device="cuda"):
        self.cfg = cfg
        self.B = batch
        self.max_pages = max_pages
        self.n_pages = n_pages if n_pages is not None else batch * max_pages
        dev = torch.device(device)
        pb = binding.page_bytes(cfg)
        if pb == 0:
            raise binding.QCacheError(f"unsupported configuration {cfg}")
        self.pool = torch.zeros((self.n_pages, pb), dtype=torch.uint8, device=dev)
        self.sink = torch.zeros((batch, cfg.n_sink, 576), dtype=torch.int16, device=dev)
        self.ring = torch.zeros((batch, cfg.n_recent, 576), dtype=torch.int16, device=dev)
        if page_table is None:
            page_table = torch.arange(batch * max_pages, dtype=torch.int32, device=dev).view(batch, max_pages)
        self.page_table = page_table.to(device=dev, dtype=torch.int32).contiguous()
        self.seq_lens = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)
        self._ws = None
        self._ws_need = {}  # workspace bytes per head count
        self._lens_alt = None  # second length array for write_advance

    def write(self, c_new: torch.Tensor, kr_new: torch.Tensor, cu_new: torch.Tensor, max_new: int,
              advance: bool = True, stream=None) -> None:
        """Append rows cu_new[b]..cu_new[b+1]-1 to sequence b (BF16 c [N,512], k_R [N,64])."""
        binding.mla_qcache_write(self.cfg, c_new, kr_new, cu_new, self.seq_lens, max_new, self.page_table, self.pool,
                                 self.sink, self.ring, self.err, stream)
        if advance:
            binding.mla_qcache_advance(cu_new, self.seq_lens, stream)

    def write_advance(self, c_new: torch.Tensor, kr_new: torch.Tensor, cu_new: torch.Tensor, max_new: int,
                      stream=None) -> None:
        """write() with the length update in the same launch: the new lengths are stored into a
        second array, which then becomes ``self.seq_lens`` (the two arrays alternate)."""
        if self._lens_alt is None:
            self._lens_alt = torch.empty_like(self.seq_lens)
        binding.mla_qcache_write_advance(self.cfg, c_new, kr_new, cu_new, self.seq_lens, self._lens_alt, max_new,
                                         self.page_table, self.pool, self.sink, self.ring, self.err, stream)
        self.seq_lens, self._lens_alt = self._lens_alt, self.seq_lens

    def workspace(self, heads: int) -> torch.Tensor:
        need = self._ws_need.get(heads)
        if need is None:
            need = self._ws_need[heads] = binding.workspace_bytes(self.cfg, self.B, heads, self.max_pages)
        if self._ws is None or self._ws.numel() < need:
            # zeroed once: the decode keeps the merge counters at its start zero between calls
            self._ws = torch.zeros(max(need, 16), dtype=torch.uint8, device=self.pool.device)
        return self._ws

    def decode(self, q_lat: torch.Tensor, q_rope: torch.Tensor, softmax_scale: float, out=None, lse=None,
               stream=None):
        """Attention readout O [B,H,512] (float32) and LSE [B,H] for one decode step."""
        B, H = q_lat.shape[0], q_lat.shape[1]
        if out is None:
            out = torch.empty((B, H, 512), dtype=torch.float32, device=q_lat.device)
        if lse is None:
            lse = torch.empty((B, H), dtype=torch.float32, device=q_lat.device)
        binding.mla_qcache_decode_attn(self.cfg, q_lat, q_rope, self.page_table, self.seq_lens, self.pool, self.sink,
                                       self.ring, softmax_scale, out, lse, self.workspace(H), self.err, stream)
        return out, lse

    def error_bits(self) -> int:
        return int(self.err.item())


class KV4Cache:
    """Grouped-query K/V cache in 4 bits of one layer: page pool, page table and lengths for B sequences, and the
    workspaces of its attention. The page table is the caller's, as for QuantizedMLACache. The lengths must not change under
    a call that reads them: appends and attend() are ordered by their stream or, on several, by the caller."""

    def __init__(self, cfg: binding.KV4Config, batch: int, max_pages: int, n_pages: int | None = None,
                 page_table: torch.Tensor | None = None, device="cuda"):
        pb = binding.kv4_page_bytes(cfg)
        if pb == 0:
            raise binding.QCacheError("unsupported 4-bit cache configuration")
        self.cfg, self.B, self.max_pages = cfg, batch, max_pages
        self.n_pages = n_pages if n_pages is not None else batch * max_pages
        dev = torch.device(device)
        self.pool = torch.zeros((self.n_pages, pb), dtype=torch.uint8, device=dev)
        if page_table is None:
            page_table = torch.arange(batch * max_pages, dtype=torch.int32, device=dev).view(batch, max_pages)
        self.page_table = page_table.to(device=dev, dtype=torch.int32).contiguous()
        self.seq_lens = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)
        self.tree_base = torch.zeros(batch, dtype=torch.int32, device=dev)  # tokens before the tree of drafted ones
        self._trees = False  # start_tree() has been called: tree_base says something
        self._ws = {}  # per stream
        self._ws_need = {}  # workspace bytes per head count and rows

    def append(self, k: torch.Tensor, v: torch.Tensor, cu_new: torch.Tensor, max_new: int, stream=None, **kw) -> None:
        """Appends rows cu_new[b]..cu_new[b+1]-1 of k, v [N,Hkv,D] to sequence b and advances ``self.seq_lens`` in place,
        by a launch behind it: a captured append goes on from there at every replay, among calls that are not captured
        too. Further arguments (cos, sin, interleaved, q, q_out, k_deq, v_deq) as for mla_qcache_kv4_append. With tree_mask the rows
        are nodes of the trees that start_tree() began (or, where a tree_base is given, of trees that begin there)."""
        if kw.get("tree_mask") is not None and "tree_base" not in kw:
            kw["tree_base"] = self._base("append() of nodes")
        binding.mla_qcache_kv4_append(self.cfg, k, v, cu_new, self.seq_lens, max_new, self.page_table, self.pool, self.err,
                                      seq_lens_next=self.seq_lens, stream=stream, **kw)

    def workspace(self, heads: int, max_q: int, stream=None) -> torch.Tensor:
        """Workspace of attend() on a stream (None: the current one), allocated and zeroed there. Each stream has one, so
        that calls on two may overlap. A call that is being captured gets one of its own in the graph's memory, zeroed at
        each replay: a graph holds nothing that this object replaces later, and shares nothing with other calls."""
        need = self._ws_need.get((heads, max_q))
        if need is None:
            need = self._ws_need[heads, max_q] = binding.kv4_workspace_bytes(self.cfg, self.B, heads, max_q, self.max_pages)
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.workspace(heads, max_q)
        device = self.pool.device
        if torch.cuda.is_current_stream_capturing():
            ws = torch.empty(max(need, 16), dtype=torch.uint8, device=device)
            ws[:binding.KV4_COUNTER_BYTES].zero_()
            return ws
        at = torch.cuda.current_stream(device).cuda_stream
        ws = self._ws.get(at)
        if ws is None or ws.numel() < need:
            # zeroed once: the attention keeps the counters at its start zero between calls
            ws = self._ws[at] = torch.zeros(max(need, 16), dtype=torch.uint8, device=device)
        return ws

    def attend(self, q: torch.Tensor, softmax_scale: float, cu_q: torch.Tensor | None = None, max_q: int = 1, out=None,
               lse=None, causal: bool = True, window: int = 0, stream=None, tree_mask: torch.Tensor | None = None):
        """Attention of query rows q [N,Hq,D], the last positions of their sequences, over the cache: out in q's type. With
        tree_mask ([N] or [N, words] int64) the rows are nodes of the trees that start_tree() began: each sees the tokens before its
        tree and the nodes that its mask names. A window cuts the tokens before the tree alone, by the node's depth: for rows deeper
        than the window, give masks of the last `window` nodes of their paths here (append() takes the whole paths)."""
        if tree_mask is not None and not causal:
            raise ValueError("nodes of a tree see what their masks name: causal=False has no meaning for them")
        base = None if tree_mask is None else self._base("attend() of nodes")
        if out is None:
            with torch.cuda.stream(stream):  # memory that this stream may write at once (None: the current one)
                out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
            if stream is not None:
                out.record_stream(torch.cuda.current_stream(q.device))
        if tree_mask is not None:
            binding.mla_qcache_kv4_attn_tree(self.cfg, q, tree_mask, cu_q, max_q, self.page_table, self.seq_lens, self.pool, softmax_scale,
                                             out, self.workspace(q.shape[1], max_q, stream), self.err, tree_base=base, lse=lse,
                                             window=window, stream=stream)
            return out
        binding.mla_qcache_kv4_attn(self.cfg, q, self.page_table, self.seq_lens, self.pool, softmax_scale, out,
                                    self.workspace(q.shape[1], max_q, stream), self.err, cu_q=cu_q, max_q=max_q, lse=lse,
                                    causal=causal, window=window, stream=stream)
        return out

    def start_tree(self, stream=None) -> None:
        """Trees of drafted tokens begin behind the tokens that the sequences hold now: rows with a tree_mask, in append() and
        attend(), are nodes of these trees until keep()."""
        with torch.cuda.stream(stream):
            self.tree_base.copy_(self.seq_lens)
        self._trees = True

    def _base(self, what: str) -> torch.Tensor:
        if not self._trees:
            raise binding.QCacheError(f"{what} needs start_tree() before it: nothing says where the trees begin")
        return self.tree_base

    def keep(self, kept: torch.Tensor, n_kept: torch.Tensor, stream=None) -> None:
        """Of each tree the nodes kept [B, most] (n_kept [B] of them, as mla_qcache_verify_sampled and _greedy give them) stay, moved to the
        places behind the tokens before the tree; ``self.seq_lens`` becomes their end."""
        binding.mla_qcache_kv4_keep(self.cfg, kept, n_kept, self._base("keep()"), self.page_table, self.pool, self.seq_lens, self.err, stream)

    def error_bits(self) -> int:
        return int(self.err.item())
