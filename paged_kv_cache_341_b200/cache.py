"""A paged KV cache for one attention layer and its decode step.

``PagedKVCache`` owns the host block pool (library pool, FIFO + refcounts),
the host block tables and lengths of a batch of sequences (one row each), and
the device K/V caches ``[num_blocks, block_size, Hkv, D]``.  ``decode_step``
is one pass of the hot path through the C ABI:

1. host: reserve one slot per appending sequence (fresh block at offset 0,
   copy-on-write of a shared partly filled block) -- ``pa_reserve_slots``;
2. device: copy the blocks named by the copy-on-write pairs -- ``pa_copy_blocks``;
3. device: write the new tokens' K/V into their slots -- ``pa_append_kv``;
4. device: single-query attention over every sequence's blocks --
   ``pa_decode_attention`` (split into partitions plus a merge when
   ``partition_size`` > 0).

``prefill_step`` does the same for a chunk of new tokens per sequence (a prompt,
or a piece of one), with rotary positions fused into the append when asked for,
and ``compact`` moves the live blocks to the front of the pool.

Host-to-device traffic of a step is one small transfer: the slot mapping, the
lengths, the table entries the reservation changed (at most one per row) and
the copy pairs, plus whatever the caller passes from host memory.  The whole
tables go over once, with ``upload_tables``.
"""

import ctypes
import math

import numpy as np
import torch

from . import pa


class PagedKVCache:
    def __init__(self, num_blocks, block_size, num_kv_heads, head_dim, dtype, num_seqs, max_blocks_per_seq,
                 device="cuda", initial_free_order=None, fill=None):
        self.num_blocks = int(num_blocks)
        self.block_size = int(block_size)
        self.num_kv_heads = int(num_kv_heads)
        self.head_dim = int(head_dim)
        self.dtype = dtype
        self.device = torch.device(device)
        self.pool = pa.Pool(self.num_blocks, self.block_size, initial_free_order)
        shape = (self.num_blocks, self.block_size, self.num_kv_heads, self.head_dim)
        if fill is None:
            self.k_cache = torch.empty(shape, dtype=dtype, device=self.device)
            self.v_cache = torch.empty(shape, dtype=dtype, device=self.device)
        else:
            self.k_cache = torch.full(shape, fill, dtype=dtype, device=self.device)
            self.v_cache = torch.full(shape, fill, dtype=dtype, device=self.device)
        self.max_blocks = int(max_blocks_per_seq)
        self.tables = np.full((num_seqs, self.max_blocks), -1, np.int32)
        self.lens = np.zeros(num_seqs, np.int32)
        # pinned staging for the per-step host -> device copies
        self._h_tables = torch.empty((num_seqs, self.max_blocks), dtype=torch.int32).pin_memory()
        self._h_lens = torch.empty(num_seqs, dtype=torch.int32).pin_memory()
        self._h_slots = torch.empty(num_seqs, dtype=torch.int64).pin_memory()
        self._h_pairs = torch.empty((max(num_seqs, 1), 2), dtype=torch.int32).pin_memory()
        self.d_tables = torch.empty((num_seqs, self.max_blocks), dtype=torch.int32, device=self.device)
        self.d_lens = torch.empty(num_seqs, dtype=torch.int32, device=self.device)
        self.d_slots = torch.empty(num_seqs, dtype=torch.int64, device=self.device)
        self.d_pairs = torch.empty((max(num_seqs, 1), 2), dtype=torch.int32, device=self.device)
        self._staged = None               # event: last copies out of the pinned staging buffers
        # per-step metadata, double-buffered: [slots int64 S][lens int32 S][updates int32 S x 3][pairs int32 S x 2]
        n = max(num_seqs, 1)
        self._meta_bytes = 8 * n + 4 * n + 12 * n + 8 * n
        self._meta_host = [torch.empty(self._meta_bytes, dtype=torch.uint8).pin_memory() for _ in range(2)]
        self._meta_dev = [torch.empty(self._meta_bytes, dtype=torch.uint8, device=self.device) for _ in range(2)]
        self._meta_done = [None, None]    # event: the H2D out of host slot b has finished
        self._meta_views = [self._views(self._meta_host[b]) for b in range(2)]
        self._meta_dviews = [self._views(self._meta_dev[b]) for b in range(2)]
        self._step = 0
        # metadata of chunk steps, double-buffered and grown on demand
        self._chunk = 0
        self._chunk_host, self._chunk_done = [None, None], [None, None]

    @property
    def num_seqs(self):
        return self.lens.size

    @property
    def step_metadata_bytes(self):
        """Bytes ``decode_step`` sends host -> device besides the caller's tensors."""
        return self._meta_bytes

    def _views(self, buf):
        n = max(self.lens.size, 1)
        o = 0
        slots = buf[o:o + 8 * n].view(torch.int64)
        o += 8 * n
        lens = buf[o:o + 4 * n].view(torch.int32)
        o += 4 * n
        upd = buf[o:o + 12 * n].view(torch.int32).view(n, 3)
        o += 12 * n
        pairs = buf[o:o + 8 * n].view(torch.int32).view(n, 2)
        return slots, lens, upd, pairs

    # ---------------------------------------------------------------- host side

    def allocate(self, row, num_tokens):
        """Give row ``row`` (empty) blocks for ``num_tokens`` tokens, front of the free list first."""
        need = -(-int(num_tokens) // self.block_size)
        ids = self.pool.pa_pool_alloc(need)
        self.tables[row, :need] = ids
        self.lens[row] = num_tokens
        return ids

    def share(self, src_row, dst_row):
        """Row ``dst_row`` becomes a sharer of all of ``src_row``'s blocks (fork)."""
        n = -(-int(self.lens[src_row]) // self.block_size)
        self.pool.pa_pool_fork(self.tables[src_row, :n])
        self.tables[dst_row] = self.tables[src_row]
        self.lens[dst_row] = self.lens[src_row]

    def release(self, row):
        n = -(-int(self.lens[row]) // self.block_size)
        self.pool.pa_pool_free(self.tables[row, :n])
        self.tables[row] = -1
        self.lens[row] = 0

    def reserve(self, rows=None):
        """Reserve one slot in each of ``rows`` (a contiguous range ``slice`` or None = all).

        Works in place on the host tables and lengths (a row range of a
        C-contiguous array is itself contiguous).
        """
        rows = slice(None) if rows is None else rows
        tables = self.tables[rows]
        lens = self.lens[rows]
        assert tables.flags.c_contiguous and lens.flags.c_contiguous
        return self.pool.pa_reserve_slots(tables, lens)

    def _wait_staging(self):
        # the pinned buffers may still be read by an earlier asynchronous copy
        if self._staged is not None:
            self._staged.synchronize()

    def _mark_staging(self, stream):
        self._staged = torch.cuda.Event()
        self._staged.record(stream)

    def upload_tables(self, stream=None):
        """Block tables and lengths to the device (pinned, asynchronous on ``stream``)."""
        stream = stream or torch.cuda.current_stream()
        self._wait_staging()
        self._h_tables.numpy()[:] = self.tables
        self._h_lens.numpy()[:] = self.lens
        with torch.cuda.stream(stream):
            self.d_tables.copy_(self._h_tables, non_blocking=True)
            self.d_lens.copy_(self._h_lens, non_blocking=True)
        self._mark_staging(stream)

    # ------------------------------------------------------------- device side

    def append(self, k_new, v_new, slot_mapping, stream=None):
        pa.pa_append_kv(k_new, v_new, slot_mapping, self.k_cache, self.v_cache, stream=stream)

    def copy_blocks(self, pairs, stream=None):
        if pairs.numel():
            pa.pa_copy_blocks(self.k_cache, self.v_cache, pairs, stream=stream)

    def attend(self, q, out, scale, partition_size=0, workspace=None, tables=None, lens=None, stream=None):
        pa.pa_decode_attention(q, self.k_cache, self.v_cache, self.d_tables if tables is None else tables,
                               self.d_lens if lens is None else lens, scale, out, partition_size=partition_size,
                               workspace=workspace, stream=stream)

    def decode_step(self, q, k_new, v_new, out, scale, partition_size=0, workspace=None, rows=None, stream=None):
        """One decode step for ``rows`` (default all): reserve, copy-on-write, append, attend.

        ``q``/``out`` cover the rows ([B, Hq, D]); ``k_new``/``v_new`` hold one
        token per row ([B, Hkv, D]); all are CUDA tensors.  The host
        reservation changes at most one table entry per row; those entries,
        the slot mapping, the lengths and the copy pairs go to the device in
        one small transfer, and ``pa_update_block_tables`` applies the entries
        (the device tables must have been uploaded once with
        ``upload_tables``).  Returns the host slot mapping and copy pairs.
        """
        stream = stream or torch.cuda.current_stream()
        sel = slice(None) if rows is None else rows
        r0 = sel.start or 0
        tables = self.tables[sel]
        lens = self.lens[sel]
        assert tables.flags.c_contiguous and lens.flags.c_contiguous
        n = lens.size
        b = self._step & 1
        if self._meta_done[b] is not None:
            self._meta_done[b].synchronize()          # the H2D out of this host slot has finished
        h_slots, h_lens, h_upd, h_pairs = self._meta_views[b]
        d_slots, d_lens, d_upd, d_pairs = self._meta_dviews[b]
        # the reservation writes the slots, pairs and changed table entries straight into the staging
        npairs, nu = self.pool.pa_reserve_slots_with_updates(tables, lens, r0, h_slots.numpy()[:n],
                                                             h_pairs.numpy(), h_upd.numpy())
        self._step += 1
        slots = h_slots.numpy()[:n].copy()
        pairs = h_pairs.numpy()[:npairs].copy()
        h_lens.numpy()[:self.lens.size] = self.lens
        with torch.cuda.stream(stream):
            self._meta_dev[b].copy_(self._meta_host[b], non_blocking=True)
            ev = torch.cuda.Event()
            ev.record(stream)
            self._meta_done[b] = ev
        pa.pa_update_block_tables(self.d_tables, d_upd[:nu], self.d_lens, d_lens[:self.lens.size], stream=stream)
        self.copy_blocks(d_pairs[:npairs], stream=stream)
        self.append(k_new, v_new, d_slots[:n], stream=stream)
        self.attend(q, out, scale, partition_size, workspace, tables=self.d_tables[sel], lens=self.d_lens[sel],
                    stream=stream)
        return slots, pairs

    # ------------------------------------------------------- chunks of tokens

    def attend_chunks(self, q, q_starts, out, scale, causal=True, tables=None, lens=None, workspace=None, stream=None):
        """Attention of ``q_starts``' chunks of ``q`` over the rows' contexts (``pa_prefill_attention``).

        ``causal=False`` is cross attention: every token sees the row's whole context (an encoder's states).
        """
        pa.pa_prefill_attention(q, self.k_cache, self.v_cache, self.d_tables if tables is None else tables,
                                self.d_lens if lens is None else lens, q_starts, scale, out, causal=causal,
                                workspace=workspace, stream=stream)

    def _here(self, stream):
        """``stream`` or the current one; refuses what is not a stream, and any device but the current one."""
        device = torch.cuda.current_device()
        if stream is None:
            stream = torch.cuda.current_stream()
        elif not isinstance(stream, torch.cuda.Stream):
            raise TypeError("stream must be a torch.cuda.Stream")
        if self.k_cache.get_device() != device or stream.device_index != device:
            raise ValueError("the cache and the stream must be on the current device")
        return stream

    def _stage(self, sizes, stream):
        """Buffers for one transfer of arrays of up to ``sizes`` bytes each; nothing is sent.

        The pinned side is double-buffered and grows on demand; the device side is a fresh buffer of ``stream``.
        """
        total = sum(-(-int(n) // 8) * 8 for n in sizes)
        b = self._chunk & 1
        if self._chunk_done[b] is not None:
            self._chunk_done[b].synchronize()             # the transfer out of this host buffer has finished
        if self._chunk_host[b] is None or self._chunk_host[b].numel() < total:
            self._chunk_host[b] = torch.empty(max(4096, 2 * total), dtype=torch.uint8).pin_memory()
        with torch.cuda.stream(stream):
            return torch.empty(max(total, 8), dtype=torch.uint8, device=self.device)

    def _send(self, arrays, dev, stream):
        """Copy int32/int64 numpy arrays to ``dev`` (of ``_stage``) in one transfer; returns their device views."""
        offsets, total = [], 0
        for a in arrays:
            offsets.append(total)
            total += -(-a.nbytes // 8) * 8
        b = self._chunk & 1
        self._chunk += 1
        host = self._chunk_host[b]
        raw = host.numpy()
        for a, o in zip(arrays, offsets):
            raw[o:o + a.nbytes] = np.ascontiguousarray(a).reshape(-1).view(np.uint8)
        with torch.cuda.stream(stream):
            dev[:total].copy_(host[:total], non_blocking=True)
            self._chunk_done[b] = torch.cuda.Event()
            self._chunk_done[b].record(stream)
        kinds = {4: torch.int32, 8: torch.int64}
        return [dev[o:o + a.nbytes].view(kinds[a.dtype.itemsize]).view(a.shape) for a, o in zip(arrays, offsets)]

    def _check_rotary(self, q, k_new, v_new, total, inv_freq, positions, pair_axis, q_out):
        """Refusals of ``pa_rope_append`` that ``prefill_step`` makes before it changes the host tables."""
        for t in (q, k_new, v_new):
            row = t.shape[1] * self.head_dim
            if total and (t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != self.head_dim) or total > 1
                          and (t.stride(0) < row or t.stride(0) * t.element_size() % 16)):
                raise ValueError("q, k_new and v_new must have contiguous, 16-byte aligned token rows")
        ints = [(positions, "positions"), (pair_axis, "pair_axis")]
        for t, name, dtype in [(inv_freq, "inv_freq", torch.float32)] + [(t, n, torch.int32) for t, n in ints]:
            if t is not None and not (t.is_cuda and t.dtype == dtype and t.is_contiguous()
                                      and t.get_device() == q.get_device()):
                raise TypeError("%s must be a contiguous %s tensor on q's device" % (name, dtype))
        if not 0 < 2 * inv_freq.numel() <= self.head_dim:
            raise ValueError("inv_freq must have between 1 and head_dim / 2 entries")
        if positions is not None and (positions.dim() not in (1, 2) or positions.shape[-1] != total
                                      or positions.numel() == 0 and total):
            raise ValueError("positions must be [axes, T] or [T]")
        if pair_axis is not None and pair_axis.numel() != inv_freq.numel():
            raise ValueError("pair_axis must have one entry per pair of inv_freq")
        if q_out is not None and not (q_out.is_cuda and q_out.dtype == self.dtype and q_out.shape == q.shape
                                      and q_out.is_contiguous() and q_out.get_device() == q.get_device()):
            raise ValueError("q_out must be a contiguous tensor like q")
        if q_out is not None and (q_out.data_ptr() % 16 or q_out.data_ptr() == q.data_ptr()
                                  and not q.is_contiguous()):
            raise ValueError("q_out must be 16-byte aligned, and may be q only when q is contiguous")

    def _check_attention(self, total, num_seqs, num_q_heads, scale, workspace):
        """Refusals of ``pa_prefill_attention`` that ``prefill_step`` makes before it changes the host tables."""
        if not math.isfinite(ctypes.c_float(ctypes.c_float(scale).value * pa.LOG2E).value):
            raise ValueError("scale * log2(e) must be finite")
        if max(self.num_blocks * self.block_size, total * num_q_heads) >= 1 << 31 \
                or self.max_blocks * self.block_size >= (1 << 31) - 128:
            raise ValueError("pool, table or chunk too large for 32-bit indices")
        if workspace is not None and total:
            if not workspace.is_cuda or workspace.get_device() != torch.cuda.current_device():
                raise ValueError("workspace must be on the current device")
            need = pa.pa_prefill_workspace_size(total, num_seqs, num_q_heads, self.num_kv_heads, self.head_dim,
                                                self.max_blocks, self.block_size)
            if (not workspace.is_contiguous() or workspace.data_ptr() % 32
                    or workspace.numel() * workspace.element_size() < need):
                raise ValueError("workspace must be contiguous, 32-byte aligned and hold %d bytes" % need)

    def prefill_step(self, q, k_new, v_new, out, scale, counts, rows=None, inv_freq=None, positions=None,
                     pair_axis=None, interleaved=False, q_out=None, workspace=None, stream=None):
        """A chunk of ``counts[i]`` new tokens for each of ``rows`` (a ``slice``, default all): reserve, copy-on-write,
        (rotate and) append, attend.

        ``q``/``out`` ([T, Hq, D]) and ``k_new``/``v_new`` ([T, Hkv, D]) hold the rows' tokens packed in row order
        (T = sum of counts); all are CUDA tensors, and the device tables must have been uploaded once
        (``upload_tables``).  With ``inv_freq``, queries and keys are turned by their rotary angles first
        (``pa_rope_append``): ``positions`` int32 [axes, T] on the device, by default each token's place in its
        sequence; the turned queries go to ``q_out`` (allocated when not given).  Returns the host slots and copy
        pairs.  A row with count 0 takes no part.

        A row that holds its prompt's blocks already (``pa_seq_alloc_prompt``) is refused until its length is the
        prompt's: its tokens go to their slots in the row's table (``append``, ``pa_rope_append``), and
        ``attend_chunks`` reads them.  ``decode_step`` and the engine append keys as they are given: the tokens that
        follow a prompt with rotary positions come as chunks of one, or turned by the caller.
        """
        # everything that can be refused is refused, and everything allocated, before the host tables change
        stream = self._here(stream)
        sel = slice(None) if rows is None else rows
        r0 = sel.start or 0
        tables, lens = self.tables[sel], self.lens[sel]
        assert tables.flags.c_contiguous and lens.flags.c_contiguous
        counts = np.ascontiguousarray(np.asarray(counts, np.int32))
        total = int(counts.sum(dtype=np.int64))
        if counts.size != lens.size or (counts.size and int(counts.min()) < 0):
            raise ValueError("counts must have one entry >= 0 per row")
        kv_shape = (total, self.num_kv_heads, self.head_dim)
        if (q.dim() != 3 or q.shape[0] != total or q.shape[2] != self.head_dim or tuple(out.shape) != tuple(q.shape)
                or tuple(k_new.shape) != kv_shape or tuple(v_new.shape) != kv_shape):
            raise ValueError("q, out [T, Hq, D] and k_new, v_new [T, Hkv, D] must hold the sum of counts tokens")
        for t in (q, k_new, v_new, out):
            if not t.is_cuda or t.dtype != self.dtype:
                raise TypeError("q, k_new, v_new and out must be CUDA tensors of the cache's dtype")
            if t.get_device() != torch.cuda.current_device():
                raise ValueError("q, k_new, v_new and out must be on the current device")
        if q.shape[1] % self.num_kv_heads or q.shape[1] // self.num_kv_heads not in (1, 2, 4, 8):
            raise ValueError("query heads per KV head must be 1, 2, 4 or 8")
        if self.head_dim not in (64, 128) or (self.block_size != 8 and self.block_size % 16):
            raise ValueError("chunk steps need head_dim 64 or 128, and blocks of 8 or a multiple of 16 tokens")
        if not out.is_contiguous():
            raise ValueError("out must be contiguous")
        if any(t.data_ptr() % 16 for t in (q, k_new, v_new, out)):
            raise ValueError("q, k_new, v_new and out must be 16-byte aligned")
        self._check_attention(total, counts.size, q.shape[1], scale, workspace)
        if inv_freq is None:
            if not (q.is_contiguous() and k_new.is_contiguous() and v_new.is_contiguous()):
                raise ValueError("q, k_new and v_new must be contiguous")
        else:
            self._check_rotary(q, k_new, v_new, total, inv_freq, positions, pair_axis, q_out)
        own_positions = inv_freq is not None and positions is None
        most_updates = int((-(-counts.astype(np.int64) // self.block_size)).sum()) + counts.size + 1
        dev = self._stage([8 * total, self.lens.nbytes, 4 * counts.size + 4, 12 * most_updates, 8 * counts.size,
                           4 * total if own_positions else 0], stream)
        with torch.cuda.stream(stream):
            if inv_freq is not None and q_out is None:
                q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
            if workspace is None and total:
                workspace = pa.prefill_workspace(total, counts.size, q.shape[1], self.num_kv_heads, self.head_dim,
                                                 self.max_blocks, self.block_size, device=self.device)
        before = lens.copy()
        slots, pairs, updates = self.pool.pa_reserve_chunks(tables, lens, counts, r0)
        starts = np.zeros(counts.size + 1, np.int32)
        np.cumsum(counts, out=starts[1:])
        arrays = [slots, self.lens, starts, updates, pairs]
        if own_positions:
            arrays.append((np.arange(total) + np.repeat(before - starts[:-1], counts)).astype(np.int32))
        sent = self._send(arrays, dev, stream)
        d_slots, d_lens, d_starts, d_upd, d_pairs = sent[:5]
        pa.pa_update_block_tables(self.d_tables, d_upd, self.d_lens, d_lens, stream=stream)
        self.copy_blocks(d_pairs, stream=stream)
        if inv_freq is not None:
            pa.pa_rope_append(q, k_new, v_new, sent[5] if positions is None else positions, inv_freq, d_slots,
                              self.k_cache, self.v_cache, q_out, pair_axis=pair_axis, interleaved=interleaved,
                              stream=stream)
            q = q_out
        else:
            self.append(k_new, v_new, d_slots, stream=stream)
        self.attend_chunks(q, d_starts, out, scale, tables=self.d_tables[sel], lens=self.d_lens[sel],
                           workspace=workspace, stream=stream)
        return slots, pairs

    def compact(self, layers=(), stream=None):
        """Move the live blocks to the front of the pool, on the host and the device.

        ``layers``: (k_cache, v_cache) pairs of further layers that share this cache's pool and tables; they move
        in the same launch.  Block tables change on both sides (the device ones must be up to date).  Returns the
        moves (int32 [M, 2] of old and new id).
        """
        # everything that can be refused is refused, and everything allocated, before the host tables change
        stream = self._here(stream)
        layers = [(self.k_cache, self.v_cache)] + [tuple(pair) for pair in layers]
        if any(len(pair) != 2 for pair in layers):
            raise ValueError("layers must be (k_cache, v_cache) pairs")
        for c in [c for pair in layers for c in pair]:
            if not c.is_cuda or c.shape != self.k_cache.shape or c.dtype != self.dtype or not c.is_contiguous():
                raise ValueError("every layer's caches must be like this cache's")
            if c.get_device() != torch.cuda.current_device() or c.data_ptr() % 16:
                raise ValueError("every layer's caches must be on the current device, 16-byte aligned")
        if len({c.data_ptr() for pair in layers for c in pair}) != 2 * len(layers):
            raise ValueError("the caches must be distinct")
        block_bytes = self.block_size * self.num_kv_heads * self.head_dim * self.k_cache.element_size()
        if block_bytes % 16:
            raise ValueError("blocks must be a multiple of 16 bytes")
        # (no more moves than free or live blocks; a launch has a CTA per move, cache of up to 64 layers and 16 KB)
        free = self.pool.pa_pool_num_free()
        if 2 * min(len(layers), 64) * min(free, self.num_blocks - free) * -(-block_bytes // 16384) >= 1 << 30:
            raise ValueError("too many moves for one launch")
        dev = self._stage([8 * (self.num_blocks // 2 + 1)], stream)
        moves = self.pool.pa_pool_compact(self.tables)
        if len(moves):
            d_moves, = self._send([moves], dev, stream)
            pa.pa_move_blocks([k for k, _ in layers], [v for _, v in layers], d_moves, self.d_tables, stream=stream)
        return moves

    def engine(self, num_q_heads, partition_size=0, stream=None):
        """A native step executor (``pa.Engine``) over this cache's pool, tables and lengths.

        Uploads the tables and lengths first; afterwards steps go through the
        engine (``pa_engine_step``, host buffers in and out).
        """
        self.upload_tables(stream)
        return pa.Engine(self.pool, self.tables, self.lens, self.d_tables, self.d_lens, self.k_cache, self.v_cache,
                         num_q_heads, partition_size, stream)
