"""Chunk-streaming driver of one attention layer's compressed KV cache.

QuantWM processes the cache chunk by chunk (English v2 summary §5.1 and §D.1;
Chinese summary steps (1)-(5)): at each chunk boundary the previous chunk's
Queries are folded into the per-head statistics and the principal basis is
recomputed, the new chunk's Keys and Values are packed once, and the Queries of
the step attend over every packed chunk.  The first chunk has no statistics
(uniform weights, PSAC off).  This module only sequences the library calls; all
arithmetic runs in libqwm.so.
"""
from __future__ import annotations

import math

import torch

from . import (ActiveChunk, Chunk, Context, PagePool, PageTable, Window, pack_psac_layout, qwm_attend, qwm_attend_merge,
               qwm_dequantize, qwm_fit_centroids_kv, qwm_norm_rope, qwm_paged_attend, qwm_paged_write,
               qwm_pages_update, qwm_quantize_kv, qwm_quantize_kv_full, qwm_rope, qwm_select_rank,
               qwm_sync_status, qwm_update_query_stats, qwm_window_attend, qwm_window_read, qwm_window_write)
from .window import _stream_of, check_rows

_MAX_CHUNKS = 128   # chunks that one call of qwm_attend or qwm_attend_merge takes


class CompressedLayer:
    """Running state of one layer: Query statistics, basis, packed chunks, last codebooks."""

    def __init__(self, ctx: Context, device=None, full_query: bool = False, rank_energy: float | None = None,
                 psac_per_head: bool = False, keep_fit_codebooks: bool = False):
        """full_query: rank the QSAC candidates by the full Query second moment (English v2 §C.4
        ablation) instead of its diagonal.  rank_energy: choose each head's PSAC rank per chunk as the
        smallest r <= config.rank whose top-r eigenvalues hold this share of tr M (qwm_select_rank);
        implies the per-head coefficient layout.  psac_per_head: repack each chunk's coefficients into
        the per-head layout (the smaller of dense and sparse per head).  keep_fit_codebooks: keep
        every chunk's bf16 codebooks (only the packing reads them; by default only the last chunk's
        stay, as the next chunk's k-means start)."""
        self.ctx = ctx
        self.full_query = full_query
        self.rank_energy = rank_energy
        self.psac_per_head = psac_per_head or rank_energy is not None
        self.keep_fit_codebooks = keep_fit_codebooks
        cfg = ctx.cfg
        H, d, r = cfg.heads, cfg.head_dim, cfg.rank
        dev = device or torch.device("cuda", torch.cuda.current_device())
        self.device = dev
        self.S = torch.zeros(H, d, d, dtype=torch.float32, device=dev)
        self.n = torch.zeros(H, dtype=torch.int64, device=dev)
        self.w = torch.ones(H, d, dtype=torch.float32, device=dev)
        self.eigvals = torch.zeros(H, d, dtype=torch.float32, device=dev)
        self.u_r = torch.zeros(H, d, max(r, 1), dtype=torch.bfloat16, device=dev)
        self.n_seen = 0          # Queries folded in so far (host copy of n)
        self.chunks: list[Chunk] = []
        self.prev_cent_k = None
        self.prev_cent_v = None
        self._side = None        # second stream for the statistics update of step()
        self._stats_pending = None  # stream_step(): the fold the next packing waits for
        self._hist = None        # stream_step(overlap=True): high-priority stream of the history attention

    def fold_queries(self, q: torch.Tensor, stream=None) -> None:
        """Step 1: fold Queries [H][nq][d] into the statistics and recompute w and U_r."""
        nq = q.shape[1] if q is not None else 0
        qwm_update_query_stats(self.ctx, q, nq, self.S, self.n, self.w, self.eigvals,
                               self.u_r if self.ctx.cfg.rank else None, stream)
        self.n_seen += nq

    def append_chunk(self, k: torch.Tensor, v: torch.Tensor, warm_start: bool = True, stream=None,
                     debug: dict | None = None, stats_done=None) -> Chunk:
        """Steps 2-4: fit the chunk's codebooks and pack its Keys and Values.  `stats_done`: an
        event the packing waits for (a statistics update running on another stream)."""
        n = k.shape[1]
        ch = Chunk.empty(self.ctx, n, self.device)
        init_k = self.prev_cent_k if warm_start else None
        init_v = self.prev_cent_v if warm_start else None
        qwm_fit_centroids_kv(self.ctx, k, v, n, init_k, init_v, ch.cent_k, ch.cent_v, stream)
        s = stream if stream is not None else torch.cuda.current_stream(self.device)
        if stats_done is not None:
            s.wait_event(stats_done)
        psac = self.n_seen > 0 and self.ctx.cfg.rank > 0
        head_rank = None
        if psac:
            with torch.cuda.stream(s):
                ch.u_r.copy_(self.u_r)   # per-chunk snapshot of the basis
            if self.rank_energy is not None:   # per-head rank: basis columns past it zeroed
                head_rank = torch.empty(self.ctx.cfg.heads, dtype=torch.int32, device=self.device)
                qwm_select_rank(self.ctx, self.eigvals, self.rank_energy, ch.u_r, head_rank, stream)
        w = self.w if self.n_seen > 0 else None
        if self.full_query and w is not None:
            qwm_quantize_kv_full(self.ctx, k, v, n, self.S, self.n, ch.u_r if psac else None, ch, debug, stream)
        else:
            qwm_quantize_kv(self.ctx, k, v, n, w, ch.u_r if psac else None, ch, debug, stream)
        if psac and self.psac_per_head:
            pack_psac_layout(self.ctx, ch, head_rank, stream)
        self.chunks.append(ch)
        self.prev_cent_k, self.prev_cent_v = ch.cent_k, ch.cent_v
        if not self.keep_fit_codebooks:
            ch.release_fit_codebooks()   # the stored fp16 codebooks remain; prev_cent_* keeps this one
        return ch

    def attend(self, q: torch.Tensor, out: torch.Tensor | None = None, scale: float | None = None,
               stream=None, active: "ActiveChunk | None" = None) -> torch.Tensor:
        """Step 5: attention of Queries [H][nq][d] over every packed chunk and, when given, the
        chunk still being generated (bf16, optionally block-causal) in the same softmax."""
        H, nq, d = q.shape
        if out is None:
            out = torch.empty(H, nq, d, dtype=torch.float32, device=q.device)
        chunks = self.chunks + ([active] if active is not None else [])
        qwm_attend(self.ctx, q, nq, chunks, 1.0 / math.sqrt(d) if scale is None else scale, out, stream)
        return out

    def dequantize(self, i: int, stream=None):
        ch = self.chunks[i]
        H, d = self.ctx.cfg.heads, self.ctx.cfg.head_dim
        kh = torch.empty(H, ch.n_tokens, d, dtype=torch.bfloat16, device=self.device)
        vh = torch.empty_like(kh)
        qwm_dequantize(self.ctx, ch, kh, vh, stream)
        return kh, vh

    def step(self, q_prev, k, v, q, stream=None) -> torch.Tensor:
        """One streaming step: fold q_prev (may be None), pack (k, v), attend with q.

        The statistics update and the codebook fits do not depend on each other, so the statistics
        run on a second stream beside the fits; the packing waits for both."""
        main = stream if stream is not None else torch.cuda.current_stream(self.device)
        done = None
        if q_prev is not None:
            if self._side is None:
                self._side = torch.cuda.Stream(self.device)
            self._side.wait_stream(main)
            q_prev.record_stream(self._side)
            self.fold_queries(q_prev, self._side)
            done = torch.cuda.Event()
            done.record(self._side)
        self.append_chunk(k, v, stream=main, stats_done=done)
        return self.attend(q, stream=main)

    def stream_step(self, k, v, q, stream=None, overlap: bool = False) -> torch.Tensor:
        """One streaming step in pipelined order: pack (k, v) with the statistics of every Query
        folded so far, attend with q, and fold q into the statistics on a second stream while the
        attention runs; the next call's packing waits for that fold.  The same work as
        step(q_prev, k, v, q) with q_prev the previous call's q, with the statistics beside the
        attention instead of beside the codebook fits.

        overlap: the attention over the chunks already in the cache runs on a high-priority stream
        beside the new chunk's fits and packing (it does not depend on them), and the new chunk's
        attention then merges into it through the rows' log-sum-exp (qwm_attend_merge); the same
        output up to rounding."""
        main = stream if stream is not None else torch.cuda.current_stream(self.device)
        H, nq, d = q.shape
        scale = 1.0 / math.sqrt(d)
        history = None
        if overlap and self.chunks:
            if self._hist is None:
                self._hist = torch.cuda.Stream(self.device, priority=-1)
            out = torch.empty(H, nq, d, dtype=torch.float32, device=q.device)
            lse = torch.empty(H, nq, dtype=torch.float32, device=q.device)
            self._hist.wait_stream(main)
            for t in (q, out, lse):
                t.record_stream(self._hist)
            qwm_attend_merge(self.ctx, q, nq, list(self.chunks), scale, out, lse, False, self._hist)
            history = True
        self.append_chunk(k, v, stream=main, stats_done=self._stats_pending)
        packed = torch.cuda.Event()
        packed.record(main)
        if self._side is None:
            self._side = torch.cuda.Stream(self.device)
        self._side.wait_event(packed)          # the packing has read w and the basis
        q.record_stream(self._side)
        self.fold_queries(q, self._side)
        self._stats_pending = torch.cuda.Event()
        self._stats_pending.record(self._side)
        if history is not None:
            # the new chunk merged in on the same high-priority stream (the statistics fold beside it
            # fills the SMs it leaves)
            self._hist.wait_event(packed)
            qwm_attend_merge(self.ctx, q, nq, [self.chunks[-1]], scale, out, lse, True, self._hist)
            main.wait_stream(self._hist)
        else:
            out = self.attend(q, stream=main)
        main.wait_event(self._stats_pending)   # the step ends when both are done
        return out

    def check(self, stream=None) -> int:
        return qwm_sync_status(self.ctx, stream)

    def nbytes(self) -> int:
        return sum(c.nbytes() for c in self.chunks)


class WindowedLayer:
    """One layer's cache with its newest chunks in a window at 8 or 4 bits and everything older packed to
    2 bits.

    The 2-bit packing is made for history; the newest frames, which the next ones lean on most, stay at 8
    or 4 bits.  A step writes its chunk into the window (Keys turned by `rope`), attends over the packed
    history and the window in one softmax, and folds its Queries into the statistics; when the window is
    full, its oldest chunk is first read back and packed with the statistics gathered so far.

    A step whose operands are refused changes nothing, and one that raises on the way (a call's error
    status) may be made again: the layer is then `length` tokens long, as before, and the chunk that was
    already packed to make room is not packed again."""

    def __init__(self, ctx: Context, chunk_tokens: int, window_chunks: int, bits: int = 8, tpf: int | None = None,
                 rope=None, device=None, **layer_options):
        """chunk_tokens: tokens of every chunk; window_chunks: chunks the window holds; tpf: tokens of a
        frame, for the block-causal mask inside the window (default: a chunk, i.e. a chunk sees itself
        whole); rope: a RopeSpec by which Queries and Keys are turned at their positions, or None;
        layer_options: CompressedLayer's."""
        if chunk_tokens < 1 or window_chunks < 1:
            raise ValueError("chunk_tokens and window_chunks must be at least 1")
        self.ctx = ctx
        self.rope = rope
        self.chunk_tokens = chunk_tokens
        self.tpf = chunk_tokens if tpf is None else tpf
        self.packed = CompressedLayer(ctx, device, **layer_options)
        self.window = Window.empty(bits, 1, ctx.heads, 0, window_chunks * chunk_tokens, self.packed.device)
        self.length = 0    # tokens seen
        self._packed = 0   # tokens of them that have left the window
        # what the layer owns was filled on this stream; a step on another one waits for the event
        self._stream = torch.cuda.current_stream(self.packed.device)
        self._done = self._stream.record_event()

    def _follow(self, main) -> None:
        """Let `main` take over from the stream that the layer was built or last stepped on."""
        if main == self._stream:
            return
        main.wait_event(self._done)
        for owner in (self.window, self.packed, *self.packed.chunks):
            for t in vars(owner).values():
                if isinstance(t, torch.Tensor):   # not handed out again before `main` is done with it
                    t.record_stream(main)
        self._stream = main

    def step(self, k: torch.Tensor, v: torch.Tensor, q: torch.Tensor, stream=None) -> torch.Tensor:
        """Add the chunk k, v [H][chunk_tokens][d] and attend with its Queries q [H][nq][d] (row i is token
        i of the chunk): fp32 [H][nq][d].  bf16 with contiguous channels and rows on 16-byte boundaries,
        otherwise of any strides."""
        n, ring, ctx = self.chunk_tokens, self.window.ring, self.ctx
        for t, name in ((k, "k"), (v, "v"), (q, "q")):
            if not isinstance(t, torch.Tensor) or t.dim() != 3:
                raise TypeError(f"{name}: expected a tensor [heads][tokens][{ctx.cfg.head_dim}]")
        H, nq, d = q.shape
        if k.shape[1] != n or v.shape[1] != n or nq > n:
            raise ValueError(f"expected a chunk of {n} tokens and at most as many Queries, got {k.shape[1]}, {v.shape[1]} and {nq}")
        for t, name, m in ((k, "k", n), (v, "v", n), (q, "q", nq)):
            check_rows(ctx, t[None], name, (1, ctx.heads, m, ctx.cfg.head_dim))
        main = stream if stream is not None else torch.cuda.current_stream(self.packed.device)
        with torch.cuda.stream(main):
            eager = not torch.cuda.is_current_stream_capturing()   # who replays a captured step orders the replays
            if eager:
                self._follow(main)
            try:
                # where the chunk that makes room began, where this one does, and the length after it
                at = torch.arange(self.length - ring, self.length + n + 1, n, dtype=torch.int64, device=k.device)
                oldest, begin, length = at[:1], at[-2:-1], at[-1:]
                if self.length - self._packed >= ring:   # the oldest chunk makes room: read back and packed
                    old = [torch.empty(1, H, n, d, dtype=torch.bfloat16, device=k.device) for _ in range(2)]
                    qwm_window_read(ctx, self.window, oldest, begin, *old, stream=main)
                    self.packed.append_chunk(old[0][0], old[1][0], stream=main)
                    self._packed += n
                qwm_window_write(ctx, self.window, k[None], v[None], begin, rope=self.rope, stream=main)
                if self.rope is not None:
                    turned = torch.empty(H, nq, d, dtype=torch.bfloat16, device=q.device)
                    qwm_rope(ctx, self.rope, q[None], begin, turned[None], stream=main)
                    q = turned
                else:
                    q = q.contiguous()   # as the calls of the packed path take them
                out = torch.empty(H, nq, d, dtype=torch.float32, device=q.device)
                lse = torch.empty(H, nq, dtype=torch.float32, device=q.device)
                scale = 1.0 / math.sqrt(d)
                for i in range(0, len(self.packed.chunks), _MAX_CHUNKS):
                    qwm_attend_merge(ctx, q, nq, self.packed.chunks[i:i + _MAX_CHUNKS], scale, out, lse, i > 0, main)
                # the window holds exactly the chunks that are not packed: every frame of it is recent
                qwm_window_attend(ctx, self.window, q[None], begin, length, self.tpf, ring // self.tpf + 2, scale,
                                  out[None], lse=lse[None], merge=bool(self.packed.chunks), stream=main)
                self.packed.fold_queries(q, main)
            finally:   # what was issued before an error too is waited for
                if eager:
                    self._done.record(main)
            self.length += n
        return out

    def check(self, stream=None) -> int:
        return self.packed.check(stream)

    def nbytes(self) -> int:
        return self.packed.nbytes() + self.window.nbytes()


class PagedBatch:
    """Many sequences of any lengths through the layers of a model, their Keys and Values at 8 or 4 bits in pages
    that all sequences share.

    A step is begun with what every sequence is shortened to and how many tokens it gets; then each layer is
    called once with the step's packed Queries, Keys and Values (rows of all sequences one after the other, as
    `begin` was told).  What a step needs of the device stays on the device, so that a step may be captured in
    a CUDA graph and replayed with other counts in the same tensors.  Calls follow one another on whatever streams
    they are made, but for captured ones, whose replays the caller orders.

    A step's tensors have `rows` rows whatever it was given: those of no sequence are stored and attended nowhere, but
    the caller brings them, and the Queries' norm and rotation pass over them.  Choose `rows` (or batches of several
    sizes) near what steps hold."""

    def __init__(self, ctx: Context, layers: int, kv_heads: int, batch: int, max_tokens: int, pages: int, rows: int,
                 page: int = 64, bits: int = 8, rope=None, norm: bool = True, eps: float = 1e-6, tpf: int = 1,
                 frames: int | None = None, sink: int = 0, device=None):
        """batch: sequences held at once; max_tokens: of one of them; pages: of the pool, shared; rows: of a step's
        packed batch; rope: a RopeSpec by which Queries and Keys are turned at their positions, or None; norm:
        whether they are divided by their rows' root mean square first; tpf, frames, sink: the mask (default:
        causal)."""
        self.ctx, self.rope, self.norm, self.eps = ctx, rope, norm, eps
        self.mask = dict(tpf=tpf, frames=frames, sink=sink)
        dev = device or torch.device("cuda", torch.cuda.current_device())
        self.table = PageTable.empty(batch, -(-max_tokens // page), page, pages, dev)
        self.pools = [PagePool.empty(bits, page, pages, kv_heads, dev) for _ in range(layers)]
        i32, i64 = dict(dtype=torch.int32, device=dev), dict(dtype=torch.int64, device=dev)
        self.first, self.granted = torch.zeros(batch, **i32), torch.zeros(batch, **i32)
        self.slot, self.at = torch.full((rows,), -1, **i64), torch.full((rows,), -1, **i64)
        self._zero = torch.zeros(1, **i64)
        # what the batch owns was filled on this stream; a call on another one waits for the event
        self._stream = torch.cuda.current_stream(self.at.device)
        self._done = self._stream.record_event()

    def _turn(self, stream):
        """The stream of a call (given as an object, a handle or None: the current one), made to follow the last
        call's."""
        handle, last = _stream_of(self.ctx, stream), self._stream
        if handle == last.cuda_stream:
            return last
        dev = self.at.device
        main = stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(handle, dev)
        with torch.cuda.stream(main):
            if not torch.cuda.is_current_stream_capturing():   # who replays a captured step orders the replays
                main.wait_event(self._done)
                for owner in (self, self.table, *self.pools):
                    for t in vars(owner).values():
                        if isinstance(t, torch.Tensor):   # not handed out again before `main` is done with it
                            t.record_stream(main)
                self._stream = main
        return main

    def _leave(self, main) -> None:
        """What a call issued on its stream is what the next one on another stream waits for."""
        if main is not self._stream:   # captured
            return
        if main.cuda_stream == _stream_of(self.ctx, None):
            eager = not torch.cuda.is_current_stream_capturing()
        else:
            with torch.cuda.stream(main):
                eager = not torch.cuda.is_current_stream_capturing()
        if eager:
            self._done.record(main)

    def begin(self, count: torch.Tensor, keep: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Shorten every sequence to keep [batch] (int64) tokens, then append count [batch] (int32) new ones: their
        rows of the packed batch follow one another.  Returns how many each was given: its count, or 0 where the
        pages do not suffice (its rows are then left out of the step)."""
        main = self._turn(stream)
        try:
            qwm_pages_update(self.ctx, self.table, self.first, self.granted, self.slot, self.at, count=count, keep=keep,
                             stream=main)
        finally:   # what was issued before an error too is waited for
            self._leave(main)
        return self.granted

    def _ready(self, q: torch.Tensor, weight, stream) -> torch.Tensor:
        """The Queries normed and turned, as the Keys are while they are stored."""
        if not self.norm and self.rope is None:
            return q
        h, n, d = q.shape
        out = torch.empty(n, h, d, dtype=torch.bfloat16, device=q.device).permute(1, 0, 2)
        if self.norm:
            qwm_norm_rope(self.ctx, self.rope, q[None], weight, self.eps, out[None],
                          at=self.at[None] if self.rope is not None else None, stream=stream)
        else:
            gh, gw = self.rope.grid_h, self.rope.grid_w
            t, y, x = self.at // (gh * gw), self.at // gw % gh, self.at % gw
            qwm_rope(self.ctx, self.rope, q[None], self._zero, out[None], pos=torch.stack([t, y, x], -1)[None].to(torch.int32),
                     stream=stream)
        return out

    def layer(self, i: int, q, k, v, q_weight=None, k_weight=None, out=None, lse=None, merge: bool = False,
              max_count: int | None = None, scale: float | None = None, stream=None) -> torch.Tensor:
        """Layer i: q [H][rows][d] attends, k and v [kv_heads][rows][d] are stored.  q_weight, k_weight: of the norms
        (fp32 [d] or one per head, None: ones); out: bf16 (default: a new one, padding rows 0) or fp32; lse and
        merge as qwm_paged_attend's; max_count: the largest count of the step, where it is known.  Unknown (None: the
        batch's rows) it launches the kernels for long prompts, too, which costs a step of single tokens 4 to 9 us a layer and
        40 MB of workspace.  A rotation without norms turns the Queries in several elementwise launches."""
        if not self.norm and (q_weight is not None or k_weight is not None):
            raise ValueError("weights of norms that this batch does not form")
        main = self._turn(stream)
        try:
            with torch.cuda.stream(main):
                qwm_paged_write(self.ctx, self.pools[i], k, v, self.slot, at=self.at if self.rope is not None else None,
                                rope=self.rope, norm=self.norm, weight=k_weight, eps=self.eps, stream=main)
                q = self._ready(q, q_weight, main)
                if out is None:
                    out = torch.zeros_like(q, dtype=torch.bfloat16)
                qwm_paged_attend(self.ctx, self.pools[i], self.table, q, self.first, self.granted,
                                 1.0 / math.sqrt(q.shape[2]) if scale is None else scale, out, lse=lse, merge=merge,
                                 max_count=max_count, stream=main, **self.mask)
        finally:   # what was issued before an error too is waited for
            self._leave(main)
        return out

    def check(self, stream=None) -> int:
        return qwm_sync_status(self.ctx, stream)

    def nbytes(self) -> int:
        return sum(p.nbytes() for p in self.pools)
