"""Layer and truncated-stack driver: issues the library calls of a Beam decoder layer in order.

Host orchestration only (buffer management and call order); the arithmetic is in libbeam.so.
Beam page: layers alternate sliding-window (RoPE) and NoPE full attention with every 6th layer
and the last one NoPE ("Attention" section); each sublayer sits between a post-norm and the
next pre-norm with the n-th residual term h <- sqrt((n-1)/n) h + x/sqrt(n), the embedding
being term 1 ("MoE and residual stream" section); layers 0-2 use the dense SwiGLU MLP.
"""
from __future__ import annotations

import contextlib

import torch

from . import beam as B


def is_nope_layer(layer: int, n_layers: int) -> bool:
    """Every 6th layer (0-based l with (l+1) % 6 == 0) and the last layer are NoPE."""
    return (layer + 1) % 6 == 0 or layer == n_layers - 1


def on(stream):
    """Context in which torch's work, and the memory it takes, belongs to `stream` (None: the current)."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


class BeamStack:
    """A truncated Beam stack on one GPU.

    weights: list (one per layer) of dicts of device tensors, keys as made by
             synth.layer_weights (attn_pre, attn_post, mlp_pre, mlp_post, w_qkvg, q_norm,
             k_norm, gate_bias, w_o, and w_gate_up/w_down (+ router, corr_bias on MoE layers);
             an MoE layer may hold "nvfp4" (synth.expert_weights_nvfp4) or "fp8"
             (synth.expert_weights_fp8) instead of w_gate_up/w_down, and then runs
             beam_moe_nvfp4 or beam_moe_fp8).
    caches : list of B.KVCache, one per layer (window = W on sliding-window layers, 0 on NoPE),
             or of B.PagedKVCache. A paged layer projects into a staging row per token, writes
             it into the pages (beam_paged_kv_write), and attends with beam_paged_attn up to
             PAGED_MAX_Q tokens per sequence; with more it reads the sequences' context back
             into a contiguous BF16 cache (beam_paged_kv_read) that beam_attn's prefill takes.
             There a token with a key in a bad page attends to nothing (beam_paged_attn leaves
             that key out); both set BEAM_DEV_BAD_PAGE. Position 0 pads a decode batch over paged
             layers; with more tokens per sequence, and over contiguous caches, it is flagged.

    Over paged caches alone, verify() runs the held layers for the drafted trees of speculative decoding and keep()
    moves the rows of the accepted nodes to the sequences' ends, in every layer's pages.

    Buffers between calls: those of the last number of tokens, one workspace, and one context copy
    for each window. What a captured call uses stays allocated as long as the stack, whatever
    calls come between its replays. All calls and replays of a stack share these buffers, so they
    run one after the other.
    """

    # A call's tokens of one sequence each read their keys in beam_paged_attn; the way through a
    # contiguous copy writes and reads them in BF16 once more, whatever the tokens' number. A NoPE
    # layer from projection to o_proj, pages against copy, for 4 / 5 / 8 tokens of each sequence (us):
    #   1 x 100,000 keys  BF16 270:313 323:322 488:347   FP8 151:289 171:298 265:323   NVFP4 140:287 162:297 227:322
    #   32 x 4000         BF16 391:415 461:440 678:479   FP8 251:382 284:407 404:443   NVFP4 226:374 257:400 345:436
    # So 4 suits BF16; over FP8 and NVFP4 the pages stay ahead up to about 12, and one bound serves all.
    PAGED_MAX_Q = 4

    # A context copy larger than this is worth a wait for the exact number of its sequences: the
    # read and the attention of so many keys take milliseconds.
    COPY_BYTES = 1 << 30

    def __init__(self, shape, weights, caches, first_layer=0, n_layers=None, device="cuda"):
        """weights[i] / caches[i] belong to global layer first_layer + i of an n_layers-deep
        stack (n_layers defaults to shape.n_layers); the layer index fixes the attention
        kind, the MLP kind and the residual term indices."""
        self.shape = shape
        self.W = weights
        self.caches = caches
        self.L = len(weights)
        self.first = first_layer
        total = shape.n_layers if n_layers is None else n_layers
        self.ids = [first_layer + i for i in range(self.L)]
        self.dense = [l in shape.dense_layers for l in self.ids]
        self.cfgs = [B.LayerCfg.from_shape(
            shape, B.BEAM_ATTN_NOPE_SSMAX if is_nope_layer(l, total) else B.BEAM_ATTN_SWA_ROPE)
            for l in self.ids]
        self.ws = B.Workspace(device)
        self.device = device
        self._bufs = {}
        self._stage = {}
        self._copies = {}
        self._trees = {}
        self._held = []
        self.paged = any(isinstance(c, B.PagedKVCache) for c in caches)

    def hold(self, x):
        """x, which a replay of the call being captured, if there is one, will use again."""
        if B.capturing() and all(x is not y for y in self._held):
            self._held.append(x)
        return x

    def held(self, buffers):
        """The entries of a dict of buffers that captured calls use."""
        return {k: x for k, x in buffers.items() if any(x is y for y in self._held)}

    def stage(self, T):
        """A row per token for the projection's K and V: a ring of one slot per "sequence"."""
        s = self._stage.get(T)
        if s is None:
            dims = (T, self.shape.n_kv, 1, self.shape.head_dim)
            k, v = (torch.empty(dims, dtype=torch.bfloat16, device=self.device) for _ in "kv")
            rows = torch.arange(T, dtype=torch.int32, device=self.device)
            s = (B.KVCache(k, v, window=1), rows, k.view(T, *dims[1::2]), v.view(T, *dims[1::2]))
            self._stage = {**self.held(self._stage), T: s}
        return self.hold(s)

    @staticmethod
    def staged_pos(pos):
        """Positions for the projection of paged layers, which knows no padding: it computes a padding
        row for nothing, and beam_paged_kv_write flags what is below 0."""
        return pos.clamp_min(1)

    @staticmethod
    def reach(kc, max_pos, max_q):
        """(Window, longest range, capacity) of a context copy; a window past the page table's
        reach is that reach, and a ring's capacity a multiple of the attention's key tiles."""
        W, max_pos = min(kc.window, kc.positions), min(max_pos, kc.positions)
        if W == 0:
            return W, max_pos, max_pos
        return W, min(max_pos, W - 1 + max_q), (W - 1 + max_q + 127) // 128 * 128

    def context(self, kc, seq_id, pos, max_pos, max_q, n_seqs=None, ranges=None):
        """What a paged layer's prefill reads: (contiguous cache, its sequences, first, last,
        longest), one row for each of the n_seqs sequences at most that have tokens in the call, in
        their order, or for every sequence of the page table where that is no more. Rows without a
        sequence read nothing. Layers of one window share the cache. ranges: (its sequences, first,
        last), where a layer before has found them."""
        n, dev = kc.page_table.shape[0], pos.device
        rows = n if n_seqs is None else max(1, min(n, n_seqs))
        max_pos = min(max_pos, kc.positions)
        W, longest, cap = self.reach(kc, max_pos, max_q)
        held = [key for key in self._copies if key[1] == W]   # one copy for a window
        copy = self._copies[held[0]] if held else None
        if copy is None or copy.k.shape[0] < rows or copy.k.shape[2] < cap:
            for key in held:
                del self._copies[key]
            if copy is not None and W == 0 and copy.k.shape[2] < cap:
                cap = min(cap + cap // 4, kc.positions)   # a context that grew will grow with the next chunk
            dims = (rows, self.shape.n_kv, cap, self.shape.head_dim)
            k, v = (torch.empty(dims, dtype=torch.bfloat16, device=self.device) for _ in "kv")
            copy = self._copies[(rows, W)] = B.KVCache(k, v, window=W)
        self.hold(copy)
        if ranges is not None:
            return copy, *ranges, longest
        # other tokens are flagged by the library, and reach into no sequence's range
        known = (seq_id >= 0) & (seq_id < n) & (pos >= 1) & (pos <= max_pos)
        s = torch.where(known, seq_id, 0).long()
        last = torch.zeros(n, dtype=torch.int32, device=dev)
        last.scatter_reduce_(0, s, torch.where(known, pos, 0), "amax")
        first = torch.full_like(last, 2 ** 31 - 1)
        first.scatter_reduce_(0, s, torch.where(known, pos, 2 ** 31 - 1), "amin")
        every = torch.arange(n, dtype=torch.int32, device=dev)
        if rows < n:
            # row r: the r-th sequence with tokens, or nothing where there are fewer
            at = (last > 0).cumsum(0) - 1
            at = torch.where((last > 0) & (at < rows), at, rows)
            every = torch.full((rows + 1,), -1, dtype=torch.int32, device=dev).scatter_(0, at, every)[:rows]
            s = every.clamp_min(0).long()
            first, last = first[s], torch.where(every < 0, 0, last[s])
            every = every.clamp_min(0)
        first = (first - W + 1).clamp_min(1) if W else torch.ones_like(last)
        first = torch.where(last > 0, first, 1)
        return copy, every, first, last, longest

    def rows(self, kc, seq_id, pos, every, first, last):
        """Each token's row of the copy (sequences `every`): its sequence's, any for a token at position
        0 of a sequence without one, else an id that is none."""
        n = kc.page_table.shape[0]
        if every.shape[0] == n:
            return seq_id
        at = torch.full((n + 1,), -1, dtype=torch.int32, device=pos.device)
        order = torch.arange(every.shape[0], dtype=torch.int32, device=pos.device)
        at.scatter_(0, torch.where(last > 0, every, n).long(), order)
        known = (seq_id >= 0) & (seq_id < n)
        row = torch.where(known, at[torch.where(known, seq_id, 0).long()], -1)
        return torch.where(known & (pos == 0) & (row < 0), 0, row)

    def readable(self, kc, row, pos, first, last, longest, every=None):
        """pos of tokens that read the ranges `row` (of sequences `every`; None: the table's), with 0
        (attends to nothing) for tokens some of whose keys beam_paged_kv_read does not bring: one
        lies in a page that is none, or the sequence's tokens lie further apart than the copy
        reaches. Either is flagged by the read; the copy holds something else there."""
        table, size = kc.page_table, kc.page_size
        if every is not None and every.shape[0] < table.shape[0]:
            table = table[every.long()]
        s = row.clamp(0, table.shape[0] - 1).long()
        none = ((table < 0) | (table >= kc.num_pages)).cumsum(1, dtype=torch.int32)   # up to each page
        p = pos.clamp(0, kc.positions)
        lo = (p - kc.window).clamp_min(0) if kc.window else torch.zeros_like(p)
        a, b = lo // size, (p - 1).clamp_min(0) // size              # pages of a token's keys
        before = torch.where(a > 0, none[s, (a - 1).clamp_min(0).long()], 0)
        whole = (none[s, b.long()] == before) & ((last - first)[s] < longest)
        return torch.where(whole, pos, 0)

    def count(self, seq_id, max_pos, stream, max_q=1):
        """The number of sequences in a call that does not say it, where every sequence that there
        could be would make a large copy: one wait for the GPU. None where it would not, and under
        a capture, which cannot wait."""
        row = 4 * self.shape.n_kv * self.shape.head_dim
        most = max((min(c.page_table.shape[0], seq_id.shape[0]) * self.reach(c, max_pos, max_q)[2] * row
                    for c in self.caches if isinstance(c, B.PagedKVCache)), default=0)
        if most <= self.COPY_BYTES:
            return None
        with on(stream):
            if B.capturing():
                return None
            return seq_id.unique().numel()

    def attention(self, i, b, seq_id, pos, max_pos, ws, stream, max_q_per_seq, n_seqs=None, call=None):
        """Projection, cache write and attention of the i-th layer held, from b["u"] to b["a"].
        call: a dict for what the layers of one call share."""
        W, cfg, kc = self.W[i], self.cfgs[i], self.caches[i]
        if not isinstance(kc, B.PagedKVCache):
            B.beam_qkv_gate(cfg, b["u"], W["w_qkvg"], W["q_norm"], W["k_norm"], seq_id, pos, b["q"],
                            b["g"], kc, ws, stream)
            B.beam_attn(cfg, b["q"], b["g"], W["gate_bias"], kc, seq_id, pos, max_pos, W["w_o"],
                        b["a"], ws, stream, max_q_per_seq)
            return
        call = {} if call is None else call
        if "tree" in call:
            ids, start, base, t = call["tree"]
            B.beam_paged_qkv_gate(cfg, b["u"], W["w_qkvg"], W["q_norm"], W["k_norm"], t["seq"], t["pos"], t["slot"],
                                  b["q"], b["g"], kc, ws, stream)
            B.beam_paged_tree_attn(cfg, b["q"], b["g"], W["gate_bias"], kc, ids, start, base, t["mask"], max_pos,
                                   W["w_o"], b["a"], ws, stream)
            return
        T = seq_id.shape[0]
        max_q = T if max_q_per_seq is None else max_q_per_seq
        # buffers that a later call may drop belong to the stream that uses them
        with on(stream):
            stage, rows, k, v = self.stage(T)
            if "staged" not in call:
                call["staged"] = self.staged_pos(pos)
        B.beam_qkv_gate(cfg, b["u"], W["w_qkvg"], W["q_norm"], W["k_norm"], rows, call["staged"],
                        b["q"], b["g"], stage, ws, stream)
        B.beam_paged_kv_write(k, v, seq_id, pos, kc, stream)
        if max_q <= self.PAGED_MAX_Q:
            B.beam_paged_attn(cfg, b["q"], b["g"], W["gate_bias"], kc, seq_id, pos, max_pos,
                              W["w_o"], b["a"], ws, stream)
            return
        with on(stream):
            # a token past the table was flagged by the write; beam_attn shares key tiles between a
            # sequence's tokens, and must not take it for the sequence's end
            max_pos = min(max_pos, kc.positions)
            most = T if n_seqs is None else min(T, n_seqs)
            # layers over one table and window read the same ranges: worked out by the first of them
            # (a chunk of 512 tokens, six layers, from projection to attention: 0.83 -> 0.23 ms a layer
            # from the host, 290 -> 187 us in a graph)
            over = (kc.page_table, kc.window, kc.page_size, kc.num_pages)
            ranges, row, reach = next((x for o, x in call.get("ranges", []) if o[0] is over[0] and o[1:] == over[1:]),
                                      (None, None, None))
            if ranges is None:
                pos = pos.masked_fill(pos > max_pos, 0)
            copy, every, first, last, longest = self.context(kc, seq_id, pos, max_pos, max_q, most, ranges)
            if ranges is None:
                row = self.rows(kc, seq_id, pos, every, first, last)
                reach = self.readable(kc, row, pos, first, last, longest, every)
                call.setdefault("ranges", []).append((over, ((every, first, last), row, reach)))
        B.beam_paged_kv_read(kc, every, first, last, longest, copy, stream)
        B.beam_attn(cfg, b["q"], b["g"], W["gate_bias"], copy, row, reach, max_pos, W["w_o"],
                    b["a"], ws, stream, max_q_per_seq)

    def buffers(self, T):
        b = self._bufs.get(T)
        if b is None:
            s, dev = self.shape, self.device
            bf = torch.bfloat16
            b = {
                "h": torch.empty((T, s.hidden), dtype=bf, device=dev),
                "u": torch.empty((T, s.hidden), dtype=bf, device=dev),
                "q": torch.empty((T, s.n_q, s.head_dim), dtype=bf, device=dev),
                "g": torch.empty((T, s.q_rows), dtype=bf, device=dev),
                "a": torch.empty((T, s.hidden), dtype=bf, device=dev),
                "m": torch.empty((T, s.hidden), dtype=bf, device=dev),
                "logits": torch.empty((T, s.n_experts), dtype=torch.float32, device=dev),
                "idx": torch.empty((T, s.topk), dtype=torch.int32, device=dev),
                "w": torch.empty((T, s.topk), dtype=torch.float32, device=dev),
            }
            self._bufs = {**self.held(self._bufs), T: b}
        return self.hold(b)

    def layer(self, i, b, seq_id, pos, max_pos, ws, stream=None, trace=None, max_q_per_seq=None,
              n_seqs=None, call=None):
        """The i-th layer held (global index l): from (h, u = its attention pre-norm) to
        (h, u of the next layer). With a trace list, appends the layer's intermediate tensors:
        u_attn, q, g, attn, h_mid (h after the attention residual), mlp_in, mlp, route
        (logits, idx, w) on MoE layers, and the output h."""
        with on(stream):
            self._layer(i, b, seq_id, pos, max_pos, ws, stream, trace, max_q_per_seq, n_seqs, call)

    def _layer(self, i, b, seq_id, pos, max_pos, ws, stream, trace, max_q_per_seq, n_seqs, call):
        W, cfg = self.W[i], self.cfgs[i]
        l = self.ids[i]
        if trace is not None:
            trace.append({"u_attn": b["u"].clone()})
        self.attention(i, b, seq_id, pos, max_pos, ws, stream, max_q_per_seq, n_seqs, call)
        B.beam_boundary_norm(b["a"], b["h"], b["u"], W["attn_post"], W["mlp_pre"], 2 * l + 2,
                             cfg.eps, stream)
        if trace is not None:
            trace[-1].update({"q": b["q"].clone(), "g": b["g"].clone(), "attn": b["a"].clone(),
                              "h_mid": b["h"].clone(), "mlp_in": b["u"].clone()})
        if self.dense[i]:
            B.beam_dense_mlp(cfg, b["u"], W["w_gate_up"], W["w_down"], b["m"], ws, stream)
        else:
            B.beam_route(cfg, b["u"], W["router"], W["corr_bias"], b["logits"], b["idx"], b["w"],
                         ws, stream)
            if "nvfp4" in W:
                B.beam_moe_nvfp4(cfg, b["u"], b["idx"], b["w"], W["nvfp4"], b["m"], ws, stream)
            elif "fp8" in W:
                B.beam_moe_fp8(cfg, b["u"], b["idx"], b["w"], W["fp8"], b["m"], ws, stream)
            else:
                B.beam_moe(cfg, b["u"], b["idx"], b["w"], W["w_gate_up"], W["w_down"], b["m"],
                           ws, stream)
        if trace is not None:
            trace[-1]["mlp"] = b["m"].clone()
            if not self.dense[i]:
                trace[-1]["route"] = (b["logits"].clone(), b["idx"].clone(), b["w"].clone())
        nxt = self.W[i + 1]["attn_pre"] if i + 1 < self.L else None
        B.beam_boundary_norm(b["m"], b["h"], b["u"] if nxt is not None else None,
                             W["mlp_post"], nxt, 2 * l + 3, cfg.eps, stream)
        if trace is not None:
            trace[-1]["h"] = b["h"].clone()

    def forward(self, e, seq_id, pos, max_pos, stream=None, trace=None, max_q_per_seq=None,
                n_seqs=None):
        """Runs the held layers for the tokens (seq_id, pos). e [T][H] (bf16) is the residual
        stream entering the first held layer (the embedding when first_layer is 0); it gets
        its pre-norm first. max_q_per_seq: most tokens of one sequence (1 for a decode batch;
        None = T). n_seqs: upper bound of the number of sequences with tokens in the call, which
        sizes the context copies of a prefill over paged caches (tokens of sequences past it are
        flagged as of a bad sequence). None: at most T, counted, with one wait for the GPU, where
        that many would take more than COPY_BYTES (not in a captured call: say it there).
        stream: where all of the call runs (None: the current one); the inputs are ready there.
        Returns h after the last residual addition (an internal buffer)."""
        with on(stream):   # torch's copies and allocations too
            return self._forward(e, seq_id, pos, max_pos, stream, trace, max_q_per_seq, n_seqs)

    def _forward(self, e, seq_id, pos, max_pos, stream, trace, max_q_per_seq, n_seqs):
        T = e.shape[0]
        max_q = T if max_q_per_seq is None else max_q_per_seq
        if self.paged and n_seqs is None and max_q > self.PAGED_MAX_Q:
            n_seqs = self.count(seq_id, max_pos, stream, max_q)
        b = self.buffers(T)
        need = B.workspace_bytes(self.cfgs[0], T, max_pos)
        if self.paged:
            need = max(need, B.paged_workspace_bytes(self.cfgs[0], T, max_pos))
        ws = self.ws.get(need)
        b["h"].copy_(e)
        B.beam_boundary_norm(None, b["h"], b["u"], None, self.W[0]["attn_pre"], 1,
                             self.cfgs[0].eps, stream)
        call = {}
        for i in range(self.L):
            self.layer(i, b, seq_id, pos, max_pos, ws, stream, trace, max_q_per_seq, n_seqs, call)
        return b["h"]

    def tree_buffers(self, T):
        t = self._trees.get(T)
        if t is None:
            t = {k: torch.empty(T, dtype=torch.int64 if k == "mask" else torch.int32, device=self.device)
                 for k in ("mask", "pos", "slot", "seq")}
            self._trees = {**self.held(self._trees), T: t}
        return self.hold(t)

    def verify(self, e, parent, row_start, seq_id, base, max_pos, stream=None, trace=None):
        """Runs the held layers for drafted trees, over paged caches. Rows row_start[i] .. row_start[i+1]-1 of e [T][H]
        are the nodes of a tree (at most 64, parents before children) behind the base[i] tokens of sequence
        seq_id[i]; parent [T] is each node's parent within its tree, -1 for a root. Node j's keys and values go to
        slot base[i] + 1 + j of every layer's pages. max_pos: upper bound of base[i] plus the tree's size. Rows outside
        all trees are padding. Returns h after the last residual addition (an internal buffer); with the tokens
        sampled from it, beam_tree_accept gives the path that keep() takes."""
        if not all(isinstance(c, B.PagedKVCache) for c in self.caches):
            raise B.BeamError("BeamStack.verify needs paged caches in every layer")
        with on(stream):
            T = e.shape[0]
            b, t = self.buffers(T), self.tree_buffers(T)
            ws = self.ws.get(max(B.workspace_bytes(self.cfgs[0], T, max_pos),
                                 B.paged_tree_workspace_bytes(self.cfgs[0], T)))
            b["h"].copy_(e)
            B.beam_tree_plan(parent, row_start, seq_id, base, t["mask"], t["pos"], t["slot"], t["seq"], stream)
            B.beam_boundary_norm(None, b["h"], b["u"], None, self.W[0]["attn_pre"], 1, self.cfgs[0].eps, stream)
            call = {"tree": (seq_id, row_start, base, t)}
            for i in range(self.L):
                self._layer(i, b, t["seq"], t["pos"], max_pos, ws, stream, trace, None, None, call)
            return b["h"]

    def keep(self, seq_id, base, count, path, stream=None):
        """After verify(): the accepted nodes path[i][:count[i]] of each tree become the count[i] tokens behind
        base[i], in every layer's pages."""
        if not all(isinstance(c, B.PagedKVCache) for c in self.caches):
            raise B.BeamError("BeamStack.keep needs paged caches in every layer")
        with on(stream):
            for kc in self.caches:
                B.beam_paged_kv_keep(kc, seq_id, base, count, path, stream)
