"""Decoding many long conversations in a bounded cache: ``BoundedDecoder``.

Sequences may begin with a shared prefix (a system prompt, a document), whose keys and
values are cached once and read once per step for all of its rows.  What a sequence
holds on its own is bounded: once it has ``budget + slack`` tokens, each (layer, KV
head) keeps the ``budget`` tokens that have drawn the most attention so far, with the
first ``sink`` and the last ``recent`` ones always among them, and the blocks behind go
back to the pool.  Positions go on counting past the evicted tokens, so the rotary
frequencies may be scaled for contexts longer than the trained one.

A step is a0 on the host (``PagedDecoder``'s, positions offset by prefix and evicted
tokens), then per layer ``pkv_rotary_append`` and ``pkv_decode_attn_shared`` with the
weights accumulated, and before it ``pkv_evict`` for the rows that have reached their
bound.
"""
import math

import numpy as np

from . import binding
from .engine import PagedDecoder


class BoundedDecoder(PagedDecoder):
    """``budget``: own tokens a sequence keeps when it is cut back, which happens before
    the step that would append to ``budget + slack`` tokens.  ``rotary``: a
    ``binding.Rotary`` (default: the whole head, plain, at ``rope_base``).  ``decay``: factor on the
    weight accumulated so far at every step.  ``max_prefixes`` prefixes of up to
    ``max_prefix_len`` tokens may be live.  The rest as ``PagedDecoder``; its captured
    forms, additive masks, layer chains (``layer_merge_helpers``) and flags other than
    ``ATTN_CHECK_PLAN`` and ``ATTN_SHORT_WAITS`` are not offered here."""

    served = False

    def __init__(self, num_blocks, Hq, Hkv, d, dtype, max_seqs, budget, slack=64, sink=4,
                 recent=None, rotary=None, decay=1.0, max_prefixes=16, max_prefix_len=131072, **kw):
        import torch
        if budget < 1 or slack < 1:
            raise ValueError("budget and slack must be at least 1")
        recent = budget // 4 if recent is None else recent
        if sink < 0 or recent < 0:
            raise ValueError("sink and recent must not be negative")
        if not math.isfinite(decay) or not math.isfinite(kw.get("scale") or 0.0):
            raise ValueError("scale and decay must be finite")
        if max_prefixes < 0 or max_prefix_len < 0:
            raise ValueError("max_prefixes and max_prefix_len must not be negative")
        if rotary is not None and kw.get("rope_base") is not None:
            raise ValueError("rotary states its own base: give rope_base or rotary")
        if kw.get("flags", 0) & ~(binding.ATTN_CHECK_PLAN | binding.ATTN_SHORT_WAITS):
            raise ValueError(f"flags {kw['flags']}: only ATTN_CHECK_PLAN and ATTN_SHORT_WAITS")
        if kw.get("layer_merge_helpers") is not None:
            raise ValueError("layer_merge_helpers: the layers are not launched as a chain")
        need = -(-(budget + slack) // binding.BLOCK_SIZE)
        bt = kw.pop("max_blocks_per_seq", need)
        if bt < need:
            raise ValueError(f"max_blocks_per_seq must be at least {need}")
        self._code = binding.F32 if dtype == "f32" else binding.BF16
        self._parts_given = bool(kw.get("num_parts"))
        if not self._parts_given:
            kw["num_parts"] = binding.shared_default_parts(max_seqs, Hq, Hkv, d, self._code, bt)
        self.max_rows = max_seqs
        super().__init__(num_blocks, Hq, Hkv, d, dtype, max_seqs, bt, **kw)
        # an allocator that also holds the prefixes, one sequence each
        self.alloc.close()
        width = max(bt, min(num_blocks, -(-max_prefix_len // binding.BLOCK_SIZE)))
        self.alloc = binding.BlockAllocator(num_blocks, max_seqs + max_prefixes, width,
                                            kw.get("initial_free"))
        self.budget, self.slack, self.sink, self.recent = budget, slack, sink, recent
        self.rotary = binding.Rotary(d, base=self.rope_base) if rotary is None else rotary
        if self.rotary.d != d:
            raise ValueError(f"rotary was made for heads of {self.rotary.d}, not {d}")
        if self.rotary.axes is not None:
            raise ValueError("rotary has sections: positions have one axis here")
        self.decay = float(decay)
        self.masses = torch.zeros((self.n_layers, num_blocks, Hkv, binding.BLOCK_SIZE),
                                  device=self.device)
        self.scores = binding.alloc_scores(num_blocks, Hq, self.device)
        self._prefix_of = {}     # sequence id -> prefix id or None
        self._prefixes = {}      # prefix id (a sequence of the allocator) -> tokens
        self._known = {}         # sequence id -> leading own tokens whose weight is known
        self._held = {}          # sequence id -> own tokens
        self._plan_key = None
        self._rows_now = None    # sequences of the last step (None: their prefixes may have changed)
        self._prefix_args = {}
        self._space = None
        self._calls = {}         # metadata buffer -> prepared calls of every layer, for this plan

    def _on(self, stream):
        """The stream of a call as torch's current one, so that the call's copies and
        small tensors are ordered with its launches."""
        torch = self.torch
        return torch.cuda.stream(stream if stream is not None
                                 else torch.cuda.current_stream(self.device))

    # -- prefixes and sequences ---------------------------------------------------
    def _write(self, seq, k, v, first, stream):
        """Keys and values ``[L,n,Hkv,d]`` (or ``[n,Hkv,d]``) of all n tokens of a
        sequence into its blocks, rotated at positions ``first ...``."""
        torch = self.torch
        if k.dim() == 3:
            k, v = k.unsqueeze(0), v.unsqueeze(0)
        n = k.shape[1]
        if n == 0:
            return
        pos, slots = self.alloc.seq_slots(seq, 0, n)
        with self._on(stream):
            pos = torch.from_numpy(pos + np.int32(first)).to(self.device)
            slots = torch.from_numpy(slots).to(self.device)
            for layer in range(self.n_layers):
                binding.rotary_append_args(binding.make_rotary_args(
                    self.rotary, None, k[layer], v[layer], pos, slot_mapping=slots,
                    k_cache=self.k_caches[layer], v_cache=self.v_caches[layer], err=self.err))

    def add_prefix(self, k, v, stream=None):
        """Caches the raw keys and values ``[n,Hkv,d]`` (``[L,n,Hkv,d]`` with layers) of a
        shared prefix at positions 0..n-1; returns its id."""
        n = k.shape[-3]
        pid = self.alloc.join(n)
        try:
            self._write(pid, k, v, 0, stream)
        except Exception:
            self.alloc.leave(pid)
            raise
        self._prefixes[pid] = n
        return pid

    def drop_prefix(self, pid):
        """Frees a prefix that no sequence uses any more."""
        if pid not in self._prefixes:
            raise ValueError(f"no prefix {pid}")
        if pid in self._prefix_of.values():
            raise ValueError(f"prefix {pid} is in use")
        self.alloc.leave(pid)
        del self._prefixes[pid]
        self._plan_key = self._rows_now = None    # (the id may come back as another prefix)

    def join(self, prefix_len=0, prefix=None, k=None, v=None, stream=None):
        """A new sequence behind ``prefix`` (an id of ``add_prefix``, or None) with
        ``prefix_len`` own tokens; ``k, v`` hold their raw keys and values (without
        them the caller writes the blocks, as with ``PagedDecoder``)."""
        if prefix is not None and prefix not in self._prefixes:
            raise ValueError(f"no prefix {prefix}")
        if len(self._prefix_of) >= self.max_rows:
            raise ValueError(f"all {self.max_rows} sequences are live")
        if prefix_len >= self.budget + self.slack:
            raise ValueError(f"{prefix_len} own tokens, but at most {self.budget + self.slack - 1} "
                             "are held")
        if k is not None and (v is None or k.shape[-3] != prefix_len or v.shape != k.shape):
            raise ValueError("k and v must hold prefix_len tokens")
        sid = self.alloc.join(prefix_len)
        first = 0 if prefix is None else self._prefixes[prefix]
        try:
            self.alloc.set_offset(sid, first)
            if k is not None:
                self._write(sid, k, v, first, stream)
        except Exception:
            self.alloc.leave(sid)
            raise
        self._prefix_of[sid], self._known[sid], self._held[sid] = prefix, 0, int(prefix_len)
        self._rows_now = None
        return sid

    def leave(self, seq_id):
        if seq_id not in self._prefix_of:
            raise binding.UnknownSequence(binding.ERR_UNKNOWN_SEQ, f"sequence {seq_id} is not live")
        self.alloc.leave(seq_id)
        del self._prefix_of[seq_id], self._known[seq_id], self._held[seq_id]
        self._rows_now = None

    # -- eviction -------------------------------------------------------------------
    def evict(self, seq_ids, keep=None, stream=None):
        """Cuts the listed sequences back to ``keep`` (default: the budget) own tokens;
        returns the kept indices ``[L,n,Hkv,keep]`` (-1 behind a shorter sequence's).  A sequence
        that would get shorter and shares blocks (``alloc.fork``) is refused before anything
        moves."""
        seq_ids = [int(s) for s in seq_ids]
        for s in seq_ids:
            if s not in self._prefix_of:
                raise binding.UnknownSequence(binding.ERR_UNKNOWN_SEQ, f"sequence {s} is not live")
        if len(set(seq_ids)) != len(seq_ids):
            raise ValueError("a sequence may be listed once")
        keep = self.budget if keep is None else int(keep)
        if keep < 0:
            raise ValueError("keep must not be negative")
        with self._on(stream):
            return self._evict(seq_ids, keep)

    def _evict(self, seq_ids, keep):
        torch = self.torch
        n = len(seq_ids)
        kept = torch.full((self.n_layers, n, self.Hkv, max(keep, 1)), -1, dtype=torch.int32,
                          device=self.device)
        if n == 0:
            return kept
        lens = np.array([self._held[s] for s in seq_ids], np.int32)
        # (the allocator refuses these too, but only after their tokens have moved)
        for s, L, shared in zip(seq_ids, lens, self.alloc.shared_blocks(seq_ids)):
            if L > keep and shared:
                raise binding.PkvError(binding.ERR_INVALID_ARG,
                                       f"sequence {s} shares {shared} blocks with another: they are not "
                                       "compacted")
        blocks = [self.alloc.seq_blocks(s) for s in seq_ids]
        tables = np.full((n, max(1, max(len(b) for b in blocks))), -1, np.int32)
        for i, b in enumerate(blocks):
            tables[i, :len(b)] = b
        dev = self.device
        t, ln = torch.from_numpy(tables).to(dev), torch.from_numpy(lens).to(dev)
        kp = torch.full((n,), keep, dtype=torch.int32, device=dev)
        for s, L in zip(seq_ids, lens):   # tokens no step has weighed yet have drawn nothing
            if self._known[s] < L:
                slots = self.alloc.seq_slots(s, self._known[s], int(L) - self._known[s])[1]
                at = torch.from_numpy(slots).to(dev)
                self.masses[:, at // binding.BLOCK_SIZE, :, at % binding.BLOCK_SIZE] = 0.0
                self._known[s] = int(L)
        space = torch.empty(binding.evict_workspace_bytes(n, self.Hkv, self.d, self._code, kept.shape[-1]),
                            dtype=torch.uint8, device=dev)
        # (all calls are made before the first moves anything)
        calls = [binding.make_evict_args(
            self.k_caches[layer], self.v_caches[layer], self.masses[layer], t, ln, kp, kept[layer],
            self.sink, self.recent, workspace=space, err=self.err) for layer in range(self.n_layers)]
        for call in calls:
            binding.evict_args(call)
        self.alloc.evict_many(seq_ids, np.full(n, keep, np.int32))
        for s in seq_ids:
            self._known[s], self._held[s] = min(self._known[s], keep), min(self._held[s], keep)
        return kept

    # -- the step -------------------------------------------------------------------
    def _prefix_state(self, seq_ids):
        """Plan, prefix tables and workspace for these rows (kept while the rows'
        prefixes stay the same)."""
        torch = self.torch
        if seq_ids == self._rows_now:
            return
        rows = tuple(self._prefix_of[s] for s in seq_ids)
        used = sorted({p for p in rows if p is not None and self._prefixes[p] > 0})
        key = (rows, tuple(used))
        if key == self._plan_key:
            self._rows_now = seq_ids
            return
        slots, args = 0, {}
        if used:
            at = {p: i for i, p in enumerate(used)}
            lens = [self._prefixes[p] for p in used]
            plan = binding.shared_plan([at.get(p, -1) for p in rows], lens, self.Hq, self.Hkv, self.d,
                                       self._code)
            blocks = [self.alloc.seq_blocks(p) for p in used]
            tables = np.full((len(used), max(len(b) for b in blocks)), -1, np.int32)
            for i, b in enumerate(blocks):
                tables[i, :len(b)] = b
            slots = int(plan[3])
            args = dict(prefix_tables=torch.from_numpy(tables).to(self.device),
                        prefix_plan=torch.from_numpy(plan).to(self.device), slots=slots,
                        num_ctas=int(plan[4]))
        parts = max(self.num_parts, binding.shared_default_parts(
            len(rows), self.Hq, self.Hkv, self.d, self._code, self.bt_stride))
        need = binding.shared_workspace_bytes(len(rows), self.Hq, self.Hkv, self.d, parts, slots)
        # a workspace of these rows' own, zero-filled once: the counters' place in it
        # depends on the number of rows
        space = torch.zeros(need, dtype=torch.uint8, device=self.device)
        # (all of it or, where something above raised, nothing)
        self._prefix_args, self._space, self._calls = args, space, {}
        self._plan_key, self._rows_now = key, seq_ids

    def _prepared(self, B, q, k, v):
        """The calls of every layer on the metadata buffer of this step, made once for
        each buffer and plan; the step's own tensors are put in by ``_launch``."""
        key = self.positions.data_ptr()     # (one of the decoder's own buffers)
        if key not in self._calls:
            ptab = self._prefix_args.get("prefix_tables")
            short = (not self._parts_given and not self.flags
                     and binding.shared_short(B, self.Hq, self.Hkv, self.d, self._code, self.bt_stride,
                                              0 if ptab is None else ptab.shape[1]))
            parts = {} if short else dict(plan=self.plan, num_parts=self.num_parts)
            self._calls[key] = [(binding.make_rotary_args(
                self.rotary, q[layer], k[layer], v[layer], self.positions,
                q_out=self.q_rots[layer, :B], k_out=self.k_rots[layer, :B],
                slot_mapping=self.slots, k_cache=self.k_caches[layer],
                v_cache=self.v_caches[layer], err=self.err), binding.make_shared_args(
                self.q_rots[layer, :B], self.k_caches[layer], self.v_caches[layer], self.tables,
                self.seq_lens, self.scale, self.outs[layer, :B], mass=self.masses[layer],
                scores=self.scores, decay=self.decay, workspace=self._space, flags=self.flags,
                err=self.err, **parts, **self._prefix_args))
                for layer in range(self.n_layers)]
        return self._calls[key]

    def _launch(self, B, q, k, v, attn_bias, stream):
        torch = self.torch
        if q.dim() == 3:
            q, k, v = q.unsqueeze(0), k.unsqueeze(0), v.unsqueeze(0)
        lens = self.last_metadata[2]
        known = np.array([self._known[s] for s in self._rows_now], np.int32)
        fresh = None
        if not np.array_equal(known, lens - 1):
            fresh = torch.from_numpy(known).to(self.device)
        calls = self._prepared(B, q, k, v)
        binding.set_rotary_inputs([rotary for rotary, _ in calls], q, k, v)
        for rotary, attend in calls:
            attend.mass_lens = None if fresh is None else fresh.data_ptr()
            binding.rotary_append_args(rotary, stream)
            binding.decode_attn_shared_args(attend, stream)

    def step(self, seq_ids, q, k, v, attn_bias=None, stream=None):
        """One decode step for the listed sequences (cutting back those at their bound
        first); returns ``out[:B]`` (with several layers, ``outs[:, :B]``)."""
        # (everything is checked before a sequence grows)
        seq_ids = [int(s) for s in seq_ids]
        if attn_bias is not None:
            raise ValueError("BoundedDecoder takes no additive mask")
        for s in seq_ids:
            if s not in self._prefix_of:
                raise binding.UnknownSequence(binding.ERR_UNKNOWN_SEQ, f"sequence {s} is not live")
        if len(set(seq_ids)) != len(seq_ids):
            raise ValueError("a sequence may be listed once")
        B, L = len(seq_ids), self.n_layers
        for t, heads in ((q, self.Hq), (k, self.Hkv), (v, self.Hkv)):
            if tuple(t.shape) not in ((L, B, heads, self.d),) + (((B, heads, self.d),) if L == 1 else ()):
                raise ValueError(f"shape {tuple(t.shape)}, expected [{L}, {B}, {heads}, {self.d}]")
            if t.dtype != self.tdtype or not t.is_cuda:
                raise ValueError(f"{t.dtype} on {t.device}, expected {self.tdtype} on the GPU")
        if not q.dim() == k.dim() == v.dim():
            raise ValueError("give q, k and v all with layers or all without")
        if B == 0:
            return self.out[:0] if L == 1 else self.outs[:, :0]
        for t, name in ((q, "q"), (k, "k"), (v, "v")):
            x = t if t.dim() == 3 else t[0]
            if binding._heads(x, name, B, self.d, self.tdtype, self.outs.device)[1] < x.shape[1] * self.d:
                raise ValueError(f"{name}: a row's heads overlap the next row's")
        torch = self.torch
        run = stream if stream is not None else torch.cuda.current_stream(self.device)
        with torch.cuda.stream(run):   # (copies and launches in one order)
            full = [s for s in seq_ids if self._held[s] >= self.budget + self.slack]
            if full:
                self.evict(full)
            self._prefix_state(seq_ids)
            try:
                out = super().step(seq_ids, q, k, v, None, run)
            except Exception:
                self._take_back(seq_ids, run)
                raise
        for s, n in zip(seq_ids, self.last_metadata[2].tolist()):
            self._known[s] = self._held[s] = n
        return out

    def _take_back(self, seq_ids, run):
        """After a step that raised: the tokens it counted but did not (everywhere) write."""
        if self._pending is not None:     # kernels launched before may read the buffer
            ev = self.torch.cuda.Event()
            ev.record(run)
            self._pending["event"], self._pending = ev, None
        # (a block that a token went into is its sequence's alone: nothing is to be copied)
        grown = [s for s in seq_ids if self.alloc.seq_len(s) > self._held[s]]
        self.alloc.truncate_many(grown, [self._held[s] for s in grown])

    def capture(self, *args, **kw):
        raise ValueError("BoundedDecoder changes its launches from step to step: not captured")

    capture_host = capture
