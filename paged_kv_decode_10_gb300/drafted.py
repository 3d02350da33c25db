"""Several tokens a row and step: ``DraftDecoder``.

A step verifies a tree of drafted tokens for every row (``verify``), after which each row
keeps the path that was accepted (``accept``), or appends a chunk of a prompt (``extend``; a
single token: ``step``).  Sequences fork (``fork``: several samples of one prompt share its
blocks), and the pool takes another size while sequences live (``resize``).  Tokens may have
positions on several axes (a ``binding.Rotary`` with sections).

Positions that a call does not name count tokens: those held, the sequence's offset and the
depth, the same on every axis.  Where earlier tokens were placed otherwise (the patches of an
image or a video share positions, so that text behind them goes on from the largest one, below
the number of tokens), every later ``verify``, ``extend`` and ``step`` has to name its own.

A step is a0 on the host (``pkv_prepare_nodes``), one copy of its metadata to the GPU, then per
layer ``pkv_rotary_append`` and ``pkv_decode_attn_tree``; ``accept`` is ``pkv_tree_accept`` over
all layers, then ``pkv_seqs_truncate`` on the host.  A call on another stream than the call
before waits for that one's; what the caller hands in is ready on the stream that it names.
"""
import math

import numpy as np

from . import binding
from .engine import PagedDecoder


def _int32(x, name):
    """Whole numbers of 32 bits (of any type that holds them) as a dense int32 array."""
    x = np.asarray(x)
    if x.dtype != np.int32 and x.size:
        whole = x.dtype.kind in "iu" or x.dtype.kind == "f" and bool((np.isfinite(x) & (x == np.rint(x))).all())
        if not whole or int(x.min()) < -2**31 or int(x.max()) >= 2**31:
            raise ValueError(f"{name}: expected whole numbers of 32 bits")
    return np.ascontiguousarray(x, np.int32)


def _words(x):
    """Mask words (signed or not) as a dense int32 array of the same bits."""
    x = np.asarray(x)
    if x.dtype != np.int32 and x.size:
        if x.dtype.kind not in "iu" or int(x.min()) < -2**31 or int(x.max()) >= 2**32:
            raise ValueError(f"mask: {x.dtype}, expected words of 32 bits")
        x = (x.astype(np.int64) & 0xffffffff).astype(np.uint32).view(np.int32)
    return np.ascontiguousarray(x, np.int32)


class DraftDecoder(PagedDecoder):
    """``rotary``: a ``binding.Rotary`` (default: the whole head, plain, at ``rope_base``).  The
    rest as ``PagedDecoder``; its captured forms, additive masks, partitions (``num_parts``,
    ``plan``, ``layer_merge_helpers``) and flags other than ``ATTN_SHORT_WAITS`` are not
    offered here."""

    served = False

    def __init__(self, num_blocks, Hq, Hkv, d, dtype, max_seqs, max_blocks_per_seq, rotary=None, **kw):
        import torch
        for name in ("num_parts", "plan", "layer_merge_helpers", "metadata"):
            if kw.get(name) is not None:
                raise ValueError(f"{name} has no meaning here")
        if kw.get("flags", 0) & ~binding.ATTN_SHORT_WAITS:
            raise ValueError(f"flags {kw['flags']}: only ATTN_SHORT_WAITS")
        if not math.isfinite(kw.get("scale") or 0.0):
            raise ValueError("scale must be finite")
        if rotary is not None and kw.get("rope_base") is not None:
            raise ValueError("rotary states its own base: give rope_base or rotary")
        if rotary is not None and rotary.d != d:
            raise ValueError(f"rotary was made for heads of {rotary.d}, not {d}")
        super().__init__(num_blocks, Hq, Hkv, d, dtype, max_seqs, max_blocks_per_seq, **kw)
        self.rotary = binding.Rotary(d, base=self.rope_base) if rotary is None else rotary
        code = binding.F32 if dtype == "f32" else binding.BF16
        self.space = torch.empty(binding.tree_workspace_bytes(Hq, Hkv, d, code), dtype=torch.uint8,
                                 device=self.device)
        # of the last verify: sequences (None: left since), lengths before, nodes, device
        # metadata, stream
        self._drafted = None
        self._last = torch.cuda.current_stream(self.device)   # stream of the last call
        self._waiting = set()       # sequences that hold drafted tokens
        self._pinned = [[None, None], [None, None]]   # host buffer, event of its last copy

    # -- helpers ------------------------------------------------------------------
    def _on(self, stream):
        """The stream of a call as torch's current one, so that copies, small tensors and
        launches are ordered, behind what the call before launched on another."""
        torch = self.torch
        now = stream if stream is not None else torch.cuda.current_stream(self.device)
        if now != self._last:
            now.wait_stream(self._last)
            self._last = now
        return torch.cuda.stream(now)

    def device_errors(self):
        """As ``PagedDecoder``'s, behind the last call on whichever stream it ran."""
        with self._on(None):
            return super().device_errors()

    def _upload(self, arrays):
        """Device copies of numpy arrays (int64 ones first), by one copy on the current
        stream out of page-locked memory."""
        torch = self.torch
        ends = np.cumsum([a.nbytes for a in arrays])
        slot = self._pinned[0]
        self._pinned.reverse()
        if slot[1] is not None:
            slot[1].synchronize()
        if slot[0] is None or slot[0].numel() < ends[-1]:
            slot[0] = torch.empty(max(4096, int(ends[-1]) * 2), dtype=torch.uint8, pin_memory=True)
        host = slot[0].numpy()
        for a, e in zip(arrays, ends):
            host[e - a.nbytes:e] = a.reshape(-1).view(np.uint8)
        dev = torch.empty(int(ends[-1]), dtype=torch.uint8, device=self.device)
        dev.copy_(slot[0][:int(ends[-1])], non_blocking=True)
        slot[1] = torch.cuda.Event()
        slot[1].record()
        types = {np.dtype(np.int32): torch.int32, np.dtype(np.int64): torch.int64}
        return [dev[int(e) - a.nbytes:int(e)].view(types[a.dtype]).view(a.shape)
                for a, e in zip(arrays, ends)]

    def _pools(self):
        return [c[layer] for layer in range(self.n_layers) for c in (self.k_caches, self.v_caches)]

    def _copy(self, src, dst, to=None):
        """Copies blocks in every layer (of one pool, or into the pools ``to``)."""
        if not len(src):
            return
        pools = self._pools()
        s, d = self._upload([np.ascontiguousarray(src, np.int32), np.ascontiguousarray(dst, np.int32)])
        for i in range(0, len(pools), binding.MAX_POOLS):
            n = i + binding.MAX_POOLS
            binding.copy_blocks_args(binding.make_copy_args(
                pools[i:n], s, d, None if to is None else to[i:n], self.err))

    def _settled(self, seq_ids):
        seq_ids = [int(s) for s in seq_ids]
        for s in seq_ids:
            if s in self._waiting:
                raise ValueError(f"sequence {s} holds drafted tokens: accept them first")
        return seq_ids

    def _axes(self, positions, T):
        """Positions ``[T]`` or ``[axes,T]`` (numpy int32) as the rotary takes them."""
        n = self.rotary.n_axes
        positions = _int32(positions, "positions")
        if n is None:
            if positions.shape != (T,):
                raise ValueError(f"positions {positions.shape}, expected [{T}]")
        elif positions.shape == (T,):
            positions = np.ascontiguousarray(np.broadcast_to(positions, (n, T)))
        elif positions.shape != (n, T):
            raise ValueError(f"positions {positions.shape}, expected [{n}, {T}]")
        return positions

    # -- sequences ------------------------------------------------------------------
    def join(self, prefix_len=0, k=None, v=None, positions=None, stream=None):
        """A new sequence of ``prefix_len`` tokens; ``k, v`` ``[n,Hkv,d]`` (``[L,n,Hkv,d]``
        with layers) hold their raw keys and values, at ``positions`` (default 0..n-1).
        Without them the caller writes the blocks."""
        n = int(prefix_len)
        if (k is None) != (v is None) or k is not None and (v.shape != k.shape or k.shape[-3] != n):
            raise ValueError("k and v must hold prefix_len tokens")
        if k is not None and (k.shape[0] if k.dim() == 4 else 1) != self.n_layers:
            raise ValueError(f"k and v must hold {self.n_layers} layers")
        if k is not None:
            pos = self._axes(np.arange(n) if positions is None else positions, n)
        sid = self.alloc.join(n)
        try:
            if k is not None and n:
                k, v = (t.unsqueeze(0) if t.dim() == 3 else t for t in (k, v))
                with self._on(stream):
                    slots, pos = self._upload([self.alloc.seq_slots(sid, 0, n)[1], pos])
                    for layer in range(self.n_layers):
                        binding.rotary_append_args(binding.make_rotary_args(
                            self.rotary, None, k[layer], v[layer], pos, slot_mapping=slots,
                            k_cache=self.k_caches[layer], v_cache=self.v_caches[layer], err=self.err))
        except Exception:
            self.alloc.leave(sid)
            raise
        return sid

    def leave(self, seq_id):
        self.alloc.leave(seq_id)
        if seq_id in self._waiting:
            self._waiting.discard(seq_id)
            rows = self._drafted[0]
            rows[rows.index(seq_id)] = None

    def fork(self, seq_id, n=1, stream=None):
        """``n`` new sequences that go on from this one; they share its whole blocks."""
        self._settled([seq_id])
        ids, src, dst = self.alloc.fork(seq_id, n)
        with self._on(stream):
            try:
                self._copy(src, dst)
            except Exception:
                self.alloc.leave_many(ids)
                raise
        return [int(s) for s in ids]

    def resize(self, num_blocks, stream=None):
        """Another size of the pool: new caches, into which the blocks in use are copied
        (those beyond a smaller pool onto free places).  The old caches are let go.  A call that
        raises changes nothing."""
        torch = self.torch
        if self._waiting:
            raise ValueError("drafted tokens are to be accepted first")
        num_blocks = int(num_blocks)
        with self._on(stream):
            shape = (self.n_layers, num_blocks) + tuple(self.k_caches.shape[2:])
            moved, onto = self.alloc.resize_pairs(num_blocks)
            used = set(range(self.num_blocks)) - set(self.alloc.free_stack())
            stay = np.array(sorted(used - set(moved.tolist())), np.int32)
            k, v = (torch.empty(shape, dtype=self.tdtype, device=self.device) for _ in range(2))
            self._copy(np.concatenate([stay, moved]), np.concatenate([stay, onto]),
                       [c[layer] for layer in range(self.n_layers) for c in (k, v)])
            # (the allocator follows once nothing can raise any more)
            self.alloc.resize(num_blocks)
            for c in (self.k_caches, self.v_caches):   # (not another's before the copy has read it)
                c.record_stream(torch.cuda.current_stream(self.device))
        self.k_caches, self.v_caches, self.num_blocks = k, v, num_blocks
        self.k_cache, self.v_cache = k[0], v[0]

    # -- steps ----------------------------------------------------------------------
    def _inputs(self, q, k, v, T):
        L = self.n_layers
        for t, heads in ((q, self.Hq), (k, self.Hkv), (v, self.Hkv)):
            if tuple(t.shape) not in ((L, T, heads, self.d),) + (((T, heads, self.d),) if L == 1 else ()):
                raise ValueError(f"shape {tuple(t.shape)}, expected [{L}, {T}, {heads}, {self.d}]")
            if t.dtype != self.tdtype or not t.is_cuda:
                raise ValueError(f"{t.dtype} on {t.device}, expected {self.tdtype} on the GPU")
        if not q.dim() == k.dim() == v.dim():
            raise ValueError("give q, k and v all with layers or all without")
        return tuple(t.unsqueeze(0) if t.dim() == 3 else t for t in (q, k, v))

    def _run(self, seq_ids, counts, q, k, v, mask, depths, positions, stream):
        """Appends ``counts[b]`` tokens to each row and attends; ``(out, lengths before,
        metadata on the device)``."""
        torch = self.torch
        L, T = self.n_layers, int(counts.sum())
        q, k, v = self._inputs(q, k, v, T)
        if positions is not None:
            positions = self._axes(positions, T)
        with self._on(stream):
            out = torch.empty((L, T, self.Hq, self.d), dtype=self.tdtype, device=self.device)
            if T == 0:
                return out[0] if L == 1 else out, None, None
            q_rot = torch.empty_like(out[0])
            before = [self.alloc.seq_len(s) for s in seq_ids]
            pos, slots, starts, lens, tables = self.alloc.prepare_nodes(seq_ids, counts, self.bt_stride,
                                                                        depths)
            try:
                pos = self._axes(pos if positions is None else positions, T)
                slots, pos, starts, lens, tables, *bits = self._upload(
                    [slots, pos, starts, lens, tables] + ([] if mask is None else [mask]))
                for layer in range(L):
                    binding.rotary_append_args(binding.make_rotary_args(
                        self.rotary, q[layer], k[layer], v[layer], pos, q_out=q_rot, slot_mapping=slots,
                        k_cache=self.k_caches[layer], v_cache=self.v_caches[layer], err=self.err))
                    binding.decode_attn_tree_args(binding.make_tree_args(
                        q_rot, self.k_caches[layer], self.v_caches[layer], tables, lens, starts,
                        self.scale, out[layer], mask=bits[0] if bits else None, workspace=self.space,
                        flags=self.flags, err=self.err))
            except Exception:
                self.alloc.truncate_many(seq_ids, before)
                raise
        return out[0] if L == 1 else out, before, (tables, lens, starts)

    def _counts(self, seq_ids, counts):
        counts = _int32(counts, "counts")
        if counts.shape != (len(seq_ids),) or (counts < 0).any():
            raise ValueError("one number of tokens per sequence, 0 or more")
        return counts

    def verify(self, seq_ids, counts, q, k, v, parents=None, depths=None, mask=None, positions=None,
               stream=None):
        """Attention of ``counts[b]`` drafted tokens of each listed sequence: ``q [T,Hq,d]``,
        ``k, v [T,Hkv,d]`` raw, row after row (``[L,T,...]`` with layers); returns the output in
        ``q``'s shape.  ``parents [T]``: the node of its own row that a token goes on from, or -1
        (None: the one before).  Instead of parents ``mask`` (int32 ``[T,words]`` of bits) and
        ``depths [T]`` may be given.  ``positions``: ``[T]`` or ``[axes,T]`` (default: the tokens
        ahead plus the depth, on every axis: not the place of text behind an image's patches).
        ``accept`` must follow."""
        if self._waiting:
            raise ValueError("the last verify's tokens are to be accepted first")
        seq_ids = self._settled(seq_ids)
        counts = self._counts(seq_ids, counts)
        T, starts = int(counts.sum()), np.concatenate([[0], np.cumsum(counts)])
        if parents is not None:
            if mask is not None or depths is not None:
                raise ValueError("give parents, or mask and depths")
            parents = _int32(parents, "parents").astype(np.int64)
            if parents.shape != (T,):
                raise ValueError(f"parents {parents.shape}, expected [{T}]")
            mask = binding.tree_mask(parents, starts)
            depths = np.zeros(T, np.int32)
            above = np.where(parents >= 0, parents + np.repeat(starts[:-1], counts), -1)
            up = above
            while (up >= 0).any():      # (a parent a turn)
                depths += up >= 0
                up = np.where(up >= 0, above[up], -1)
        elif mask is not None:
            mask = _words(mask)
            if mask.ndim != 2 or len(mask) != T or 32 * mask.shape[1] < counts.max(initial=0):
                raise ValueError(f"mask {mask.shape}, expected [{T}, words] with a bit for every node")
            if depths is None and positions is None:
                raise ValueError("a mask needs depths or positions")
        if depths is not None:
            depths = _int32(depths, "depths")
        out, before, meta = self._run(seq_ids, counts, q, k, v, mask, depths, positions, stream)
        run = stream if stream is not None else self.torch.cuda.current_stream(self.device)
        self._drafted = (seq_ids, before, counts, meta, run)
        self._waiting.update(s for s, n in zip(seq_ids, counts) if n)
        return out

    def accept(self, paths, stream=None):
        """Keeps ``paths[b]`` (ascending nodes, possibly none) of the row's drafted tokens, for
        the sequences of the last ``verify`` in their order (of one that has left since, the path
        counts for nothing); the other nodes are forgotten."""
        torch = self.torch
        if self._drafted is None:
            raise ValueError("no drafted tokens: verify comes first")
        seq_ids, before, counts, meta, run = self._drafted
        paths = [[int(i) for i in p] for p in paths]
        if len(paths) != len(seq_ids):
            raise ValueError("one path per sequence of the last verify")
        for p, n in zip(paths, counts):
            if any(not 0 <= i < n for i in p) or any(a >= b for a, b in zip(p, p[1:])):
                raise ValueError(f"path {p} does not ascend within {n} nodes")
        paths = [[] if s is None else p for s, p in zip(seq_ids, paths)]
        # (a path that is the first nodes stays where it is)
        if any(p != list(range(len(p))) for p in paths):
            path = np.full((len(paths), max(map(len, paths))), -1, np.int32)
            for b, p in enumerate(paths):
                path[b, :len(p)] = p
            kept = np.array([len(p) for p in paths], np.int32)
            pools = self._pools()
            with self._on(stream):
                now = torch.cuda.current_stream(self.device)
                if now != run:
                    for t in meta:
                        t.record_stream(now)
                path, kept = self._upload([path, kept])
                # (all calls are made before the first moves anything: moved tokens must not
                # move again when the caller tries once more)
                for call in [binding.make_accept_args(pools[i:i + binding.MAX_POOLS], *meta, path, kept,
                                                      self.err)
                             for i in range(0, len(pools), binding.MAX_POOLS)]:
                    binding.accept_nodes_args(call)
        rows = [b for b, (s, n) in enumerate(zip(seq_ids, counts)) if s is not None and n]
        self.alloc.truncate_many([seq_ids[b] for b in rows], [before[b] + len(paths[b]) for b in rows])
        self._waiting.clear()
        self._drafted = None

    def extend(self, seq_ids, counts, q, k, v, positions=None, stream=None):
        """Appends ``counts[b]`` tokens (a chunk of a prompt) to each listed sequence and
        attends, each token over all before it; they are kept.  Arguments as ``verify``."""
        seq_ids = self._settled(seq_ids)
        counts = self._counts(seq_ids, counts)
        return self._run(seq_ids, counts, q, k, v, None, None, positions, stream)[0]

    def step(self, seq_ids, q, k, v, attn_bias=None, stream=None, positions=None):
        """One token of each listed sequence."""
        if attn_bias is not None:
            raise ValueError("DraftDecoder takes no additive mask")
        return self.extend(seq_ids, np.ones(len(seq_ids), np.int32), q, k, v, positions, stream)

    def capture(self, *args, **kw):
        raise ValueError("DraftDecoder changes its launches from step to step: not captured")

    capture_host = capture
