"""Drafted tokens on the host: shared blocks, truncation, several tokens a row, another size of the
pool, trees' masks, rotary tables with axes, and what is refused."""
import ctypes

import numpy as np
import pytest

from oracle import drafted


@pytest.fixture
def bind(host_lib):
    from paged_kv_decode_10_gb300 import binding
    return binding


class Model:
    """The policy of include/pkv.h with plain lists: who has which block."""

    def __init__(self, n):
        self.free, self.rows, self.size = list(range(n)), {}, n   # rows: id -> [length, blocks]

    def refs(self, b):
        return sum(b in blocks for _, blocks in self.rows.values())

    def release(self, blocks):   # (their row no longer has them)
        self.free += [b for b in blocks if self.refs(b) == 0]

    def new_id(self):
        return min(set(range(len(self.rows) + 1)) - set(self.rows))

    def join(self, n):
        s = self.new_id()
        self.rows[s] = [n, [self.free.pop() for _ in range(-(-n // 16))]]
        return s

    def leave(self, s):
        self.release(self.rows.pop(s)[1])

    def append(self, s, n):
        L, blocks = self.rows[s]
        blocks += [self.free.pop() for _ in range(-(-(L + n) // 16) - len(blocks))]
        self.rows[s][0] = L + n
        return [blocks[t // 16] * 16 + t % 16 for t in range(L, L + n)]

    def fork(self, s, n):
        L, blocks = self.rows[s]
        ids, pairs = [], []
        for _ in range(n):
            c = self.new_id()
            mine = list(blocks)
            if L % 16:
                mine[-1] = self.free.pop()
                pairs.append((blocks[-1], mine[-1]))
            self.rows[c] = [L, mine]
            ids.append(c)
        return ids, pairs

    def truncate(self, ids, lens):
        pairs = []
        for s, n in zip(ids, lens):
            L, blocks = self.rows[s]
            if n % 16 and n < L and self.refs(blocks[n // 16]) > 1:
                b = self.free.pop()
                pairs.append((blocks[n // 16], b))
                blocks[n // 16] = b
        for s, n in zip(ids, lens):
            L, blocks = self.rows[s]
            gone = blocks[-(-n // 16):]
            self.rows[s] = [n, blocks[:-(-n // 16)]]
            self.release(gone)
        return pairs

    def resize(self, n):
        pairs = []
        if n >= self.size:
            self.free += list(range(self.size, n))
        else:
            self.free = [b for b in self.free if b < n]
            to = {}
            for s in sorted(self.rows):
                blocks = self.rows[s][1]
                for j, b in enumerate(blocks):
                    if b >= n:
                        if b not in to:
                            to[b] = self.free.pop()
                            pairs.append((b, to[b]))
                        blocks[j] = to[b]
        self.size = n
        return pairs


def same(a, m):
    assert a.free_stack() == m.free and a.num_free() == len(m.free)
    for s, (L, blocks) in m.rows.items():
        assert a.seq_len(s) == L and a.seq_blocks(s) == blocks
    for b in range(m.size):
        assert a.block_refs(b) == m.refs(b)
    used = [b for b in range(m.size) if m.refs(b)]
    assert sorted(m.free + used) == list(range(m.size))
    for L, blocks in m.rows.values():          # what is appended to is its row's alone
        assert L % 16 == 0 or m.refs(blocks[-1]) == 1


@pytest.mark.parametrize("seed", range(6))
def test_random_life_of_an_allocator(bind, seed):
    rng = np.random.default_rng(seed)
    a, m = bind.BlockAllocator(60, 12, 20), Model(60)
    refused = 0
    for _ in range(300):
        op = rng.choice(["join", "leave", "nodes", "fork", "truncate", "resize", "step"])
        live = sorted(m.rows)
        try:
            if op == "join":
                n = int(rng.integers(0, 120))
                if len(live) < 12 and -(-n // 16) <= len(m.free):
                    assert a.join(n) == m.join(n)
                else:
                    with pytest.raises(bind.PkvError):
                        a.join(n)
            elif not live:
                continue
            elif op == "leave":
                s = int(rng.choice(live))
                a.leave(s)
                m.leave(s)
            elif op in ("nodes", "step"):
                ids = [int(s) for s in rng.permutation(live)[:3]]
                counts = [int(rng.integers(0, 40)) if op == "nodes" else 1 for _ in ids]
                before = [m.rows[s][0] for s in ids]
                need = [-(-(L + n) // 16) for L, n in zip(before, counts)]
                if max(need) > 20 or sum(need) - sum(len(m.rows[s][1]) for s in ids) > len(m.free):
                    refused += 1
                    with pytest.raises(bind.PkvError):
                        a.prepare_nodes(ids, counts, 20)
                elif op == "nodes":
                    pos, slots, starts, lens, tables = a.prepare_nodes(ids, counts, 20)
                    want = [m.append(s, n) for s, n in zip(ids, counts)]
                    assert slots.tolist() == sum(want, [])
                    assert starts.tolist() == [0] + np.cumsum(counts).tolist()
                    assert lens.tolist() == [m.rows[s][0] for s in ids]
                    assert pos.tolist() == [L + i for L, n in zip(before, counts) for i in range(n)]
                    for row, s in zip(tables, ids):
                        blocks = m.rows[s][1]
                        assert row.tolist() == blocks + [-1] * (20 - len(blocks))
                else:
                    _, slots, lens, _ = a.prepare_step(ids, 20)
                    assert slots.tolist() == [m.append(s, 1)[0] for s in ids]
            elif op == "fork":
                s, n = int(rng.choice(live)), int(rng.integers(0, 4))
                if len(live) + n > 12 or (m.rows[s][0] % 16 and n > len(m.free)):
                    refused += 1
                    with pytest.raises(bind.PkvError):
                        a.fork(s, n)
                else:
                    ids, src, dst = a.fork(s, n)
                    mids, pairs = m.fork(s, n)
                    assert ids.tolist() == mids and list(zip(src.tolist(), dst.tolist())) == pairs
            elif op == "truncate":
                ids = [int(s) for s in rng.permutation(live)[:4]]
                lens = [int(rng.integers(0, m.rows[s][0] + 1)) for s in ids]
                shared = sum(n % 16 != 0 and n < m.rows[s][0] and m.refs(m.rows[s][1][n // 16]) > 1
                             for s, n in zip(ids, lens))
                if shared > len(m.free):
                    refused += 1
                    with pytest.raises(bind.OutOfBlocks):
                        a.truncate_many(ids, lens)
                else:
                    src, dst = a.truncate_many(ids, lens)
                    assert list(zip(src.tolist(), dst.tolist())) == m.truncate(ids, lens)
                    assert not set(src) & set(dst)
            else:
                n = int(rng.integers(20, 90))
                if m.size - len(m.free) > n:
                    refused += 1
                    with pytest.raises(bind.OutOfBlocks):
                        a.resize(n)
                else:
                    src, dst = a.resize(n)
                    assert list(zip(src.tolist(), dst.tolist())) == m.resize(n)
                    assert a.num_blocks == n and (src >= n).all() and (dst < n).all()
        finally:
            same(a, m)
    assert refused


def test_depths_and_offsets_make_the_positions(bind):
    a = bind.BlockAllocator(16, 4, 8)
    s, t = a.join(17), a.join(0)
    a.set_offset(s, 100)
    pos, _, starts, lens, _ = a.prepare_nodes([t, s], [2, 4], 8, depths=[0, 1, 0, 1, 1, 2])
    assert pos.tolist() == [0, 1, 117, 118, 118, 119] and starts.tolist() == [0, 2, 6]
    assert lens.tolist() == [2, 21]
    a.truncate_many([s], [19])
    assert a.prepare_step([s], 8)[0].tolist() == [119] and a.offset(s) == 100   # positions go back


def test_prepare_nodes_refuses_and_changes_nothing(bind):
    a = bind.BlockAllocator(8, 4, 4)
    s, t = a.join(30), a.join(1)
    state = a.free_stack()
    for ids, counts, kw in (([s, s], [1, 1], {}), ([s, 3], [1, 1], {}), ([s, t], [1, -1], {}),
                            ([s], [40], {}), ([s, t], [33, 64], {}), ([s], [2], dict(depths=[0, -1])),
                            ([s], [2], dict(depths=[0])), ([s], [1, 2], {}), ([s], [3], dict(bt=2))):   # (33 tokens need three entries)
        bt = kw.pop("bt", 4)
        with pytest.raises(bind.PkvError):
            a.prepare_nodes(ids, counts, bt, **kw)
        assert a.free_stack() == state and a.seq_len(s) == 30 and a.seq_len(t) == 1
    a.set_offset(t, 2**31 - 3)
    with pytest.raises(bind.PkvError):
        a.prepare_nodes([t], [3], 4)
    assert a.prepare_nodes([t], [2], 4)[0].tolist() == [2**31 - 2, 2**31 - 1]
    assert a.prepare_nodes([], [], 4)[2].tolist() == [0]


def test_sequences_that_share_blocks_are_not_evicted(bind):
    a = bind.BlockAllocator(16, 4, 8)
    s = a.join(40)
    (c,), _, _ = a.fork(s, 1)
    for x in (s, c):
        with pytest.raises(bind.PkvError):
            a.evict_many([x], [20])
        a.evict_many([x], [40])        # gets no shorter: nothing to refuse
    a.leave(c)
    a.evict_many([s], [20])
    assert a.seq_len(s) == 20


def test_cached_tables_follow_truncation_and_resize(bind):
    a = bind.BlockAllocator(20, 4, 8)
    s = a.join(40)
    out = (np.empty(1, np.int32), np.empty(1, np.int64), np.empty(1, np.int32), np.empty((1, 8), np.int32))
    state = np.full(3, -1, np.int32)

    def step():
        a.prepare_step_cached([s], 8, out, state)
        blocks = a.seq_blocks(s)
        assert out[3][0].tolist() == blocks + [-1] * (8 - len(blocks))
    step()
    a.truncate_many([s], [5])
    step()
    a.join(60)
    a.resize(8)
    step()


def test_list_and_size_refusals(bind):
    a = bind.BlockAllocator(16, 3, 8)
    s = a.join(20)
    for call in (lambda: a.truncate_many([s], [21]), lambda: a.truncate_many([s], [-1]),
                 lambda: a.truncate_many([s, s], [1, 1]), lambda: a.truncate_many([2], [0]),
                 lambda: a.truncate_many([s], [1, 2]), lambda: a.fork(s, 3), lambda: a.fork(2, 1),
                 lambda: a.fork(s, -1), lambda: a.resize(0), lambda: a.resize(1),
                 lambda: a.block_refs(16), lambda: a.block_refs(-1)):
        state = a.free_stack(), a.seq_blocks(s), a.seq_len(s)
        with pytest.raises((bind.PkvError, ValueError)):
            call()
        assert (a.free_stack(), a.seq_blocks(s), a.seq_len(s)) == state
    lib, n = bind.load(), ctypes.c_int32(-1)
    assert lib.pkv_alloc_resize(a._h, 14, None, None, 0, ctypes.byref(n)) == bind.ERR_INVALID_ARG
    assert n.value == 2 and a.num_blocks == 16     # two blocks would move
    assert lib.pkv_seq_fork(a._h, s, 1, np.empty(1, np.int32).ctypes.data_as(bind._p_i32), None, None,
                            ctypes.byref(n)) == bind.ERR_INVALID_ARG


# --------------------------------------------------------------------------- masks and tables
def test_tree_mask(bind):
    parents = [-1, 0, 0, 1, 3, -1, -1, 0]
    starts = [0, 5, 5, 8]
    words = bind.tree_mask(parents, starts)
    assert words.shape == (8, 1) and words.dtype == np.int32
    assert words[:, 0].tolist() == [1, 3, 5, 11, 27, 1, 2, 5]
    deep = bind.tree_mask(np.arange(70) - 1, [0, 70])
    assert deep.shape == (70, 3)
    sees = drafted.tree_visible(deep, 0, 70, 0)
    assert (sees == np.tril(np.ones((70, 70), bool))).all()
    for bad in ([0], [-2], [-1, 1], [-1, 5]):
        with pytest.raises(bind.PkvError):
            bind.tree_mask(bad, [0, len(bad)])


def turns_of(f):
    return int(np.ldexp(f / (2 * np.pi), 64))


@pytest.mark.parametrize("order", ["blocked", "cyclic"])
@pytest.mark.parametrize("ladder", ["shared", "own"])
@pytest.mark.parametrize("sections", [(16, 24, 24), (5, 0, 3), (64,), (1,) * 8])
def test_rotary_axes_tables(bind, sections, order, ladder):
    rot = bind.Rotary(128, rot_dim=2 * sum(sections), sections=sections, order=order, ladder=ladder)
    axis, number = drafted.axes_of(sections, order)
    assert rot.n_axes == len(sections) and list(rot.axes.axis)[:len(axis)] == axis
    for i, (a, k) in enumerate(zip(axis, number)):
        f = 10000.0 ** (-k / sections[a]) if ladder == "own" else 10000.0 ** (-i / sum(sections))
        assert abs(rot.table.turns[i] - turns_of(f)) <= 2.0**-50 * 2**64 * f
    if ladder == "shared":
        plain = bind.Rotary(128, rot_dim=2 * sum(sections))
        assert list(plain.table.turns) == list(rot.table.turns)


def test_rotary_axes_refuse(bind):
    for kw in (dict(sections=(16, 16)), dict(sections=()), dict(sections=(64, -1, 1)),
               dict(sections=(8,) * 9, rot_dim=128), dict(sections=(64,), order="else"),
               dict(sections=(64,), ladder="else"), dict(sections=(63, 1), scaling="ntk", ladder="own",
                                                         factor=2.0)):
        with pytest.raises(bind.PkvError):
            bind.Rotary(128, **kw)


# --------------------------------------------------------------------------- device calls, refused
def fake(n=1 << 20):
    return 256 * (n // 256)


def tree_args(bind, **kw):
    a = bind.TreeArgs()
    base = dict(q_rot=fake(), k_cache=fake(1 << 24), v_cache=fake(1 << 25), block_tables=fake(), seq_lens=fake(),
                node_starts=fake(), mask=fake(), workspace=fake(), workspace_bytes=1 << 40,
                out=fake(1 << 26), num_blocks=4, bt_stride=2, mask_words=1, B=1, T=4, Hq=8, Hkv=2, d=64,
                dtype=1, flags=0, scale=0.1)
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("bad", [
    dict(q_rot=None), dict(k_cache=None), dict(node_starts=None), dict(out=None), dict(workspace=None),
    dict(B=-1), dict(B=65537), dict(T=-1), dict(Hq=6), dict(Hq=32), dict(Hkv=0), dict(d=96), dict(dtype=2),
    dict(flags=1), dict(flags=16), dict(scale=float("nan")), dict(scale=float("inf")), dict(num_blocks=0),
    dict(bt_stride=0), dict(bt_stride=1 << 26), dict(mask_words=0), dict(mask_words=-1),
    dict(q_rot=8 + (1 << 20)), dict(out=1 << 20), dict(out=(1 << 20) + 512), dict(k_cache=(1 << 24) + 4),
    dict(num_blocks=1 << 27)])
def test_tree_call_refuses_before_it_reaches_the_gpu(bind, bad):
    rc = bind.load().pkv_decode_attn_tree(ctypes.byref(tree_args(bind, **bad)), None)
    assert rc in (bind.ERR_INVALID_ARG, bind.ERR_UNSUPPORTED)
    assert bind.load().pkv_last_error()


def test_tree_call_with_nothing_to_do(bind):
    for kw in (dict(B=0), dict(T=0)):
        assert bind.load().pkv_decode_attn_tree(ctypes.byref(tree_args(bind, **kw)), None) == bind.OK
    assert bind.load().pkv_decode_attn_tree(None, None) == bind.ERR_INVALID_ARG


def pointers(bind, *values):
    arr = (ctypes.c_void_p * len(values))(*values)
    return ctypes.cast(arr, ctypes.POINTER(ctypes.c_void_p)), arr


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(n_pools=-1), dict(n_pools=257), dict(src_blocks=None), dict(dst_blocks=None),
    dict(block_bytes=0), dict(block_bytes=24), dict(block_bytes=1 << 31), dict(n=2**31 - 1), dict(src_num_blocks=0), dict(dst_num_blocks=0),
    dict(dst=(1 << 20, 0)), dict(dst=(1 << 20, (1 << 21) + 8)), dict(dst=(1 << 20, 1 << 20)),
    dict(dst=(1 << 20, (1 << 20) + 64)), dict(dst=((1 << 21) + 64, 1 << 23)), dict(src=None), dict(dst=None)])
def test_copy_call_refuses(bind, bad):
    a, keep = bind.CopyArgs(), []
    base = dict(src=(1 << 20, 1 << 21), dst=(1 << 20, 1 << 21), src_blocks=256, dst_blocks=256, n=3,
                n_pools=2, block_bytes=64, src_num_blocks=8, dst_num_blocks=8)
    for k, v in {**base, **bad}.items():
        if k in ("src", "dst") and v is not None:
            v, arr = pointers(bind, *v)
            keep.append(arr)
        setattr(a, k, v)
    assert bind.load().pkv_copy_blocks(ctypes.byref(a), None) in (bind.ERR_INVALID_ARG, bind.ERR_UNSUPPORTED)


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(B=65537), dict(T=-1), dict(n_pools=-1), dict(n_pools=257), dict(path=None),
    dict(accept_lens=None), dict(block_tables=None), dict(Hkv=0), dict(d=0), dict(d=6), dict(dtype=9),
    dict(num_blocks=0), dict(num_blocks=1 << 27), dict(bt_stride=0), dict(path_stride=0),
    dict(pools=(1 << 20, (1 << 20) + 4096)), dict(pools=(1 << 20, 8)), dict(pools=(1 << 20, 0))])
def test_accept_call_refuses(bind, bad):
    a, keep = bind.AcceptArgs(), []
    base = dict(pools=(1 << 20, 1 << 24), block_tables=256, seq_lens=256, node_starts=256, path=256,
                accept_lens=256, n_pools=2, num_blocks=4, bt_stride=2, path_stride=3, B=1, T=4, Hkv=2, d=64,
                dtype=1)
    for k, v in {**base, **bad}.items():
        if k == "pools":
            v, arr = pointers(bind, *v)
            keep.append(arr)
        setattr(a, k, v)
    assert bind.load().pkv_tree_accept(ctypes.byref(a), None) in (bind.ERR_INVALID_ARG, bind.ERR_UNSUPPORTED)


def test_axes_call_refuses(bind):
    lib = bind.load()
    rot = bind.Rotary(64, sections=(16, 16))
    other = bind.Rotary(64, rot_dim=32, sections=(8, 8))
    a = bind.RotaryArgs()
    a.rotary = ctypes.pointer(rot.table)
    a.T, a.Hkv, a.d, a.dtype = 4, 1, 64, bind.F32
    a.k = a.k_out = a.positions = 1 << 20
    a.k_stride = a.k_out_stride = 64
    for axes, stride in ((None, 4), (bind.RotaryAxes(), 4), (other.axes, 4), (rot.axes, 3), (rot.axes, -4)):
        rc = lib.pkv_rotary_axes_append(ctypes.byref(a), None if axes is None else ctypes.byref(axes), stride,
                                        None)
        assert rc == bind.ERR_INVALID_ARG


def test_positions_near_the_limit_are_refused_not_wrapped(bind):
    """length + offset may pass 32 bits before the depth is added."""
    a = bind.BlockAllocator(16, 4, 8)
    s = a.join(20)
    for offset, count, good in ((2**31 - 1, 1, False), (2**31 - 21, 1, True), (2**31 - 22, 2, True),
                                (2**31 - 10, 2, False), (2**31 - 22, 5, False)):
        a.set_offset(s, offset)
        state = a.free_stack()
        if not good:
            for depths in (None, np.arange(count)):
                with pytest.raises(bind.PkvError):
                    a.prepare_nodes([s], [count], 8, depths)
                assert a.seq_len(s) == 20 and a.free_stack() == state
            continue
        pos = a.prepare_nodes([s], [count], 8)[0]
        assert pos.tolist() == [20 + offset + i for i in range(count)]
        a.truncate_many([s], [20])
