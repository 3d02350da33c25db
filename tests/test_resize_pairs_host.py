"""The moves of a pool that takes another size, asked for before it does (pkv_alloc_resize_pairs)."""
import ctypes

import numpy as np
import pytest


@pytest.fixture
def bind(host_lib):
    from paged_kv_decode_10_gb300 import binding
    return binding


def state(a):
    return a.free_stack(), a.num_blocks, [a.block_refs(b) for b in range(a.num_blocks)]


@pytest.mark.parametrize("seed", range(8))
def test_pairs_are_those_of_the_resize_that_follows(bind, seed):
    rng = np.random.default_rng(seed)
    a = bind.BlockAllocator(60, 12, 20, rng.permutation(60))
    live = []
    for turn in range(40):
        if live and rng.random() < 0.4:
            a.leave(live.pop(int(rng.integers(0, len(live)))))
        elif len(live) < 9:
            n = int(rng.integers(0, 150))
            if -(-n // 16) <= a.num_free():
                live.append(a.join(n))
                if n % 16 == 0:         # (its blocks belong to two sequences)
                    live += a.fork(live[-1], 1)[0].tolist()
        blocks = {s: a.seq_blocks(s) for s in live}
        used = {b for row in blocks.values() for b in row}
        size, before = int(rng.integers(max(1, len(used) - 3), 80)), state(a)
        if size < len(used):
            for call in (a.resize_pairs, a.resize):
                with pytest.raises(bind.OutOfBlocks):
                    call(size)
                assert state(a) == before
            continue
        src, dst = a.resize_pairs(size)
        assert state(a) == before and {s: a.seq_blocks(s) for s in live} == blocks
        assert sorted(src) == sorted(b for b in used if b >= size) and len(set(dst)) == len(dst)
        assert all(b < size and b not in used for b in dst)
        again = a.resize(size)
        assert again[0].tolist() == src.tolist() and again[1].tolist() == dst.tolist()
        to = dict(zip(src.tolist(), dst.tolist()))
        for s in live:
            assert a.seq_blocks(s) == [to.get(b, b) for b in blocks[s]]


def test_pairs_are_refused_like_the_resize(bind):
    a = bind.BlockAllocator(16, 3, 8)
    a.join(20)
    lib, n = bind.load(), ctypes.c_int32(-1)
    for call in (lib.pkv_alloc_resize_pairs, lib.pkv_alloc_resize):
        assert call(a._h, 14, None, None, 0, ctypes.byref(n)) == bind.ERR_INVALID_ARG
        assert n.value == 2 and a.num_free() == 14      # two blocks would move
        assert call(a._h, 0, None, None, 0, ctypes.byref(n)) == bind.ERR_INVALID_ARG
        assert call(a._h, 14, None, None, 0, None) == bind.ERR_INVALID_ARG
        assert call(None, 14, None, None, 0, ctypes.byref(n)) == bind.ERR_INVALID_ARG


def test_prepare_nodes_into_given_arrays(bind):
    a, b = (bind.BlockAllocator(20, 4, 8) for _ in range(2))
    for x in (a, b):
        assert [x.join(17), x.join(0)] == [0, 1]
    out = (np.empty(7, np.int32), np.empty(7, np.int64), np.empty(3, np.int32), np.empty(2, np.int32),
           np.empty((2, 8), np.int32))
    got = a.prepare_nodes([1, 0], [5, 2], 8, out=out)
    assert all(x is y for x, y in zip(got, out))
    for x, y in zip(out, b.prepare_nodes([1, 0], [5, 2], 8)):
        assert np.array_equal(x, y)
    short = (out[0][:6],) + out[1:]
    state = a.free_stack()
    with pytest.raises(bind.PkvError):
        a.prepare_nodes([1, 0], [5, 2], 8, out=short)
    assert a.free_stack() == state and a.seq_len(1) == 5
