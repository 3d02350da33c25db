"""Which of a sequence's blocks belong to others too (pkv_seqs_shared)."""
import ctypes

import numpy as np
import pytest


@pytest.fixture
def bind(host_lib):
    from paged_kv_decode_10_gb300 import binding
    return binding


def test_shared_blocks(bind):
    a = bind.BlockAllocator(40, 8, 10)
    s, t, empty = a.join(70), a.join(32), a.join(0)
    assert a.shared_blocks([s, t, empty]).tolist() == [0, 0, 0] and a.shared_blocks([]).tolist() == []
    (c,), _, _ = a.fork(s, 1)
    assert a.shared_blocks([s, c, t, s]).tolist() == [4, 4, 0, 4]      # (the last of 5 is its own)
    a.fork(t, 2)
    a.truncate_many([c], [35])                                         # a block of its own for 32..34
    assert a.shared_blocks([s, c, t]).tolist() == [2, 2, 2]
    a.leave(c)
    assert a.shared_blocks([s, t]).tolist() == [0, 2]


def test_refusals(bind):
    a = bind.BlockAllocator(8, 4, 4)
    s = a.join(5)
    for ids in ([c for c in (s, 3)], [-1], [4]):
        with pytest.raises(bind.UnknownSequence):
            a.shared_blocks(ids)
    one, p = np.array([s], np.int32), ctypes.POINTER(ctypes.c_int32)
    at = one.ctypes.data_as(p)
    for args in ((None, at, 1, at), (a._h, None, 1, at), (a._h, at, 1, None), (a._h, at, -1, at)):
        assert bind.load().pkv_seqs_shared(*args) == bind.ERR_INVALID_ARG
