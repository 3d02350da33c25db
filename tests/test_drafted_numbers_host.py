"""What ``DraftDecoder`` takes as positions, depths and mask words: whole numbers of 32 bits, which
nothing rounds or wraps on the way."""
import numpy as np
import pytest


@pytest.fixture
def dec(host_lib):
    """A decoder up to its launches (none of which these calls reach)."""
    from paged_kv_decode_10_gb300 import binding
    from paged_kv_decode_10_gb300.drafted import DraftDecoder
    dec = DraftDecoder.__new__(DraftDecoder)
    dec.rotary, dec._waiting = binding.Rotary(64, sections=(12, 20)), set()
    dec.reached = []
    dec._run = lambda *args: dec.reached.append(args) or (None, None, None)
    dec.torch = type("torch", (), {"cuda": type("cuda", (), {"current_stream": staticmethod(lambda d: None)})})
    dec.device = None
    return dec


def test_positions(dec):
    for good in ([3, 2**31 - 1], np.array([-2**31, 5]), np.array([1, 2], np.uint8), np.array([[1, 2], [3, 4]], np.int64),
                 [3.0, 2**31 - 1]):
        got = dec._axes(good, 2)
        assert got.dtype == np.int32 and got.shape == (2, 2)
        assert got.tolist() == np.broadcast_to(np.asarray(good, np.int64), (2, 2)).tolist()
    assert dec._axes([], 0).shape == (2, 0)
    for bad in ([0.5, 1], [np.nan, 1], [np.inf, 1], [2.0**31, 1], [True, False], [2**31, 0], [-2**31 - 1, 0], np.array([2**63, 0], np.uint64)):
        with pytest.raises(ValueError):
            dec._axes(bad, 2)


def test_masks_and_depths(dec):
    call = lambda **kw: dec.verify([0], [2], None, None, None, **kw)
    call(mask=np.array([[1], [2**31 + 3]]), depths=[0, 1])
    _, _, _, _, _, mask, depths, _, _ = dec.reached[-1]
    assert mask.dtype == np.int32 and mask.tolist() == [[1], [3 - 2**31]] and depths.tolist() == [0, 1]
    for mask in (np.array([[-1], [3]]), np.array([[2**32 - 1], [3]], np.uint32), np.array([[-1], [3]], np.int8)):
        dec._waiting.clear()
        call(mask=mask, depths=[0, 1])
        assert dec.reached[-1][5].dtype == np.int32 and dec.reached[-1][5].tolist() == [[-1], [3]]
    n = len(dec.reached)
    seen = np.tril(np.ones((2, 2)))
    for kw in (dict(mask=seen.astype(bool), depths=[0, 1]), dict(mask=seen, depths=[0, 1]),
               dict(mask=[[1], [2**32]], depths=[0, 1]), dict(mask=[[1], [3]], depths=[0.0, 1.5]),
               dict(depths=[0, 2**32])):
        dec._waiting.clear()
        with pytest.raises(ValueError):
            call(**kw)
        assert len(dec.reached) == n


@pytest.mark.parametrize("L,given", [(1, (2,)), (2, (3,)), (2, (1,)), (2, ()), (3, (2,))])
def test_join_takes_keys_and_values_of_every_layer(dec, L, given):
    import torch
    from paged_kv_decode_10_gb300 import binding
    dec.n_layers, dec.alloc = L, binding.BlockAllocator(4, 2, 4)
    k = torch.zeros(given + (5, 2, 64))
    with pytest.raises(ValueError):
        dec.join(5, k, k)
    assert dec.alloc.num_free() == 4


def test_counts_and_parents(dec):
    call = lambda counts=(2,), **kw: dec.verify([0], counts, None, None, None, **kw)
    call(np.array([2], np.uint16), parents=np.array([-1, 0], np.int8))
    dec._waiting.clear()
    call([2.0], parents=[-1.0, 0.0])
    assert dec.reached[-1][5].tolist() == [[1], [3]] and dec.reached[-1][6].tolist() == [0, 1]
    n = len(dec.reached)
    for kw in (dict(counts=[2.5]), dict(counts=[2**32 + 2]), dict(counts=[True]),
               dict(parents=[-0.5, 0.5]), dict(parents=[-1, 2**32])):
        dec._waiting.clear()
        with pytest.raises(ValueError):
            call(**kw)
        assert len(dec.reached) == n
