"""``BoundedDecoder`` over sequences that share blocks with a fork: eviction, which moves tokens within
their blocks, is refused before anything has moved, and a step that raises is taken back."""
import numpy as np
import pytest
import torch

from helpers import dev
from paged_kv_decode_10_gb300 import binding, workloads
from paged_kv_decode_10_gb300.bounded import BoundedDecoder

pytestmark = pytest.mark.gpu

Hq, Hkv, d, L = 4, 2, 64, 2


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def normal(n, heads, seed):
    return workloads.normal((L, n, heads, d), "f32", seed).to(dev())


def make(lengths):
    dec = BoundedDecoder(40, Hq, Hkv, d, "f32", 6, budget=32, slack=16, sink=2, recent=4, n_layers=L,
                         device=dev())
    ids = [dec.join(n, k=normal(n, Hkv, 10 + n), v=normal(n, Hkv, 50 + n)) for n in lengths]
    return dec, ids


def state(dec, ids):
    torch.cuda.synchronize()
    return ([x.clone() for x in (dec.k_caches, dec.v_caches, dec.masses)],
            (dec.alloc.free_stack(), [(dec.alloc.seq_blocks(s), dec.alloc.seq_len(s), dec.alloc.offset(s))
                                      for s in ids], dict(dec._known), dict(dec._held)))


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a[0], b[0])) and a[1] == b[1]


def step(dec, ids, seed):
    n = len(ids)
    return dec.step(ids, normal(n, Hq, seed), normal(n, Hkv, seed + 1), normal(n, Hkv, seed + 2))


def test_an_eviction_of_shared_blocks_is_refused_before_anything_moves():
    dec, (s, t) = make([40, 35])
    for x in (dec.k_caches, dec.v_caches):            # (blocks of nobody compare as equal)
        x[torch.isnan(x)] = 0.0
    (child,), src, dst = dec.alloc.fork(s, 1)
    binding.copy_blocks([c[i] for c in (dec.k_caches, dec.v_caches) for i in range(L)],
                        *(torch.from_numpy(b).to(dev()) for b in (src, dst)))
    before = state(dec, [s, t, child])
    for ids in ([s], [t, s]):
        with pytest.raises(binding.PkvError):
            dec.evict(ids, keep=16)
        assert same(state(dec, [s, t, child]), before)
    dec.evict([s], keep=40)                           # gets no shorter: nothing to refuse
    assert dec.alloc.seq_len(s) == 40
    dec.evict([t], keep=16)                           # shares nothing
    assert dec.alloc.seq_len(t) == 16
    dec.alloc.leave(child)
    dec.evict([s], keep=16)
    assert dec.alloc.seq_len(s) == 16 and dec.device_errors() == 0


def test_a_step_at_the_bound_of_a_shared_sequence_changes_nothing():
    dec, (s, t) = make([47, 20])
    for x in (dec.k_caches, dec.v_caches):
        x[torch.isnan(x)] = 0.0
    step(dec, [s, t], 70)                             # 48 tokens, whole blocks
    (child,), src, _ = dec.alloc.fork(s, 1)
    assert len(src) == 0
    before = state(dec, [s, t, child])
    with pytest.raises(binding.PkvError):
        step(dec, [t, s], 80)
    assert same(state(dec, [s, t, child]), before)
    dec.alloc.leave(child)
    step(dec, [t, s], 80)
    assert dec.alloc.seq_len(s) == 33 and dec.alloc.seq_len(t) == 22 and dec.device_errors() == 0


def test_a_step_that_raises_is_taken_back_where_blocks_are_shared(monkeypatch):
    dec, (s, t) = make([32, 20])
    (child,), src, _ = dec.alloc.fork(s, 1)
    assert len(src) == 0
    positions = [dec.alloc.offset(x) for x in (s, t)]
    free = sorted(dec.alloc.free_stack())

    def raises(*args, **kw):
        raise RuntimeError("planted")
    with monkeypatch.context() as m:
        m.setattr(binding, "decode_attn_shared_args", raises)
        with pytest.raises(RuntimeError):
            step(dec, [s, t], 60)
    assert [dec.alloc.seq_len(x) for x in (s, t, child)] == [32, 20, 32]
    assert [dec.alloc.offset(x) for x in (s, t)] == positions and sorted(dec.alloc.free_stack()) == free
    alone, ids = make([32, 20])
    assert torch.equal(step(dec, [s, t], 60), step(alone, ids, 60))
    assert dec.device_errors() == 0
