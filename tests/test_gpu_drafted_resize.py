"""``DraftDecoder.resize`` that raises changes nothing: not the allocator, not the caches, not what the
next steps give."""
import numpy as np
import pytest
import torch

from helpers import dev
from paged_kv_decode_10_gb300 import binding, workloads
from paged_kv_decode_10_gb300.drafted import DraftDecoder

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def batch(dtype):
    """A decoder whose sequences lie all over its pool, and what one step of them takes."""
    Hq, Hkv, d, L = 4, 2, 64, 2
    order = np.random.default_rng(5).permutation(40)
    dec = DraftDecoder(40, Hq, Hkv, d, dtype, 6, 10, device=dev(), n_layers=L, initial_free=order)
    x = workloads.normal((L, 150, Hq + 2 * Hkv, d), dtype, 3).to(dev())
    k, v = x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    ids = [dec.join(n, k[:, :n], v[:, :n]) for n in (150, 33, 64)]
    ids += dec.fork(ids[2])
    step = x[:, :4, :Hq].contiguous(), k[:, 4:8].contiguous(), v[:, 8:12].contiguous()
    return dec, ids, step


def state(dec, ids):
    return (dec.num_blocks, dec.alloc.num_blocks, dec.alloc.free_stack(), [dec.alloc.seq_blocks(s) for s in ids],
            [dec.alloc.seq_len(s) for s in ids], dec.k_caches.data_ptr(), dec.v_caches.data_ptr(),
            dec.k_cache.data_ptr(), dec.v_cache.data_ptr())


def raises(*args, **kw):
    raise torch.cuda.OutOfMemoryError("planted")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [19, 39, 80])
@pytest.mark.parametrize("where", ["upload", "second launch", "allocator"])
def test_a_resize_that_raises_changes_nothing(where, size, dtype, monkeypatch):
    twin, ids, step = batch(dtype)
    want = [twin.step(ids, *step) for _ in range(3)]
    dec, ids, step = batch(dtype)
    before = state(dec, ids)
    with monkeypatch.context() as m:
        if where == "upload":
            m.setattr(dec, "_upload", raises)
        elif where == "allocator":
            m.setattr(dec.alloc, "resize", raises)
        else:
            real, calls = binding.copy_blocks_args, []

            def second_fails(args, stream=None):
                calls.append(args)
                if len(calls) == 2:
                    raises()
                real(args, stream)
            m.setattr(binding, "MAX_POOLS", 1)       # (a launch for every pool)
            m.setattr(binding, "copy_blocks_args", second_fails)
        with pytest.raises(torch.cuda.OutOfMemoryError):
            dec.resize(size)
    assert state(dec, ids) == before
    assert torch.equal(dec.step(ids, *step), want[0])
    dec.resize(size)
    assert dec.num_blocks == dec.alloc.num_blocks == dec.k_caches.shape[1] == size
    for w in want[1:]:
        assert torch.equal(dec.step(ids, *step), w)
    assert dec.device_errors() == 0
