"""``DraftDecoder.accept`` that raises has moved nothing, so that it can be called again."""
import pytest
import torch

from helpers import dev
from paged_kv_decode_10_gb300 import binding, workloads
from paged_kv_decode_10_gb300.drafted import DraftDecoder

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def drafted_batch():
    dec = DraftDecoder(20, 4, 2, 64, "f32", 4, 8, device=dev(), n_layers=2)
    x = workloads.normal((2, 40, 8, 64), "f32", 5).to(dev())
    q, k, v = x[:, :, :4], x[:, :, 4:6], x[:, :, 6:]
    ids = [dec.join(n, k[:, :n], v[:, :n]) for n in (30, 7)]
    dec.verify(ids, [6, 3], q[:, 30:39], k[:, 30:39], v[:, 30:39], parents=[-1, 0, 0, 1, 2, 4, -1, 0, 0])
    return dec, ids, [t[:, :2].contiguous() for t in (q, k, v)]


def test_an_accept_that_raises_can_be_called_again(monkeypatch):
    paths = [[0, 2, 4, 5], [0, 2]]
    twin, ids, step = drafted_batch()
    twin.accept(paths)
    want = twin.step(ids, *step)
    dec, ids, step = drafted_batch()
    torch.cuda.synchronize()
    before = [c.clone().view(torch.int32) for c in (dec.k_caches, dec.v_caches)]
    real, calls = binding.make_accept_args, []

    def second_fails(*args, **kw):
        calls.append(args)
        if len(calls) == 2:
            raise torch.cuda.OutOfMemoryError("planted")
        return real(*args, **kw)
    with monkeypatch.context() as m:
        m.setattr(binding, "MAX_POOLS", 2)
        m.setattr(binding, "make_accept_args", second_fails)
        with pytest.raises(torch.cuda.OutOfMemoryError):
            dec.accept(paths)
    torch.cuda.synchronize()
    for x, c in zip(before, (dec.k_caches, dec.v_caches)):
        assert torch.equal(x, c.view(torch.int32))
    assert [dec.alloc.seq_len(s) for s in ids] == [36, 10]
    with pytest.raises(ValueError):
        dec.step(ids, *step)
    dec.accept(paths)
    assert [dec.alloc.seq_len(s) for s in ids] == [34, 9]
    assert torch.equal(dec.step(ids, *step), want) and dec.device_errors() == 0
