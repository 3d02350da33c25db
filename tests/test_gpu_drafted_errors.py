"""``DraftDecoder.device_errors`` sees what the calls before it reported, on whichever stream they ran."""
import numpy as np
import pytest
import torch

from helpers import dev
from paged_kv_decode_10_gb300 import binding
from paged_kv_decode_10_gb300.drafted import DraftDecoder

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def test_errors_of_a_side_stream_are_read_and_cleared_behind_it(monkeypatch):
    dec = DraftDecoder(40, 8, 2, 64, "bf16", 4, 20, device=dev())
    s = dec.join(100)
    dec.k_caches.zero_()
    dec.v_caches.zero_()
    x = [torch.zeros((3, h, 64), dtype=torch.bfloat16, device=dev()) for h in (8, 2, 2)]
    real = dec.alloc.prepare_nodes

    def a_bad_block(*args, **kw):
        out = real(*args, **kw)
        out[4][0, 2] = 10**6                    # (the kernel checks it against the pool)
        return out
    dec.extend([s], [3], *x)                    # (kernels loaded, buffers made)
    side, busy = torch.cuda.Stream(), torch.randn(8192, 8192, device=dev())
    torch.cuda.synchronize()
    assert dec.device_errors() == 0
    for _ in range(3):
        with torch.cuda.stream(side):
            for _ in range(10):
                busy = busy @ busy * 1e-4
        with monkeypatch.context() as m:
            m.setattr(dec.alloc, "prepare_nodes", a_bad_block)
            dec.extend([s], [3], *x, stream=side)
        assert dec.device_errors() == binding.DEVERR_BAD_BLOCK
        torch.cuda.synchronize()
        assert int(dec.err) == 0
