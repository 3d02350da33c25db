"""``BoundedDecoder`` on the host: what it makes of its arguments and how it keeps its state,
with the device part of ``PagedDecoder`` replaced by plain attributes."""
import numpy as np
import pytest
import torch

from paged_kv_decode_10_gb300 import bounded


@pytest.fixture
def bind(host_lib):
    from paged_kv_decode_10_gb300 import binding
    return binding


@pytest.fixture
def make(bind, monkeypatch):
    """``BoundedDecoder`` without a GPU: buffers on the CPU, nothing launched."""
    def paged_init(self, num_blocks, Hq, Hkv, d, dtype, max_seqs, max_blocks_per_seq,
                   initial_free=None, device="cuda", num_parts=None, rope_base=10000.0, scale=None,
                   flags=0, k_cache=None, v_cache=None, metadata="copy", n_layers=1, plan=True,
                   layer_merge_helpers=None):
        self.torch, self.device, self.n_layers = torch, torch.device("cpu"), n_layers
        self.Hq, self.Hkv, self.d, self.dtype = Hq, Hkv, d, dtype
        self.tdtype = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
        self.bt_stride, self.num_parts, self.scale = max_blocks_per_seq, num_parts, scale or d**-0.5
        self.rope_base, self.flags = rope_base, flags
        self.alloc = bind.BlockAllocator(num_blocks, max_seqs, max_blocks_per_seq, initial_free)
    monkeypatch.setattr(bounded.PagedDecoder, "__init__", paged_init)
    monkeypatch.setattr(bind, "shared_default_parts", lambda *a: 4)
    base = dict(num_blocks=64, Hq=8, Hkv=2, d=64, dtype="f32", max_seqs=4, budget=24, slack=8)
    return lambda **kw: bounded.BoundedDecoder(**{**base, **kw})


def test_rope_base_reaches_the_rotary_table(bind, make):
    for kw, base in (({}, 10000.0), (dict(rope_base=500000.0), 500000.0), (dict(rope_base=1.0), 1.0)):
        want = bind.Rotary(64, base=base)
        assert list(make(**kw).rotary.table.turns) == list(want.table.turns)
    own = bind.Rotary(64, rot_dim=32, base=77.0)
    assert make(rotary=own).rotary is own


def test_rope_base_beside_a_rotary_is_refused(bind, make):
    with pytest.raises(ValueError):
        make(rotary=bind.Rotary(64), rope_base=500000.0)
