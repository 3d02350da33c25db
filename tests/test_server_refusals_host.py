"""A server captures ``pkv_decode_step`` over a decoder's buffers: decoders with a step (and a rotary, and
caches that may be replaced) of their own are refused."""
import pytest


@pytest.mark.parametrize("name", ["bounded.BoundedDecoder", "drafted.DraftDecoder"])
def test_decoders_with_a_step_of_their_own(host_lib, name):
    import importlib
    from paged_kv_decode_10_gb300 import binding
    module, cls = name.split(".")
    cls = getattr(importlib.import_module("paged_kv_decode_10_gb300." + module), cls)
    with pytest.raises(binding.PkvError, match=cls.__name__):
        binding.Server(cls.__new__(cls), [0], 16)
