"""Calls on a side stream that make their own outputs and scratch, while the current stream
is busy and takes and fills memory of its own: the same bits as on the current stream."""
import numpy as np
import pytest
import torch

from helpers import dev
from paged_kv_decode_10_gb300 import binding
from test_gpu_cache_ops import bits, evict_case, i32, make_case, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def beside_a_busy_stream(call):
    """``call(side)`` while the current stream sleeps some 20 ms and then fills new memory."""
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(40_000_000)
    got = call(side)
    junk = [torch.full((n,), 255, dtype=torch.uint8, device=dev()) for n in
            (1 << 10, 1 << 14, 1 << 17, 1 << 20, 5 << 20) for _ in range(8)]
    side.synchronize()
    torch.cuda.synchronize()
    del junk
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_shared_attention_beside_a_busy_stream(dtype):
    c = make_case(9, 8, 2, 128, dtype, [40, 3, 0, 170, 90, 1, 640, 200, 33], [1000, 130],
                  [i % 3 - 1 for i in range(9)], 91)
    plan = binding.shared_plan(c["rows"], c["plens"], 8, 2, 128, binding.dtype_code(c["q"]))
    args = (c["q"], c["kc"], c["vc"], torch.from_numpy(c["tab"]).to(dev()), i32(c["lens"]), c["scale"])
    kw = dict(prefix_tables=torch.from_numpy(c["ptab"]).to(dev()), num_parts=40,
              prefix_plan=torch.from_numpy(plan).to(dev()), slots=int(plan[3]), num_ctas=int(plan[4]))
    want = binding.decode_attention_shared(*args, **kw)
    for _ in range(3):
        got = beside_a_busy_stream(lambda s: binding.decode_attention_shared(*args, stream=s, **kw))
        assert torch.equal(got, want)


def test_eviction_beside_a_busy_stream():
    first = evict_case(2, 2, 64, "bf16", [9000, 5000], [4001, 2000], 5)
    tab, lens, keeps = (torch.from_numpy(first["tab"]).to(dev()), i32(first["lens"]), i32(first["keeps"]))

    want = [first[k].clone() for k in ("kc", "vc", "mass")]
    want.append(binding.evict(*want, tab, lens, keeps, 4001, 4, 100))
    cache = [first[k].clone() for k in ("kc", "vc", "mass")]
    kept = beside_a_busy_stream(
        lambda s: binding.evict(*cache, tab, lens, keeps, 4001, 4, 100, stream=s))
    for x, y in zip(want, cache + [kept]):
        np.testing.assert_array_equal(bits(x), bits(y))


def test_rotary_append_beside_a_busy_stream():
    q, k = normal((9, 8, 64), "bf16", 1), normal((9, 2, 64), "bf16", 2)
    rot, pos = binding.Rotary(64), i32(np.arange(9) * 14563)
    want = binding.rotary_append(rot, q, k, None, pos)
    got = beside_a_busy_stream(lambda s: binding.rotary_append(rot, q, k, None, pos, stream=s))
    assert all(torch.equal(x, y) for x, y in zip(got, want))
