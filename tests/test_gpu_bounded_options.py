"""``BoundedDecoder``'s arguments and its states between steps, on the GPU.

Tolerance of an output against the float64 replay: as in test_gpu_bounded."""
import numpy as np
import pytest
import torch

from helpers import dev, f64
from oracle import cache_ops
from paged_kv_decode_10_gb300 import binding, workloads
from paged_kv_decode_10_gb300.bounded import BoundedDecoder
from test_gpu_bounded import Replay

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rope_base_against_a_replay(dtype):
    """The default rotary turns at the decoder's ``rope_base``."""
    Hq, Hkv, d, base = 8, 2, 64, 500000.0
    dec = BoundedDecoder(16, Hq, Hkv, d, dtype, 1, 64, 16, rope_base=base, device=dev())
    spec = dict(freq=cache_ops.rotary_frequencies(d, "plain", base=base), layout="half")
    ref = Replay(dec, spec, dtype)

    def draw(n, heads, seed):
        x = workloads.normal((n, heads, d), dtype, seed)
        return x.to(dev()), f64(x)

    (k, k64), (v, v64) = draw(40, Hkv, 1), draw(40, Hkv, 2)
    s = dec.join(40, None, k, v)
    ref.add(k64[None], v64[None])
    u = 2.0**-8 if dtype == "bf16" else 2.0**-24
    for step in range(4):
        (q, q64), (k, k64), (v, v64) = (draw(1, h, 10 + 3 * step + i)
                                        for i, h in enumerate((Hq, Hkv, Hkv)))
        out = f64(dec.step([s], q, k, v))[0]
        assert dec.device_errors() == 0
        ref.add(k64[None], v64[None])
        want, swing, top = ref.attend(q64[0], 0)
        eps = 2 * (d + 8) * 2.0**-23 * swing + 2.0**-18
        if dtype == "bf16":
            eps += 2 * 2.0**-8 * top + u
        size = np.abs(np.array(ref.v[0])).max()
        err = np.abs(out - want).max()
        assert err <= eps * size + u * np.abs(want).max(), (step, err)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_checked_plan_gives_the_same_bits(dtype):
    """ATTN_CHECK_PLAN reaches the attention call, which finds the decoder's plan right."""
    outs = []
    for flags in (0, binding.ATTN_CHECK_PLAN):
        dec = BoundedDecoder(40, 8, 2, 64, dtype, 3, 24, 8, num_parts=6, flags=flags, device=dev())
        x = workloads.normal((40, 2, 64), dtype, 1).to(dev())
        p = dec.add_prefix(x, x.flip(0))
        ids = [dec.join(prefix=p), dec.join(), dec.join(5, p, x[:5], x[5:10])]
        for step in range(30):
            q, k, v = (workloads.normal((3, h, 64), dtype, 50 + 3 * step + i).to(dev())
                       for i, h in enumerate((8, 2, 2)))
            out = dec.step(ids, q, k, v).clone()
        torch.cuda.synchronize()
        assert dec.device_errors() == 0
        outs.append(out)
    assert torch.equal(*outs)


@pytest.mark.parametrize("metadata", ["copy", "mapped"])
def test_a_step_without_blocks_leaves_everything_as_it_was(metadata):
    """Rows of 16, 16 and 4 tokens in 5 blocks: step 1 takes the last two, step 13 needs
    another for the third row and changes neither allocator, weights nor caches."""
    dec = BoundedDecoder(5, 4, 2, 64, "f32", 3, 40, 8, device=dev(), metadata=metadata)
    kv = [workloads.normal((16, 2, 64), "f32", i).to(dev()) for i in range(6)]
    ids = [dec.join(n, None, kv[2 * i][:n], kv[2 * i + 1][:n]) for i, n in enumerate((16, 16, 4))]
    x = [workloads.normal((3, h, 64), "f32", 20 + h + i).to(dev()) for i, h in enumerate((4, 2, 2))]

    def state():
        torch.cuda.synchronize()
        a = dec.alloc
        return ([a.seq_len(s) for s in ids], [a.offset(s) for s in ids], [a.seq_blocks(s) for s in ids],
                a.num_free(), dict(dec._held), dict(dec._known)), \
            [t.clone() for t in (dec.masses, dec.k_caches, dec.v_caches)]

    for step in range(12):
        dec.step(ids, *x)
    host, device = state()
    assert host[0] == [28, 28, 16] and host[3] == 0
    for _ in range(2):
        with pytest.raises(binding.OutOfBlocks):
            dec.step(ids, *x)
        now, tensors = state()
        assert now == host
        # (bit for bit: slots that no token has written hold whatever was there)
        assert all(torch.equal(a.view(torch.int32), b.view(torch.int32)) for a, b in zip(device, tensors))
    dec.leave(ids[0])
    out = dec.step(ids[1:], *(t[1:] for t in x))
    torch.cuda.synchronize()
    assert [dec.alloc.seq_len(s) for s in ids[1:]] == [29, 17] and dec.device_errors() == 0
    assert bool(out.isfinite().all())
