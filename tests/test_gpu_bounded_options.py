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


def ready(metadata="copy", n_layers=1):
    """Two rows, one behind a prefix, and a step's inputs."""
    dec = BoundedDecoder(40, 8, 2, 64, "f32", 2, 24, 8, device=dev(), metadata=metadata,
                         n_layers=n_layers)
    x = workloads.normal((n_layers, 32, 2, 64), "f32", 1).to(dev())
    p = dec.add_prefix(x, x.flip(1))
    ids = [dec.join(16, p, x[:, :16], x[:, 16:]), dec.join(5, None, x[:, :5], x[:, 5:10])]
    q, k, v = (workloads.normal((n_layers, 2, h, 64), "f32", 50 + i).to(dev())
               for i, h in enumerate((8, 2, 2)))
    return dec, ids, (q, k, v)


def lengths(dec, ids):
    a = dec.alloc
    return ([(a.seq_len(s), a.offset(s), a.seq_blocks(s), dec._held[s], dec._known[s]) for s in ids],
            a.num_free())


@pytest.mark.parametrize("what", ["rows expanded", "heads apart", "elements apart", "strange scale"])
def test_inputs_that_no_launch_takes_are_refused_before_a_sequence_grows(what):
    dec, ids, (q, k, v) = ready()
    before = lengths(dec, ids)
    if what == "rows expanded":
        bad = (q, k[:, :1].expand(1, 2, 2, 64), v)
    elif what == "heads apart":
        bad = (q, k, torch.cat([v, v], -1)[..., :64])
    elif what == "elements apart":
        bad = (torch.cat([q, q], -1)[..., ::2], k, v)
    else:
        with pytest.raises(ValueError):
            BoundedDecoder(40, 8, 2, 64, "f32", 2, 24, 8, device=dev(), scale=float("nan"))
        with pytest.raises(ValueError):
            BoundedDecoder(40, 8, 2, 64, "f32", 2, 24, 8, device=dev(), decay=float("inf"))
        return
    for _ in range(2):
        with pytest.raises((ValueError, binding.PkvError)):
            dec.step(ids, *bad)
        assert lengths(dec, ids) == before
    got = dec.step(ids, q, k, v).clone()
    ref, ids2, same = ready()
    assert torch.equal(got, ref.step(ids2, *same))
    torch.cuda.synchronize()
    assert dec.device_errors() == 0


@pytest.mark.parametrize("metadata", ["copy", "mapped"])
@pytest.mark.parametrize("layer", [0, 1])
def test_a_step_whose_launch_fails_takes_the_token_back(metadata, layer, monkeypatch):
    """An exception between a0 and the last launch: lengths, positions and blocks are as
    before, and the step can be made again."""
    dec, ids, x = ready(metadata, 2)
    before = lengths(dec, ids)
    calls, real = [], binding.decode_attn_shared_args

    def fail(args, stream=None):
        calls.append(args)
        if len(calls) > layer:
            raise RuntimeError("no memory")
        real(args, stream)

    with monkeypatch.context() as m:
        m.setattr(binding, "decode_attn_shared_args", fail)
        with pytest.raises(RuntimeError, match="no memory"):
            dec.step(ids, *x)
    now = lengths(dec, ids)
    assert [r[:2] + r[3:] for r in now[0]] == [r[:2] + r[3:] for r in before[0]]
    assert [r[2] for r in now[0]] == [r[2] for r in before[0]] and now[1] == before[1]
    assert dec._pending is None
    got = dec.step(ids, *x).clone()
    ref, ids2, same = ready(metadata, 2)
    want = ref.step(ids2, *same)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and dec.device_errors() == 0
    assert dec.last_metadata[0].tolist() == ref.last_metadata[0].tolist() == [32 + 16, 5]
