"""``BoundedDecoder``: rotary append, shared-prefix attention with weights and eviction run
together as a server would, against a float64 replay.

The replay takes the decoder's own choice of kept tokens (weights that differ by less than
their rounding may be chosen either way) and checks it: no dropped candidate outweighs a
kept one by more than the weights' error.  Tolerances: every attention weight of the
decoder is within a factor 1 +- eps_w of the replay's, eps_w = 2 * (d + 8) * 2^-23 * swing +
2^-18 (scores, see test_gpu_cache_ops) plus, in bf16, what keys and queries rounded after
the rotation may do: none, the replay rounds them likewise, except where the two
rotations differ by a rounding boundary; a bf16 key element off by 2^-8 relative in one of
d products moves a score by at most 2^-8 |q_i k_i| scale.  The bound below allows that for
one element per key: eps_s = 2^-8 * max|q| * max|k| * scale.
"""
import numpy as np
import pytest
import torch

from helpers import dev, f64
from oracle import cache_ops
from oracle.numerics import round_to
from paged_kv_decode_10_gb300 import binding, workloads
from paged_kv_decode_10_gb300.bounded import BoundedDecoder

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


class Replay:
    """One sequence, float64: per layer and KV head the cached keys, values, weights."""

    def __init__(self, dec, rot, dtype, prefix=None):
        self.dec, self.rot, self.dtype = dec, rot, dtype
        self.prefix = prefix     # (keys, values) [L][Hkv][n][d]
        L, H = dec.n_layers, dec.Hkv
        self.k = [[[] for _ in range(H)] for _ in range(L)]
        self.v = [[[] for _ in range(H)] for _ in range(L)]
        self.m = [[[] for _ in range(H)] for _ in range(L)]
        self.pos = 0 if prefix is None else prefix[0].shape[2]

    def turn(self, x, pos):      # [n, H, d] at positions pos
        return round_to(cache_ops.rotary(x, pos, **self.rot), self.dtype)

    def add(self, k, v):         # [L, n, Hkv, d] raw
        n = k.shape[1]
        for layer in range(self.dec.n_layers):
            kr = self.turn(k[layer], np.arange(self.pos, self.pos + n))
            for h in range(self.dec.Hkv):
                self.k[layer][h] += list(kr[:, h])
                self.v[layer][h] += list(v[layer][:, h])
                self.m[layer][h] += [0.0] * n
        self.pos += n

    def evict(self, kept):       # [L, Hkv, keep]
        d = self.dec
        for layer in range(d.n_layers):
            for h in range(d.Hkv):
                n = len(self.m[layer][h])
                src = kept[layer, h][kept[layer, h] >= 0]
                assert len(src) == min(n, kept.shape[-1]) and (np.diff(src) > 0).all()
                m = np.array(self.m[layer][h])
                r = min(d.recent, len(src))
                s = min(d.sink, len(src) - r)
                if len(src) < n:
                    assert set(range(s)) | set(range(n - r, n)) <= set(src.tolist())
                    chosen = [t for t in src if s <= t < n - r]
                    dropped = sorted(set(range(s, n - r)) - set(chosen))
                    if chosen and dropped:
                        assert m[chosen].min() >= m[dropped].max() * (1 - 2e-2) - 1e-6
                for x in (self.k, self.v, self.m):
                    x[layer][h] = [x[layer][h][t] for t in src]

    def attend(self, q, layer):  # q [Hq, d] raw; the step's token was added
        d = self.dec
        G = d.Hq // d.Hkv
        qr = self.turn(q[None], [self.pos - 1])[0]
        out, swing = np.zeros_like(qr), 0.0
        for h in range(d.Hkv):
            k, v = np.array(self.k[layer][h]), np.array(self.v[layer][h])
            at = 0
            if self.prefix is not None:
                at = self.prefix[0].shape[2]
                k = np.concatenate([self.prefix[0][layer][h], k])
                v = np.concatenate([self.prefix[1][layer][h], v])
            m = np.array(self.m[layer][h]) * d.decay
            for i in range(h * G, h * G + G):
                s = (k @ qr[i]) * d.scale
                w = np.exp(s - s.max())
                w /= w.sum()
                out[i] = w @ v
                m += w[at:]
                swing = max(swing, (np.abs(k) @ np.abs(qr[i])).max() * d.scale)
            self.m[layer][h] = list(m)
        top = max(np.abs(np.array(self.k[layer])).max() * np.abs(qr).max() * d.scale, 0.0)
        return out, swing, top


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L,metadata,width", [(1, "copy", 3), (2, "mapped", 3), (1, "mapped", 150),
                                              (2, "copy", 150)])   # (150: not a short context)
def test_bounded_decoding_against_a_replay(dtype, L, metadata, width):
    Hq, Hkv, d, budget, slack = 8, 2, 64, 24, 9
    rot = binding.Rotary(d, rot_dim=32, layout="interleaved", scaling="bands", factor=4.0, low=1.0,
                         high=4.0, original_len=64)
    spec = dict(freq=cache_ops.rotary_frequencies(32, "bands", factor=4.0, low=1.0, high=4.0,
                                                  original_len=64), layout="interleaved")
    dec = BoundedDecoder(96, Hq, Hkv, d, dtype, 6, budget, slack, sink=2, recent=5, rotary=rot,
                         decay=0.95, n_layers=L, metadata=metadata, device=dev(), max_blocks_per_seq=width,
                         initial_free=np.random.default_rng(1).permutation(96).astype(np.int32))
    free0 = dec.alloc.num_free()

    def draw(n, heads, seed):
        x = workloads.normal((L, n, heads, d), dtype, seed)
        return x.to(dev()), f64(x)

    prefixes = []
    for i, n in enumerate((150, 16)):
        (k, k64), (v, v64) = draw(n, Hkv, 10 + i), draw(n, Hkv, 20 + i)
        pid = dec.add_prefix(k if L > 1 else k[0], v if L > 1 else v[0])
        kr = np.stack([round_to(cache_ops.rotary(k64[layer], np.arange(n), **spec), dtype)
                       for layer in range(L)])
        prefixes.append((pid, (kr.transpose(0, 2, 1, 3), v64.transpose(0, 2, 1, 3))))
    live, seed = {}, 100

    def join(which, n):
        nonlocal seed
        (k, k64), (v, v64) = draw(n, Hkv, seed), draw(n, Hkv, seed + 1)
        seed += 2
        pid, ref = (None, None) if which is None else prefixes[which]
        sid = dec.join(n, pid, k if L > 1 else k[0], v if L > 1 else v[0])
        live[sid] = Replay(dec, spec, dtype, ref)
        live[sid].add(k64, v64)
        return sid

    for which, n in ((0, 3), (0, 0), (1, 20), (None, 30)):
        join(which, n)
    evictions = 0
    real = dec.evict

    def watched(ids, keep=None, stream=None):
        nonlocal evictions
        kept = real(ids, keep, stream)
        for i, s in enumerate(ids):
            evictions += 1
            live[s].evict(kept[:, i].cpu().numpy())
        return kept

    dec.evict = watched
    for step in range(45):
        if step == 12:
            dec.leave(min(live))
            del live[min(live)]
        if step == 13:
            join(1, 32)
        if step == 20:
            join(0, 1)
        ids = sorted(live) if step % 3 else sorted(live, reverse=True)
        B = len(ids)
        (q, q64), (k, k64), (v, v64) = (draw(B, h, 1000 + 3 * step + i)
                                        for i, h in enumerate((Hq, Hkv, Hkv)))
        out = dec.step(ids, *((q, k, v) if L > 1 else (q[0], k[0], v[0])))
        torch.cuda.synchronize()
        assert dec.device_errors() == 0
        out = f64(out).reshape(L, B, Hq, d)
        for b, s in enumerate(ids):
            live[s].add(k64[:, b:b + 1], v64[:, b:b + 1])
            assert dec.alloc.seq_len(s) == len(live[s].m[0][0]) <= budget + slack
            assert int(dec.last_metadata[0][b]) == live[s].pos - 1
            for layer in range(L):
                want, swing, top = live[s].attend(q64[layer, b], layer)
                u = 2.0**-8 if dtype == "bf16" else 2.0**-24
                eps = 2 * (d + 8) * 2.0**-23 * swing + 2.0**-18
                if dtype == "bf16":
                    eps += 2 * 2.0**-8 * top + u
                size = max(np.abs(np.array(live[s].v[layer])).max(),
                           0 if live[s].prefix is None else np.abs(live[s].prefix[1][layer]).max())
                err = np.abs(out[layer, b] - want).max()
                assert err <= eps * size + u * np.abs(want).max(), (step, s, layer, err)
    assert evictions >= 6
    # every block comes back
    for s in list(live):
        dec.leave(s)
    with pytest.raises(ValueError):
        dec.drop_prefix(99)
    for pid, _ in prefixes:
        dec.drop_prefix(pid)
    assert dec.alloc.num_free() == free0


def test_bounded_decoder_refuses():
    kw = dict(num_blocks=16, Hq=4, Hkv=2, d=64, dtype="f32", max_seqs=2, budget=8, device=dev())
    for bad in (dict(budget=0), dict(slack=0), dict(sink=-1), dict(recent=-1),
                dict(rotary=binding.Rotary(128)), dict(max_blocks_per_seq=0), dict(max_prefixes=-1)):
        with pytest.raises(ValueError):
            BoundedDecoder(**{**kw, **bad})
    dec = BoundedDecoder(**kw, slack=8)
    x = torch.zeros((3, 2, 64), device=dev())
    pid = dec.add_prefix(x, x)
    for bad in (dict(prefix_len=16), dict(prefix=7), dict(prefix_len=2, k=x, v=x),
                dict(prefix_len=3, k=x, v=None)):
        with pytest.raises(ValueError):
            dec.join(**bad)
    free = dec.alloc.num_free()
    a, b = dec.join(3, pid, x, x), dec.join(0)
    with pytest.raises(ValueError):
        dec.join(0)                      # all rows are live
    with pytest.raises(ValueError):
        dec.drop_prefix(pid)             # in use
    with pytest.raises(binding.UnknownSequence):
        dec.step([a, pid], *(torch.zeros((2, h, 64), device=dev()) for h in (4, 2, 2)))
    with pytest.raises(binding.UnknownSequence):
        dec.leave(pid)
    with pytest.raises(ValueError):
        dec.evict([a, a])
    with pytest.raises(ValueError):
        dec.evict([a], keep=-1)
    with pytest.raises(ValueError):
        dec.capture(2)
    one = [torch.zeros((1, h, 64), device=dev()) for h in (4, 2, 2)]
    for args, kw2 in ((([a], *one), dict(attn_bias=torch.zeros((1, 16), device=dev()))),
                      (([a, a], *one), {}), (([a, b], *one), {}), (([a], one[1], one[1], one[2]), {}),
                      (([a], one[0].bfloat16(), one[1], one[2]), {}),
                      (([a], one[0].cpu(), one[1], one[2]), {})):
        with pytest.raises(ValueError):
            dec.step(*args, **kw2)
    assert dec.alloc.seq_len(a) == 3 and dec.alloc.seq_len(b) == 0     # nothing grew
    assert dec.step([], *(t[:0] for t in one)).shape[0] == 0
    dec.leave(a), dec.leave(b)
    dec.drop_prefix(pid)
    assert dec.alloc.num_free() == free + 1


def test_eviction_before_the_first_step_on_another_stream():
    """Tokens no step has weighed are all alike: the lowest indices stay; a call on a side
    stream orders its own copies."""
    dec = BoundedDecoder(32, 4, 2, 64, "bf16", 2, 16, 16, sink=1, recent=2, device=dev())
    dec.masses.fill_(float("nan"))
    k, v = (workloads.normal((31, 2, 64), "bf16", i).to(dev()) for i in (1, 2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s = dec.join(31, None, k, v, stream=side)
    kept = dec.evict([s], 10, stream=side)
    q1, k1, v1 = (workloads.normal((1, h, 64), "bf16", 3 + h).to(dev()) for h in (4, 2, 2))
    side.wait_stream(torch.cuda.current_stream())
    out = dec.step([s], q1, k1, v1, stream=side)
    side.synchronize()
    assert kept[0, 0].tolist() == [list(range(8)) + [29, 30]] * 2
    assert dec.alloc.seq_len(s) == 11 and int(dec.last_metadata[0][0]) == 31
    assert bool(out.float().isfinite().all()) and dec.device_errors() == 0


def test_a_step_that_runs_out_of_blocks_changes_nothing():
    """Blocks for two of three rows: the step raises, and runs after a sequence has left."""
    dec = BoundedDecoder(5, 4, 2, 64, "f32", 3, 40, 8, device=dev())
    draw = (workloads.normal((16, 2, 64), "f32", i).to(dev()) for i in range(8))
    ids = [dec.join(n, None, next(draw)[:n], next(draw)[:n]) for n in (16, 16, 4)]
    x = [workloads.normal((3, h, 64), "f32", 20 + h + i).to(dev()) for i, h in enumerate((4, 2, 2))]
    first = [t[2:] for t in x]
    with pytest.raises(binding.OutOfBlocks):
        for _ in range(40):
            dec.step(ids, *x)
    lens = [dec.alloc.seq_len(s) for s in ids]
    assert lens[0] == lens[1] == 32 and lens[2] == 20 or max(lens) <= 48
    assert lens == [dec._held[s] for s in ids]
    dec.leave(ids[0])
    out = dec.step(ids[1:], *(t[1:] for t in x)).clone()
    # the same sequence alone, whole
    ref = BoundedDecoder(5, 4, 2, 64, "f32", 3, 40, 8, device=dev())
    draw = [workloads.normal((16, 2, 64), "f32", i).to(dev()) for i in (4, 5)]
    one = ref.join(4, None, draw[0][:4], draw[1][:4])
    for _ in range(lens[2] - 4 + 1):
        want = ref.step([one], *first)
    torch.cuda.synchronize()
    assert dec.device_errors() == 0
    torch.testing.assert_close(out[1], want[0], rtol=2.0**-18, atol=2.0**-18)


def test_steps_in_other_orders_reuse_prepared_calls():
    """The same batch in either order, strided inputs, and one metadata buffer in turn after
    the other give each row the same output as a batch of its own."""
    made = []
    for metadata in ("copy", "mapped"):
        dec = BoundedDecoder(40, 8, 2, 64, "bf16", 4, 24, 8, device=dev(), metadata=metadata)
        x = workloads.normal((40, 2, 64), "bf16", 1).to(dev())
        p = dec.add_prefix(x, x.flip(0))
        ids = [dec.join(prefix=p), dec.join(), dec.join(5, p, x[:5], x[5:10])]
        outs = []
        for step in range(9):
            qkv = workloads.normal((3, 12, 64), "bf16", 50 + step).to(dev())
            order = [0, 1, 2] if step % 2 else [2, 0, 1]
            if step == 6:
                order = [1]
            rows = qkv[torch.tensor(order, device=dev())]
            if step % 3 == 0:       # slices of one projection's output
                q, k, v = rows[:, :8], rows[:, 8:10], rows[:, 10:]
            else:
                q, k, v = (t.contiguous() for t in (rows[:, :8], rows[:, 8:10], rows[:, 10:]))
            out = dec.step([ids[i] for i in order], q, k, v)
            outs.append({i: out[b].clone() for b, i in enumerate(order)})
        torch.cuda.synchronize()
        assert dec.device_errors() == 0
        made.append(outs)
    for a, b in zip(*made):
        for i in a:
            assert torch.equal(a[i], b[i])
    # sequence 1 alone
    dec = BoundedDecoder(40, 8, 2, 64, "bf16", 1, 24, 8, device=dev())
    s = dec.join()
    for step in range(9):
        qkv = workloads.normal((3, 12, 64), "bf16", 50 + step).to(dev())[1:2]
        out = dec.step([s], qkv[:, :8], qkv[:, 8:10], qkv[:, 10:])
        torch.testing.assert_close(out[0].float(), made[0][step][1].float(), rtol=2.0**-6, atol=2.0**-6)
