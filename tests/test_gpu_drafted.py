"""``DraftDecoder``: drafted tokens, forks, chunks, single steps and a pool that changes its size, run
together against a replay in float64 from the raw queries, keys and values.

Tolerance: as for the attention alone (tests/test_gpu_tree.py), with what the rotation adds: rotated
queries and keys are off by u of their size (bf16) or 2^-20 (float32: angle, cos, sin, products) each,
so a score by delta2 = (2 u or 2^-19) * swing more; swing is taken over a token's |q| |k| in pairs,
where a rotation may turn one element's size into its partner's: sqrt(2)^2 on each product, 2 in all.
"""
import numpy as np
import pytest
import torch

from helpers import dev, f64
from oracle import cache_ops, drafted
from paged_kv_decode_10_gb300 import binding, workloads
from paged_kv_decode_10_gb300.drafted import DraftDecoder

pytestmark = pytest.mark.gpu

U = {"bf16": 2.0**-8, "f32": 2.0**-24}


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


class Replay:
    """What every sequence holds: raw keys and values and their positions, per layer."""

    def __init__(self, dec, sections=None):
        self.dec, self.rows = dec, {}
        self.axis, _ = drafted.axes_of(sections or (dec.d // 2,))
        self.freq = cache_ops.rotary_frequencies(dec.d)
        self.n_axes = len(sections or (1,))

    def positions(self, pos):
        pos = np.asarray(pos)
        return pos if pos.ndim == 2 else np.broadcast_to(pos, (self.n_axes, len(pos)))

    def rotated(self, x, pos):
        return drafted.rotary_axes(x, self.positions(pos), self.freq, self.axis)

    def check(self, out, sid, first, q, pos, sees):
        """Output rows of one sequence's n new tokens (the last of what it holds)."""
        dec, row = self.dec, self.rows[sid]
        for layer in range(dec.n_layers):
            k, v, p = (np.concatenate([x[layer] for x in row["k"]]), np.concatenate([x[layer] for x in row["v"]]),
                       np.concatenate(row["p"], axis=1))
            kr, qr = self.rotated(k, p), self.rotated(q[layer], pos)
            for i in range(len(qr)):
                for h in range(dec.Hq):
                    g = h // (dec.Hq // dec.Hkv)
                    ks, vs = kr[sees[i], g], v[sees[i], g]
                    s = ks @ qr[i, h] * dec.scale
                    w = np.exp(s - s.max())
                    w /= w.sum()
                    want, absv = w @ vs, w @ np.abs(vs)
                    swing = dec.scale * (np.abs(ks) @ np.abs(qr[i, h])).max()
                    u = U[dec.dtype]
                    delta = (dec.d + 8) * 2.0**-23 * swing + 2.0**-20
                    delta += 2 * (2 * u if dec.dtype == "bf16" else 2.0**-19) * swing
                    tol = (2 * delta + 2.0**-18 + (u if dec.dtype == "bf16" else 0)) * absv + u * np.abs(want)
                    got = out[layer, first + i, h]
                    assert (np.abs(got - want) <= tol).all(), (sid, layer, i, h, np.abs(got - want).max(), tol.min())

    def hold(self, sid, k, v, pos):
        self.rows[sid]["k"].append(k)
        self.rows[sid]["v"].append(v)
        self.rows[sid]["p"].append(self.positions(pos))

    def held(self, sid):
        return sum(p.shape[1] for p in self.rows[sid]["p"])

    def keep(self, sid, base, path):
        row = self.rows[sid]
        at = list(range(base)) + [base + i for i in path]
        for name, axis in (("k", 1), ("v", 1), ("p", 1)):
            row[name] = [np.take(np.concatenate(row[name], axis=axis), at, axis=axis)]


@pytest.mark.parametrize("dtype,L,sections", [("f32", 2, None), ("bf16", 1, (8, 12, 12)), ("bf16", 3, None),
                                              ("f32", 1, (16, 16))])
def test_life_of_a_drafting_batch(dtype, L, sections):
    Hq, Hkv, d = 4, 2, 64
    rot = None if sections is None else binding.Rotary(d, sections=sections)
    dec = DraftDecoder(120, Hq, Hkv, d, dtype, 10, 30, rotary=rot, n_layers=L, device=dev())
    m = Replay(dec, sections)
    rng = np.random.default_rng(L)
    seed = [100]

    def new(n):
        """Raw q, k, v of n tokens in every layer: on the GPU, and in float64."""
        seed[0] += 1
        x = workloads.normal((L, n, Hq + 2 * Hkv, d), dtype, seed[0])
        parts = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
        return [p.to(dev()) for p in parts], [f64(p) for p in parts]

    def outs(out):
        out = f64(out)
        return out if out.ndim == 4 else out[None]

    def call(x):     # (layers in front only where there are several)
        return x if L > 1 else [t[0] for t in x]

    def join(n):
        (_, k, v), (_, k64, v64) = new(n)
        sid = dec.join(n, *call([k.contiguous(), v.contiguous()]))
        m.rows[sid] = dict(k=[], v=[], p=[])
        m.hold(sid, k64, v64, np.arange(n))
        return sid

    ids = [join(n) for n in (33, 0, 16, 70)]
    for turn in range(12):
        # ---- a tree for every sequence; a path of it stays
        rows = [int(s) for s in rng.permutation(ids)[:4]]
        counts = rng.integers(0, 20, len(rows))
        parents = np.concatenate([[-1] + [int(rng.integers(0, i)) for i in range(1, n)] for n in counts if n]
                                 or [[]]).astype(int)
        starts = np.concatenate([[0], np.cumsum(counts)])
        T = int(counts.sum())
        x, (q64, k64, v64) = new(T)
        base = [m.held(s) for s in rows]
        depth = np.zeros(T, int)
        sees = []
        for b in range(len(rows)):
            a, n = starts[b], counts[b]
            seen = np.ones((n, base[b] + n), bool)
            seen[:, base[b]:] = np.eye(n, dtype=bool)
            for i in range(n):
                if parents[a + i] >= 0:
                    depth[a + i] = depth[a + parents[a + i]] + 1
                    seen[i, base[b]:] |= seen[parents[a + i], base[b]:]
            sees.append(seen)
        pos = np.concatenate([base[b] + depth[starts[b]:starts[b + 1]] for b in range(len(rows))])
        given = None
        if sections is not None and turn % 2:       # each axis at its own place
            given = np.stack([pos + 3 * a for a in range(len(sections))]).astype(np.int32)
        out = outs(dec.verify(rows, counts, *call(x), parents=parents, positions=given))
        for b, s in enumerate(rows):
            if not counts[b]:
                continue
            span = slice(starts[b], starts[b + 1])
            at = pos[span] if given is None else given[:, span]
            m.hold(s, k64[:, span], v64[:, span], at)
            m.check(out, s, starts[b], q64[:, span], at, sees[b])
        paths = []
        for b in range(len(rows)):
            path, at = [], counts[b] - 1
            while at >= 0 and counts[b]:            # from a node up to its root
                path.append(int(at))
                at = parents[starts[b] + at]
            paths.append(sorted(path)[:int(rng.integers(0, len(path) + 1))])
        if T:
            dec.accept(paths)
            for b, s in enumerate(rows):
                m.keep(s, base[b], paths[b])
                assert dec.alloc.seq_len(s) == m.held(s) == base[b] + len(paths[b])
        # ---- now and then: a fork, a chunk, a leave, another pool, a single step
        if turn % 3 == 0:
            s = int(rng.choice(ids))
            for c in dec.fork(s, 2):
                m.rows[c] = {key: list(x) for key, x in m.rows[s].items()}
                ids.append(c)
        if turn % 4 == 1:
            dec.resize(int(rng.integers(100, 160)))
        rows = [int(s) for s in rng.permutation(ids)[:3]]
        counts = np.ones(3, int) if turn % 2 else rng.integers(0, 9, 3)
        x, (q64, k64, v64) = new(int(counts.sum()))
        out = outs(dec.step(rows, *call(x)) if turn % 2 else dec.extend(rows, counts, *call(x)))
        at = 0
        for s, n in zip(rows, counts):
            base = m.held(s)
            span = slice(at, at + n)
            m.hold(s, k64[:, span], v64[:, span], np.arange(base, base + n))
            seen = np.arange(base + n)[None] <= base + np.arange(n)[:, None]
            if n:
                m.check(out, s, at, q64[:, span], np.arange(base, base + n), seen)
            at += n
        while len(ids) > 5:
            s = ids.pop(int(rng.integers(0, len(ids))))
            dec.leave(s)
            del m.rows[s]
    assert dec.device_errors() == 0
    for s in ids:
        dec.leave(s)
    assert dec.alloc.num_free() == dec.num_blocks


def inputs(T, dec, L=None):
    shape = (T,) if L is None else (L, T)
    return [torch.zeros(shape + (h, dec.d), dtype=dec.tdtype, device=dev()) for h in (dec.Hq, dec.Hkv, dec.Hkv)]


def test_what_a_drafting_decoder_refuses():
    make = lambda **kw: DraftDecoder(20, 4, 2, 64, "f32", 4, 8, device=dev(), **kw)
    for kw in (dict(num_parts=4), dict(plan=False), dict(layer_merge_helpers=True), dict(metadata="mapped"),
               dict(flags=binding.ATTN_SIMT), dict(scale=float("nan")), dict(rotary=binding.Rotary(128)),
               dict(rotary=binding.Rotary(64), rope_base=10000.0)):
        with pytest.raises(ValueError):
            make(**kw)
    dec = make()
    s, t = dec.join(20, *inputs(20, dec)[1:]), dec.join()
    state = dec.alloc.free_stack()
    q, k, v = inputs(3, dec)
    for call in (lambda: dec.verify([s], [2], q, k, v), lambda: dec.verify([s], [3, 0], q, k, v),
                 lambda: dec.verify([s, t], [4, -1], q, k, v), lambda: dec.verify([s], [3], q[:, :2], k, v),
                 lambda: dec.verify([s], [3], q.bfloat16(), k, v), lambda: dec.verify([s], [3], q.cpu(), k, v),
                 lambda: dec.verify([s], [3], q, k, v, parents=[-1, 0]),
                 lambda: dec.verify([s], [3], q, k, v, parents=[-1, 1, 0]),
                 lambda: dec.verify([s], [3], q, k, v, parents=[-1, 0, 0], depths=[0, 1, 1]),
                 lambda: dec.verify([s], [3], q, k, v, mask=np.ones((3, 0), np.int32), depths=[0, 1, 2]),
                 lambda: dec.verify([s], [3], q, k, v, mask=np.ones((3, 1), np.int32)),
                 lambda: dec.verify([s], [3], q, k, v, positions=np.zeros((2, 3), np.int32)),
                 lambda: dec.verify([s, s], [2, 1], q, k, v), lambda: dec.verify([9], [3], q, k, v),
                 lambda: dec.extend([s], [200], *inputs(200, dec)),
                 lambda: dec.step([s], q, k, v), lambda: dec.step([s], q[:1], k[:1], v[:1], attn_bias=q),
                 lambda: dec.accept([[0]]), lambda: dec.capture(1), lambda: dec.fork(9), lambda: dec.resize(1),
                 lambda: dec.join(3, k, None), lambda: dec.join(4, k, v)):
        with pytest.raises((ValueError, binding.PkvError)):
            call()
        assert dec.alloc.free_stack() == state and dec.alloc.seq_len(s) == 20 and dec.alloc.seq_len(t) == 0
    # between verify and accept
    dec.verify([s, t], [2, 1], q, k, v)
    for call in (lambda: dec.step([s], q[:1], k[:1], v[:1]), lambda: dec.fork(s), lambda: dec.resize(30),
                 lambda: dec.verify([s, t], [2, 1], q, k, v), lambda: dec.accept([[0]]),
                 lambda: dec.accept([[0, 2], []]), lambda: dec.accept([[1, 0], []]), lambda: dec.accept([[-1], []])):
        with pytest.raises(ValueError):
            call()
    dec.leave(t)                     # its path counts for nothing then
    u = dec.join()                   # (takes over its id)
    assert u == t
    dec.step([u], q[:1], k[:1], v[:1])
    dec.accept([[1], [0]])
    assert dec.alloc.seq_len(s) == 21 and dec.alloc.seq_len(u) == 1
    assert dec.device_errors() == 0


def test_a_step_that_raises_takes_its_tokens_back(monkeypatch):
    dec = DraftDecoder(20, 4, 2, 64, "bf16", 4, 8, device=dev(), n_layers=2)
    s = dec.join(15)
    (c,) = dec.fork(s)
    state = dec.alloc.free_stack()
    real, calls = binding.decode_attn_tree_args, []

    def second_fails(args, stream=None):
        calls.append(args)
        if len(calls) == 2:
            raise RuntimeError("planted")
        real(args, stream)
    monkeypatch.setattr(binding, "decode_attn_tree_args", second_fails)
    with pytest.raises(RuntimeError):
        dec.verify([s, c], [20, 3], *inputs(23, dec, 2))
    assert dec.alloc.seq_len(s) == dec.alloc.seq_len(c) == 15 and sorted(dec.alloc.free_stack()) == sorted(state)
    dec.verify([s, c], [20, 3], *inputs(23, dec, 2))
    dec.accept([[0, 5], [2]])
    assert dec.alloc.seq_len(s) == 17 and dec.alloc.seq_len(c) == 16 and dec.device_errors() == 0


def test_steps_on_a_side_stream():
    """The same life on a stream of its own, the accept on another: the same bits."""
    got = []
    for side in (None, torch.cuda.Stream()):
        dec = DraftDecoder(40, 8, 2, 128, "bf16", 4, 20, device=dev())
        torch.cuda.synchronize()
        x = [workloads.normal((60, h, 128), "bf16", h).to(dev()) for h in (8, 2, 3)]
        x[2] = x[2][:, :2].contiguous()
        torch.cuda.synchronize()
        s = dec.join(30, x[1][:30], x[2][:30], stream=side)
        (c,) = dec.fork(s, stream=side)
        outs = []
        for _ in range(5):
            outs.append(dec.verify([s, c], [9, 4], *(t[:13] for t in x), parents=[-1, 0, 0, 1, 2, 2, 3, 3, 5,
                                                                                  -1, 0, 0, 2], stream=side))
            dec.accept([[0, 2, 5], [0, 2]], stream=None if side is None else torch.cuda.Stream())
            torch.cuda.synchronize()
            outs.append(dec.step([c, s], *(t[20:22] for t in x), stream=side))
        torch.cuda.synchronize()
        got.append(outs)
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_readme_example_of_drafted_tokens_runs():
    import os
    import re
    readme = os.path.join(os.path.dirname(os.path.dirname(__file__)), "README.md")
    blocks = re.findall(r"```python\n(.*?)```", open(readme).read(), flags=re.S)
    example, = [b for b in blocks if "DraftDecoder" in b]
    scope = dict(torch=torch, np=np, binding=binding, dev=dev())
    exec(compile(example, "readme example", "exec"), scope)
    torch.cuda.synchronize()
    dec, a, b = scope["dec"], scope["a"], scope["b"]
    assert tuple(scope["out"].shape) == (9, 32, 128) and bool(scope["out"].float().isfinite().all())
    assert dec.alloc.seq_len(a) == 703 and dec.alloc.seq_len(b) == 701 and dec.k_cache.shape[0] == 2048
    assert dec.device_errors() == 0


def test_a_bounded_decoder_takes_no_rotary_with_sections():
    from paged_kv_decode_10_gb300.bounded import BoundedDecoder
    with pytest.raises(ValueError):
        BoundedDecoder(20, 4, 2, 64, "f32", 4, 24, 8, rotary=binding.Rotary(64, sections=(16, 16)),
                       device=dev())


def test_a_verify_without_nodes_is_accepted_like_any():
    dec = DraftDecoder(20, 4, 2, 64, "f32", 4, 8, device=dev())
    s, t = dec.join(5, *inputs(5, dec)[1:]), dec.join()
    out = dec.verify([s, t], [0, 0], *inputs(0, dec), parents=[])
    assert tuple(out.shape) == (0, 4, 64)
    with pytest.raises(ValueError):
        dec.accept([[0], []])
    dec.accept([[], []])
    with pytest.raises(ValueError):
        dec.accept([[], []])
    assert dec.alloc.seq_len(s) == 5 and dec.alloc.seq_len(t) == 0
    dec.step([s, t], *inputs(2, dec))
    assert dec.alloc.seq_len(s) == 6 and dec.alloc.seq_len(t) == 1 and dec.device_errors() == 0


def test_every_call_on_another_stream():
    """A life whose calls change the stream each time, nobody waiting in between: the bits of
    the same life on one stream."""
    got = []
    for sides in (1, 4):
        dec = DraftDecoder(4000, 8, 2, 128, "bf16", 8, 600, device=dev(), n_layers=2)
        x = [workloads.normal((2, 5200, h, 128), "bf16", h).to(dev()) for h in (8, 2, 3)]
        x[2] = x[2][:, :, :2].contiguous()
        streams = [torch.cuda.Stream() for _ in range(sides)]
        torch.cuda.synchronize()
        turn = [0]

        def on():
            turn[0] += 1
            return streams[turn[0] % sides]
        at = lambda a, n: [t[:, a:a + n].contiguous() for t in x]
        many, nine, two = at(0, 5000), at(5000, 9), at(5100, 2)
        torch.cuda.synchronize()
        s = dec.join(5000, many[1], many[2], stream=on())
        (c,) = dec.fork(s, stream=on())
        outs = []
        for turns in range(4):
            outs.append(dec.verify([s, c], [5, 4], *nine, parents=[-1, 0, 0, 1, 2, -1, 0, 0, 2], stream=on()))
            dec.accept([[0, 2, 4], [0, 2]], stream=on())
            if turns == 1:
                dec.resize(1000, stream=on())
            outs.append(dec.step([c, s], *two, stream=on()))
        torch.cuda.synchronize()
        assert dec.device_errors() == 0
        got.append(outs)
    for a, b in zip(*got):
        assert torch.equal(a, b)
