"""GPU parity of the attention of drafted tokens (pkv_decode_attn_tree) against its float64
oracle.

Tolerances, from the arithmetic (u: half a step of the storage type, 2^-8 for bf16 and 2^-24 for
float32): a score is d products accumulated in float32 (d + 4 roundings of up to 2^-23 each,
accumulators that truncate included) times scale, relative to the node's largest score, which
is bounded by swing = scale * max_t sum |q||k|: delta = (d + 8) * 2^-23 * swing + 2^-20.  A weight is
off by a factor within exp(2 delta) and by ex2's 2^-22; in bf16 it is rounded once, ahead of
the product with V.  Sums over the tokens in float32 add at most 2^-18 (steps of 128 tokens
accumulated exactly enough: one rounding a step and token group, below 2^5 * 2^-23 * 8192 / 128).
  |out - out*| <= (2 delta + 2^-18 [+ u for bf16]) * sum p|v| + u |out|
  |lse - lse*| <= delta + 2^-19 (1 + |lse|)
"""
import numpy as np
import pytest
import torch

from helpers import dev, f64
from oracle import drafted
from paged_kv_decode_10_gb300 import binding, workloads

pytestmark = pytest.mark.gpu

U = {"bf16": 2.0**-8, "f32": 2.0**-24}
TD = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def normal(shape, dtype, seed):
    return workloads.normal(shape, dtype, seed).to(dev())


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev())


def tables_of(lens, seed, spare=2):
    need = [-(-int(n) // 16) for n in lens]
    nb = sum(need) + spare
    free = list(np.random.default_rng(seed).permutation(nb))
    t = np.full((len(lens), max([1] + need)), -1, np.int32)
    for i, n in enumerate(need):
        for j in range(n):
            t[i, j] = free.pop()
    return nb, t


def random_parents(nodes, seed):
    rng = np.random.default_rng(seed)
    return np.concatenate([[-1] + [int(rng.integers(i // 3, i)) for i in range(1, n)] for n in nodes if n]
                          or [[]]).astype(np.int64)


class Case:
    """Inputs of a call; blocks of nobody and tokens behind a row's last hold NaN."""

    def __init__(self, cached, nodes, Hq, Hkv, d, dtype, kind="tree", seed=1, extra=0):
        self.dtype, self.d = dtype, d
        self.lens = np.array([c + n for c, n in zip(cached, nodes)], np.int32)
        self.starts = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        self.T = int(self.starts[-1]) + extra
        nb, self.tables = tables_of(self.lens, seed)
        self.q = normal((self.T, Hq, d), dtype, seed)
        self.k, self.v = normal((nb, Hkv, 16, d), dtype, seed + 1), normal((nb, Hkv, 16, d), dtype, seed + 2)
        self.scale = d**-0.5
        used = np.zeros((nb, 16), bool)
        for b, L in enumerate(self.lens):
            for t in range(int(L)):
                used[self.tables[b, t // 16], t % 16] = True
        un = torch.from_numpy(~used).to(dev())
        self.k.permute(0, 2, 1, 3)[un] = float("nan")
        self.v.permute(0, 2, 1, 3)[un] = float("nan")
        self.mask = None
        if kind != "chain":
            words = binding.tree_mask(random_parents(nodes, seed), self.starts)
            rng = np.random.default_rng(seed + 3)
            if kind == "hollow":     # some nodes see nothing of the tree
                words[rng.random(len(words)) < 0.3] = 0
            if kind == "any":        # any bits, later nodes and bits behind the last included
                words = rng.integers(-2**31, 2**31, (len(words), words.shape[1] + 1)).astype(np.int32)
            self.mask = np.zeros((self.T, words.shape[1]), np.int32)
            self.mask[:len(words)] = words

    def args(self, out, **kw):
        mask = None if self.mask is None else i32(self.mask)
        return binding.make_tree_args(self.q, self.k, self.v, i32(self.tables), i32(self.lens),
                                      i32(self.starts), self.scale, out, mask=mask, **kw)

    def run(self, **kw):
        out = torch.full_like(self.q, 7.0)
        lse = torch.full(self.q.shape[:2], 7.0, device=dev())
        err = torch.zeros(1, dtype=torch.int32, device=dev())
        binding.decode_attn_tree_args(self.args(out, lse=lse, err=err, **kw))
        torch.cuda.synchronize()
        assert int(err) == 0
        return out, lse

    def check(self, out, lse=None):
        n = int(self.starts[-1])
        want = drafted.tree_attention(f64(self.q), f64(self.k), f64(self.v), self.tables, self.lens,
                                      self.starts, self.scale, self.mask)
        check(f64(out)[:n], None if lse is None else f64(lse)[:n], [x[:n] for x in want], self.dtype, self.d)
        assert (f64(out)[n:] == 7.0).all()


def check(out, lse, want, dtype, d):
    o, l, absv, swing = want
    delta = (d + 8) * 2.0**-23 * swing + 2.0**-20
    tol = (2 * delta[..., None] + 2.0**-18 + (U[dtype] if dtype == "bf16" else 0)) * absv + U[dtype] * np.abs(o)
    nan = ~np.isfinite(o)
    assert np.array_equal(nan, ~np.isfinite(out)), (np.argwhere(nan != ~np.isfinite(out))[:5], nan.sum())
    bad = (np.abs(out - o) > tol) & ~nan
    assert not bad.any(), (np.argwhere(bad)[:5], out[bad][:5], o[bad][:5], tol[bad][:5], bad.sum())
    if lse is not None:
        same = np.isneginf(l) & np.isneginf(lse) | np.isnan(l) & np.isnan(lse)
        with np.errstate(invalid="ignore"):
            bad = ~(np.abs(lse - l) <= delta + 2.0**-19 * (1 + np.abs(l))) & ~same
        assert not bad.any(), (np.argwhere(bad)[:5], lse[bad][:5], l[bad][:5])


SHAPES = [
    # cached, nodes, Hq, Hkv, d
    ([0], [1], 2, 2, 64),
    ([1], [1], 8, 1, 128),
    ([0, 0, 3], [3, 1, 0], 4, 2, 64),
    ([15, 16, 17, 1], [1, 16, 17, 5], 4, 4, 128),
    ([127, 128, 129, 0], [2, 33, 64, 31], 16, 4, 64),
    ([300, 0, 5, 1000, 250], [9, 130, 0, 65, 32], 8, 2, 128),
    ([700], [270], 8, 1, 64),
    ([0, 90], [513, 4], 4, 1, 128),
    ([3000, 37], [8, 3], 16, 2, 128),
    ([5] * 40, list(range(40)), 2, 1, 64),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["tree", "chain", "hollow", "any"])
@pytest.mark.parametrize("cached,nodes,Hq,Hkv,d", SHAPES)
def test_tree_attention(cached, nodes, Hq, Hkv, d, kind, dtype):
    c = Case(cached, nodes, Hq, Hkv, d, dtype, kind, seed=len(cached) + d, extra=3)
    out, lse = c.run()
    c.check(out, lse)
    again, lse2 = c.run()       # the partition and the joins' order are fixed
    assert torch.equal(out, again) and torch.equal(lse.nan_to_num(9.0), lse2.nan_to_num(9.0))
