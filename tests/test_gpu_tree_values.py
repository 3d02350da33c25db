"""What is not finite in the attention of drafted tokens: infinities keep their sign and NaN stays NaN,
in whole items, in items that several CTAs share, and in items of both row tiles.  Tolerances of
what is finite: tests/test_gpu_tree.py."""
import numpy as np
import pytest
import torch

import test_gpu_tree as tree
from helpers import dev, f64
from oracle import drafted
from paged_kv_decode_10_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def check(c, out, lse):
    """Weights here are far from underflow, so that an infinite value that a row sees is an
    infinity of its sign in the formula and in the kernel alike."""
    n = int(c.starts[-1])
    with np.errstate(invalid="ignore"):
        o, l, absv, swing = (x[:n] for x in drafted.tree_attention(
            f64(c.q), f64(c.k), f64(c.v), c.tables, c.lens, c.starts, c.scale, c.mask))
    out, lse = f64(out)[:n], f64(lse)[:n]
    assert np.array_equal(np.isnan(o), np.isnan(out)), np.argwhere(np.isnan(o) != np.isnan(out))[:5]
    inf = np.isinf(o)
    assert np.array_equal(inf, np.isinf(out)) and np.array_equal(o[inf], out[inf])
    assert np.array_equal(np.isnan(l), np.isnan(lse)) and np.array_equal(np.isneginf(l), np.isneginf(lse))
    with np.errstate(invalid="ignore"):
        tree.check(out, lse, (o, l, absv, swing), c.dtype, c.d)
    return o


def spoil(c, b, tokens, value, every=3, first=0):
    for t in tokens:
        c.v[c.tables[b, t // 16], :, t % 16, first::every] = value


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G,kind", [(1, "tree"), (8, "tree"), (8, "chain"), (4, "any"), (2, "hollow")])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf"), "both"])
def test_values_that_are_not_finite(value, G, kind, dtype):
    nodes, cached = [40, 150, 3, 33], [130, 0, 17, 3000]     # (the last: shared by many CTAs)
    c = tree.Case(cached, nodes, 2 * G, 2, 128, dtype, kind, seed=8, extra=1)
    signs = [value] * 2 if value != "both" else [float("inf"), float("-inf")]
    for b, some in enumerate(([5, 38], [60, 130, 149], [1], [2, 20, 32])):
        for i, t in enumerate(some):
            spoil(c, b, [cached[b] + t], signs[i % 2])
    spoil(c, 0, [7], signs[0], every=5, first=1)             # cached tokens, seen by all
    spoil(c, 3, [2000], signs[1], every=5, first=2)
    o = check(c, *c.run())
    assert (~np.isfinite(o)).any() and np.isfinite(o).any()
    if value not in ("both",) and value == value:
        assert (o == value).any() and not (o == -value).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_keys_and_queries_that_are_not_finite(value, dtype):
    nodes, cached = [40, 70], [130, 900]
    c = tree.Case(cached, nodes, 16, 2, 64, dtype, "tree", seed=18)
    for b, some in enumerate(([5, 39], [1, 60])):
        for t in some:
            c.k[c.tables[b, (cached[b] + t) // 16], :, (cached[b] + t) % 16] = value
    c.q[3], c.q[nodes[0] + 9, 5] = value, value
    check(c, *c.run())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nodes", [64, 40])
def test_shared_tiles_with_values_that_are_not_finite(nodes, d):
    """Items of both row tiles whose last tiles hold such values, many at once, again and
    again: one of the two issuers of a tile cleans it for both."""
    B = 64
    c = tree.Case([100 + 7 * b for b in range(B)], [nodes] * B, 8, 2, d, "bf16", "tree", seed=4)
    for b in range(B):
        base = int(c.lens[b]) - nodes
        spoil(c, b, [base + 1 + b % (nodes - 1), base + nodes - 1], float("nan") if b % 2 else float("inf"))
    first, lse = c.run()
    check(c, first, lse)
    for _ in range(20):
        again, _ = c.run()
        assert torch.equal(first.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_mask_without_words_is_refused(dtype):
    """(Its address is that of no mask at all, which is a chain.)"""
    c = tree.Case([20], [3], 4, 2, 64, dtype, "tree", seed=1)
    c.mask = np.zeros((3, 0), np.int32)
    with pytest.raises(binding.PkvError):
        c.args(torch.empty_like(c.q))
    with pytest.raises(binding.PkvError):
        binding.decode_attention_tree(c.q, c.k, c.v, tree.i32(c.tables), tree.i32(c.lens), tree.i32(c.starts),
                                      c.scale, mask=torch.empty((3, 0), dtype=torch.int32, device=dev()))
