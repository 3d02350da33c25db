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


@pytest.mark.parametrize("scale", [0.0, -0.11, 3.0])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scales(scale, dtype):
    c = Case([200, 3], [40, 7], 8, 2, 64, dtype, "any", seed=5)
    c.scale = scale
    c.check(*c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G,kind", [(1, "tree"), (8, "tree"), (8, "chain"), (2, "chain"), (4, "any")])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_what_a_node_does_not_see_may_be_anything(value, G, kind, dtype):
    """Nodes whose key and value (and query) are not finite: those that see them get what the
    formula gives, the others nothing of it."""
    nodes = [40, 150, 3]
    c = Case([130, 0, 17], nodes, 2 * G, 2, 128, dtype, kind, seed=8, extra=1)
    if kind == "chain":
        spoiled = {0: [38, 39], 1: [140], 2: [2]}
    else:
        spoiled = {0: [5, 39], 1: [60, 130, 149], 2: [1]}
    for b, some in spoiled.items():
        base = int(c.lens[b]) - nodes[b]
        for i in some:
            blk, r = c.tables[b, (base + i) // 16], (base + i) % 16
            if i % 2:
                c.k[blk, :, r] = value
            c.v[blk, :, r, ::3] = value
    c.q[int(c.starts[1]) + 7] = value
    c.check(*c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scores_that_are_all_minus_infinity_give_nan(dtype):
    c = Case([0, 20], [2, 3], 2, 2, 64, dtype, "chain", seed=2)
    c.k.fill_(float("-inf"))
    c.q.copy_(c.q.abs() + 1)
    out, lse = c.run()
    assert torch.isnan(out).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_do_not_fit_are_left_alone(dtype):
    c = Case([30] * 6, [4] * 6, 4, 2, 64, dtype, "tree", seed=3, extra=2)
    good = c.run()[0]
    c.lens[1] = 3                                   # fewer tokens than nodes
    c.lens[2] = 16 * c.tables.shape[1] + 1          # more than its table
    c.lens[4] = -1
    out = torch.full_like(good, 7.0)
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    binding.decode_attn_tree_args(c.args(out, err=err))
    torch.cuda.synchronize()
    assert int(err) == binding.DEVERR_BAD_LEN
    for b in range(6):
        a, e = int(c.starts[b]), int(c.starts[b + 1])
        assert torch.equal(out[a:e], torch.full_like(out[a:e], 7.0) if b in (1, 2, 4) else good[a:e])
    # starts that do not ascend, or leave the queries
    for starts in ([0, 4, 2, 12, 16, 20, 24], [-4, 4, 8, 12, 16, 20, 24], [0, 4, 8, 12, 16, 20, 99]):
        c.starts = np.array(starts, np.int32)
        err.zero_()
        binding.decode_attn_tree_args(c.args(out, err=err))
        torch.cuda.synchronize()
        assert int(err) & binding.DEVERR_BAD_LEN
    # a row with more nodes than mask bits
    c = Case([0, 30], [33, 4], 4, 2, 64, dtype, "tree", seed=3)
    good = c.run()[0]
    c.mask = np.ascontiguousarray(c.mask[:, :1])
    out, err = torch.full_like(good, 7.0), torch.zeros(1, dtype=torch.int32, device=dev())
    binding.decode_attn_tree_args(c.args(out, err=err))
    torch.cuda.synchronize()
    assert int(err) == binding.DEVERR_BAD_LEN
    assert (out[:33] == 7.0).all() and torch.equal(out[33:], good[33:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["tree", "chain"])
def test_blocks_outside_the_pool_are_left_out(kind, dtype):
    c = Case([400, 90], [20, 70], 8, 2, 128, dtype, kind, seed=4)
    whole = c.run()[0]
    for b, j, bad in ((0, 3, -1), (0, 25, 10**6), (1, 5, -7)):
        c.tables[b, j] = bad
    out, err = torch.full_like(whole, 7.0), torch.zeros(1, dtype=torch.int32, device=dev())
    lse = torch.empty(whole.shape[:2], device=dev())
    binding.decode_attn_tree_args(c.args(out, lse=lse, err=err))
    torch.cuda.synchronize()
    assert int(err) == binding.DEVERR_BAD_BLOCK
    # the same as not seeing those tokens: every row alone, its tokens as nodes of a wide mask
    for b in range(2):
        L, n = int(c.lens[b]), int(c.starts[b + 1] - c.starts[b])
        a = int(c.starts[b])
        there = np.array([0 <= c.tables[b, t // 16] < len(c.k) for t in range(L)])
        sees = drafted.tree_visible(c.mask, a, n, L - n) & there
        tab = np.where((c.tables[b] >= 0) & (c.tables[b] < len(c.k)), c.tables[b], 0)[None]
        words = np.packbits(np.pad(sees, ((L - n, 0), (0, -L % 32))), axis=1, bitorder="little").view("<i4")
        q = np.zeros((L,) + tuple(c.q.shape[1:]))
        q[L - n:] = f64(c.q)[a:a + n]
        kv = [np.nan_to_num(f64(x)) for x in (c.k, c.v)]
        want = drafted.tree_attention(q, *kv, tab, [L], [0, L], c.scale, words)
        check(f64(out)[a:a + n], f64(lse)[a:a + n], [x[L - n:] for x in want], dtype, 128)


def test_rows_that_share_blocks_and_rows_without_nodes():
    """Forks: three rows over the same whole blocks, each with nodes of its own; one has none."""
    c = Case([64, 64, 64], [5, 0, 9], 8, 2, 64, "bf16", "tree", seed=6)
    for b in (1, 2):
        c.tables[b, :4] = c.tables[0, :4]
    c.check(*c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_replayed_graphs_that_share_a_workspace(dtype):
    cases = [Case([300, 20], [30, 9], 8, 2, 128, dtype, "tree", seed=1),
             Case([10] * 9, [3] * 9, 8, 2, 128, dtype, "chain", seed=2)]
    space = torch.full((binding.tree_workspace_bytes(8, 2, 128, binding.dtype_code(cases[0].q)),), 255,
                       dtype=torch.uint8, device=dev())
    side = torch.cuda.Stream()
    graphs, outs = [], []
    for c in cases:
        out = torch.zeros_like(c.q)
        args = c.args(out, workspace=space)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            binding.decode_attn_tree_args(args)
        graphs.append((g, args))
        outs.append(out)
    for _ in range(3):
        for (g, _), out in zip(graphs, outs):
            out.zero_()
            g.replay()
    torch.cuda.synchronize()
    for c, out in zip(cases, outs):
        assert torch.equal(out, c.run()[0])


def test_side_stream_and_plain_call():
    c = Case([100, 7], [12, 5], 8, 2, 64, "bf16", "tree", seed=9)
    want = c.run()[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = binding.decode_attention_tree(c.q, c.k, c.v, i32(c.tables), i32(c.lens), i32(c.starts), c.scale,
                                        mask=i32(c.mask), stream=side)
    side.synchronize()
    assert torch.equal(out, want)


def test_metadata_in_mapped_host_memory():
    c = Case([100, 7], [12, 5], 8, 2, 64, "bf16", "tree", seed=9)
    want = c.run()[0]
    host = [torch.from_numpy(np.ascontiguousarray(x, np.int32)).pin_memory()
            for x in (c.tables, c.lens, c.starts)]
    out = binding.decode_attention_tree(c.q, c.k, c.v, *host, c.scale, mask=i32(c.mask))
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_waits_that_give_up_leave_nan_and_the_next_call_is_whole():
    c = Case([4000, 50], [40, 9], 8, 2, 128, "bf16", "tree", seed=9)
    want = c.run()[0]
    space = torch.zeros(binding.tree_workspace_bytes(8, 2, 128, binding.BF16), dtype=torch.uint8,
                        device=dev())
    out, err = torch.full_like(want, 7.0), torch.zeros(1, dtype=torch.int32, device=dev())
    binding.decode_attn_tree_args(c.args(out, workspace=space, err=err, flags=binding.ATTN_SHORT_WAITS))
    torch.cuda.synchronize()
    assert int(err) == binding.DEVERR_TIMEOUT
    assert torch.isnan(out).any() and (torch.isnan(out) | (out == want)).all()
    err.zero_()
    binding.decode_attn_tree_args(c.args(out, workspace=space, err=err))
    torch.cuda.synchronize()
    assert int(err) == 0 and torch.equal(out, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_caches_beyond_32_bit_offsets(dtype):
    """Blocks whose first byte lies beyond 2^32 elements."""
    Hkv, d = 8, 128
    nb = 2**32 // (Hkv * 16 * d) + 40
    small = Case([200, 33], [20, 5], 16, Hkv, d, dtype, "tree", seed=11)
    want = small.run()[0]
    far = nb - 1 - np.arange(len(small.k))
    k, v = (torch.empty((nb, Hkv, 16, d), dtype=TD[dtype], device=dev()) for _ in range(2))
    idx = torch.from_numpy(far).to(dev())
    k[idx], v[idx] = small.k, small.v
    small.k, small.v = k, v
    small.tables = np.where(small.tables >= 0, far[np.maximum(small.tables, 0)], -1).astype(np.int32)
    assert torch.equal(small.run()[0], want)


def test_a_batch_of_many_rows():
    """More rows than threads that look for a CTA's share, lengths and nodes of every kind."""
    rng = np.random.default_rng(5)
    B = 1000
    nodes = rng.integers(0, 5, B)
    cached = np.where(rng.random(B) < 0.1, 0, rng.integers(0, 40, B))
    for dtype in ("bf16", "f32"):
        c = Case(cached, nodes, 2, 1, 64, dtype, "tree", seed=12)
        c.check(*c.run())


@pytest.mark.parametrize("d,Hkv", [(128, 8), (64, 4)])
@pytest.mark.parametrize("kind", ["tree", "chain"])
def test_many_items_of_many_steps_to_a_cta(d, Hkv, kind):
    """Several items to a CTA, of one or both row tiles and of 1 to 20 steps, in every order."""
    rng = np.random.default_rng(d)
    B = 48
    nodes = rng.choice([1, 3, 8, 16, 40, 70], B)
    cached = rng.choice([0, 5, 100, 600, 1100, 2400], B)
    c = Case(cached, nodes, 4 * Hkv, Hkv, d, "bf16", kind, seed=13)
    first, lse = c.run()
    for _ in range(3):
        again, _ = c.run()
        assert torch.equal(first, again)
    c.check(first, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tensors_aligned_to_16_bytes(dtype):
    """Queries and outputs that begin 16 bytes into a buffer."""
    c = Case([100, 7, 900], [12, 5, 70], 8, 2, 128, dtype, "tree", seed=9)
    want = c.run()[0]
    skip = 16 // c.q.element_size()
    buf = torch.empty(2, c.q.numel() + 2 * skip, dtype=c.q.dtype, device=dev())
    q, out = (b[skip:skip + c.q.numel()].view(c.q.shape) for b in buf)
    q.copy_(c.q)
    buf[1] = 7.0
    assert out.data_ptr() % 32 == 16 or q.data_ptr() % 32 == 16
    c.q = q
    binding.decode_attn_tree_args(c.args(out))
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert (buf[1, :skip] == 7.0).all() and (buf[1, -skip:] == 7.0).all()


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("f32", 128), ("bf16", 64)])
def test_whatever_a_wait_gave_up_on_is_nan(dtype, d):
    """Items of many parts and whole ones: every output is its value or NaN, none is left as it was."""
    c = Case([4000, 50, 3, 900], [40, 9, 1, 70], 8, 2, d, dtype, "tree", seed=9)
    want = c.run()[0]
    for _ in range(5):
        out, err = torch.full_like(want, 7.0), torch.zeros(1, dtype=torch.int32, device=dev())
        binding.decode_attn_tree_args(c.args(out, err=err, flags=binding.ATTN_SHORT_WAITS))
        torch.cuda.synchronize()
        assert int(err) == binding.DEVERR_TIMEOUT
        assert torch.isnan(out).any() and (torch.isnan(out) | (out == want)).all()
    assert torch.equal(c.run()[0], want)


def test_lengths_written_by_the_kernel_before():
    """Metadata that a kernel ahead on the stream writes (its call may start while that one runs)."""
    c = Case([300, 7], [12, 5], 8, 2, 128, "bf16", "tree", seed=9)
    want = c.run()[0]
    out = torch.zeros_like(want)
    args = c.args(out)
    block_tables, lens, starts, mask = (args.keep[i] for i in (3, 4, 5, 7))
    wrong, right = [], []
    for t in (block_tables, lens, starts, mask):
        right.append(t.clone())
        wrong.append(torch.zeros_like(t))
    busy = torch.randn(4096, 4096, device=dev())
    for _ in range(3):
        for t, w in zip((block_tables, lens, starts, mask), wrong):
            t.copy_(w)
        busy = busy @ busy * 1e-3
        for t, r in zip((block_tables, lens, starts, mask), right):
            t.copy_(r)
        binding.decode_attn_tree_args(args)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        out.zero_()
