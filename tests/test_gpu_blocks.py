"""Copies of blocks and accepted paths (pkv_copy_blocks, pkv_tree_accept): bytes move as they are,
so everything is compared for equality."""
import numpy as np
import pytest
import torch

from helpers import dev
from oracle import drafted
from paged_kv_decode_10_gb300 import binding, workloads
from test_gpu_tree import i32, tables_of

pytestmark = pytest.mark.gpu

TD = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def pools_of(n, shape, dtype, seed):
    return [workloads.normal(shape, dtype, seed + i).to(dev()) for i in range(n)]


@pytest.mark.parametrize("n_pools,blocks,pairs,Hkv,d,dtype", [
    (1, 2, 1, 1, 64, "bf16"), (2, 64, 16, 8, 128, "bf16"), (3, 50, 25, 3, 80, "f32"),
    (256, 9, 4, 1, 8, "bf16"), (6, 900, 450, 8, 128, "f32")])
def test_copy_blocks(n_pools, blocks, pairs, Hkv, d, dtype):
    pools = pools_of(n_pools, (blocks, Hkv, 16, d), dtype, 3)
    pools[0][0] = float("nan")
    order = np.random.default_rng(pairs).permutation(blocks)
    src, dst = order[:pairs].copy(), order[pairs:2 * pairs].copy()
    want = [p.clone() for p in pools]
    for w in want:
        w[torch.from_numpy(dst).to(dev())] = w[torch.from_numpy(src).to(dev())]
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    binding.copy_blocks(pools, i32(src), i32(dst), err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    for p, w in zip(pools, want):
        assert torch.equal(p.view(torch.uint8), w.view(torch.uint8))


def test_copy_blocks_between_pools_and_bad_pairs():
    a, b = pools_of(2, (8, 2, 16, 64), "bf16", 1), pools_of(2, (20, 2, 16, 64), "bf16", 5)
    keep = [x.clone() for x in a + b]
    src, dst = [7, -1, 3, 8, 2, 1], [19, 4, -5, 6, 20, 0]
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    binding.copy_blocks(a, i32(src), i32(dst), dst_pools=b, err=err)
    torch.cuda.synchronize()
    assert int(err) == binding.DEVERR_BAD_BLOCK       # 8 of 8 and 20 of 20
    for i in range(2):
        keep[2 + i][19], keep[2 + i][0] = keep[i][7], keep[i][1]
    for x, w in zip(a + b, keep):
        assert torch.equal(x, w)
    err.zero_()
    binding.copy_blocks(a, i32([-1, -1]), i32([0, 1]), err=err)   # padding of a captured call
    binding.copy_blocks(a, i32([]), i32([]), err=err)
    torch.cuda.synchronize()
    assert int(err) == 0 and torch.equal(a[0], keep[0])


def test_copy_blocks_from_mapped_host_memory():
    """A pool swapped out to page-locked host memory and back (the kernel reads it there)."""
    pool = pools_of(1, (6, 1, 16, 64), "f32", 1)[0]
    host = torch.zeros((4, 1, 16, 64)).pin_memory()
    a = binding.make_copy_args([pool], i32([5, 0]), i32([1, 3]), dst_pools=[torch.empty_like(pool[:4])])
    a.dst[0] = binding.mapped_pointer(host).value
    binding.copy_blocks_args(a)
    torch.cuda.synchronize()
    assert torch.equal(host[1], pool[5].cpu()) and torch.equal(host[3], pool[0].cpu())
    assert not host[0].any() and not host[2].any()


def accept_case(cached, nodes, accepted, seed):
    rng = np.random.default_rng(seed)
    lens = np.array([c + n for c, n in zip(cached, nodes)], np.int32)
    starts = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    nb, tables = tables_of(lens, seed)
    most = max([1] + list(accepted))
    path = np.full((len(lens), most), -1, np.int32)
    for b, (n, a) in enumerate(zip(nodes, accepted)):
        path[b, :a] = np.sort(rng.permutation(n)[:a])
    return lens, starts, nb, tables, path, np.array(accepted, np.int32)


@pytest.mark.parametrize("n_pools,Hkv,d,dtype", [(2, 1, 64, "f32"), (2, 8, 128, "bf16"), (7, 3, 8, "bf16"),
                                                 (64, 2, 128, "f32")])
@pytest.mark.parametrize("cached,nodes,accepted", [
    ([0], [1], [1]), ([0], [1], [0]), ([5, 16, 0, 31], [12, 3, 0, 64], [4, 3, 0, 12]),
    ([100, 1], [700, 33], [600, 1]), ([7] * 20, list(range(1, 21)), [n // 2 for n in range(1, 21)])])
def test_accept_nodes(cached, nodes, accepted, n_pools, Hkv, d, dtype):
    lens, starts, nb, tables, path, counts = accept_case(cached, nodes, accepted, 3)
    pools = pools_of(n_pools, (nb, Hkv, 16, d), dtype, 11)
    want = [drafted.accept(p.float().cpu().numpy(), tables, lens, starts, path, counts) for p in pools]
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    binding.accept_nodes(pools, i32(tables), i32(lens), i32(starts), i32(path), i32(counts), err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    for p, w in zip(pools, want):
        assert np.array_equal(p.float().cpu().numpy(), w)


def test_accept_nodes_bad_rows_are_left_alone():
    nodes, cached = [6] * 9, [20] * 9
    lens, starts, nb, tables, path, counts = accept_case(cached, nodes, [3] * 9, 4)
    path[:] = [1, 3, 4]
    path[1] = [1, 1, 2]                  # does not ascend
    path[2] = [2, 4, 6]                  # a node that is not there
    path[3] = [-1, 2, 3]
    counts[4] = 4                        # longer than the path
    counts[5] = -1
    lens[6] = 5                          # fewer tokens than nodes
    tables[7, 1] = nb                    # the block of the nodes
    pools = pools_of(2, (nb, 2, 16, 64), "bf16", 2)
    ok = np.array([0, 8])
    want = [drafted.accept(p.float().cpu().numpy(), tables[ok], lens[ok],
                           np.array([0, 6, 12]), path[ok], counts[ok]) for p in pools]
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    binding.accept_nodes(pools, i32(tables), i32(lens), i32(starts), i32(path), i32(counts), err=err)
    torch.cuda.synchronize()
    assert int(err) == binding.DEVERR_BAD_LEN | binding.DEVERR_BAD_BLOCK
    for p, w in zip(pools, want):
        assert np.array_equal(p.float().cpu().numpy(), w)
