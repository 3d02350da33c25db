"""Eviction of 76 and more (row, KV head) pairs behind tables of more than 512 tokens: each
pair's keys, values and weights are walked by CTAs of their own, 1024 kept tokens to a list.
Equality, as in test_gpu_cache_ops (eviction moves bytes and picks by exact comparison)."""
import numpy as np
import pytest

from test_gpu_cache_ops import check_evict, evict_case, widened

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def test_short_rows_behind_wide_tables():
    lens = [(37 * i) % 300 for i in range(40)]
    c = evict_case(40, 2, 64, "bf16", lens, [(11 * i) % 200 for i in range(40)], 17, ties=True)
    check_evict(widened(c, 33), 3, 9, 200)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [1023, 1024, 1025, 2048, 2049, 3001])
def test_rows_of_several_lists(dtype, K):
    """The lists' ends, rows that keep fewer, all or one less than all of their tokens; the
    first tokens weigh least, so that nearly every kept token moves, across lists."""
    B, Hkv = 19, 4
    lens = [K + (97 * i) % 800 for i in range(B)]
    lens[3], lens[4], lens[5] = K, K + 1, max(K // 2, 1)
    keeps = [K if i % 4 else K - (13 * i) % 700 for i in range(B)]
    c = evict_case(B, Hkv, 64, dtype, lens, keeps, K)
    for b in range(B):
        for t in range(0, min(40, lens[b]), 1 + b % 3):     # drops near the front
            c["mass"][int(c["tab"][b, t // 16]), :, t % 16] = 0.0
    check_evict(c, 0, 16, K)


@pytest.mark.parametrize("d,dtype", [(8, "f32"), (24, "bf16"), (256, "f32"), (128, "bf16")])
def test_lists_of_other_row_sizes(d, dtype):
    lens = [1700 + 11 * i for i in range(26)]
    c = evict_case(26, 3, d, dtype, lens, [1100 + 7 * i for i in range(26)], d, ties=True)
    check_evict(c, 0, 0, 1100 + 7 * 25)


def test_one_token_dropped_at_the_front_shifts_every_list():
    c = evict_case(80, 1, 64, "bf16", [2500] * 80, [2499] * 80, 9)
    first = c["tab"][:, 0].astype(np.int64)
    c["mass"][first, :, 0] = -1.0
    check_evict(c, 0, 0, 2499)
    np.testing.assert_array_equal(c["mass"].cpu().numpy()[first, 0, 0] >= 0, True)
