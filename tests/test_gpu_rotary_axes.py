"""Rotary positions with several axes (pkv_rotary_axes_append) against the float64 oracle.

Tolerance, from the arithmetic (u: half a step of the storage type): the angle is rounded once to
float32 (|angle| <= pi: 2^-23 absolute at most) and sincosf is good to 2 units (2^-23), so cos
and sin are off by at most 2^-22 each; two products, their sum and the amplitude on each of cos
and sin add roundings of 2^-24; then the rounding to storage:
|y - y*| <= u |y| + amplitude * (|x1| + |x2|) * 2^-21.
"""
import numpy as np
import pytest
import torch

from helpers import dev, f64
from oracle import cache_ops, drafted
from paged_kv_decode_10_gb300 import binding
from test_gpu_tree import U, i32, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def frequencies(sections, axis, number, ladder, scaling, **kw):
    if ladder == "shared":
        return cache_ops.rotary_frequencies(2 * sum(sections), scaling, **kw)
    own = [cache_ops.rotary_frequencies(2 * n, scaling, **kw) if n else [] for n in sections]
    return np.array([own[a][k] for a, k in zip(axis, number)])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("order", ["blocked", "cyclic"])
@pytest.mark.parametrize("d,sections,ladder,scaling,T,Hq,Hkv", [
    (128, (16, 24, 24), "shared", "plain", 1, 8, 2), (128, (24, 20, 20), "own", "linear", 300, 4, 1),
    (64, (16, 16), "own", "plain", 33, 3, 3), (64, (5, 6, 7), "shared", "bands", 700, 8, 8),
    (80, (3, 0, 4, 1), "own", "plain", 17, 5, 1), (256, (128,), "shared", "ramp", 3, 2, 2),
    (128, (8,) * 8, "own", "ntk", 40, 12, 4)])
def test_rotary_axes(d, sections, ladder, scaling, T, Hq, Hkv, order, layout, dtype):
    extra = {"plain": {}, "linear": dict(factor=8.0), "ntk": dict(factor=4.0),
             "ramp": dict(factor=16.0, original_len=4096),
             "bands": dict(factor=8.0, original_len=8192, low=1.0, high=4.0, base=500000.0)}[scaling]
    rng = np.random.default_rng(T + d)
    wide = normal((T, Hq + 2 * Hkv, d), dtype, 7)
    q, k, v = wide[:, :Hq], wide[:, Hq:Hq + Hkv], wide[:, Hq + Hkv:]
    pos = rng.integers(-5, 1 << 20, (len(sections), T))
    pos[0, 0] = 2**31 - 1
    nb = -(-T // 16) + 2
    slots = rng.permutation(nb * 16)[:T].astype(np.int64)
    kc, vc = normal((nb, Hkv, 16, d), dtype, 8), normal((nb, Hkv, 16, d), dtype, 9)
    k0, v0, keep = kc.clone(), vc.clone(), wide.clone()
    rot = 2 * sum(sections)
    table = binding.Rotary(d, rot_dim=rot, layout=layout, scaling=scaling, amplitude=1.25,
                           sections=sections, order=order, ladder=ladder, **extra)
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    qo, ko = binding.rotary_append(table, q, k, v, i32(pos), torch.from_numpy(slots).to(dev()), kc, vc,
                                   err=err)
    torch.cuda.synchronize()
    assert int(err) == 0 and torch.equal(wide, keep)
    axis, number = drafted.axes_of(sections, order)
    freq = frequencies(sections, axis, number, ladder, scaling, **extra)
    n = rot // 2
    first = np.arange(n) if layout == "half" else 2 * np.arange(n)
    second = first + n if layout == "half" else first + 1
    for got, x in ((qo, q), (ko, k)):
        x = f64(x)
        want = drafted.rotary_axes(x, pos, freq, axis, layout, 1.25)
        size = np.abs(x[..., first]) + np.abs(x[..., second])
        tol = np.zeros_like(x)
        tol[..., first] = tol[..., second] = 1.25 * size * 2.0**-21
        tol[..., :rot] += U[dtype] * np.abs(want[..., :rot])
        bad = np.abs(f64(got) - want) > tol
        assert not bad.any(), (np.argwhere(bad)[:3], f64(got)[bad][:3], want[bad][:3])
    for t in range(T):
        b, r = divmod(int(slots[t]), 16)
        k0[b, :, r], v0[b, :, r] = ko[t], v[t]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_equal_positions_turn_like_one_axis(dtype):
    """The same position on every axis gives the values without axes, bit for bit."""
    x = normal((50, 6, 128), dtype, 1)
    pos = np.random.default_rng(1).integers(0, 1 << 17, 50)
    one = binding.rotary_append(binding.Rotary(128), x, None, None, i32(pos))[0]
    for order in ("blocked", "cyclic"):
        rot = binding.Rotary(128, sections=(16, 24, 24), order=order)
        got = binding.rotary_append(rot, x, None, None, i32(np.stack([pos] * 3)))[0]
        assert torch.equal(got, one)
