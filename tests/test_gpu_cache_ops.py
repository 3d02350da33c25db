"""GPU parity of the cache operators (rotary layouts and scalings with the append,
shared-prefix attention with weights, eviction) against their float64 oracle.

Tolerances, from the arithmetic (u = unit roundoff of the storage type, 2^-8 for bf16 and
2^-24 for float32):
* rotary: the angle is rounded once to float32 (|angle| <= pi: 2^-23 absolute at most) and
  sincosf is good to 2 units (2^-23), so cos and sin are off by at most 2^-22 each; the two
  products and their sum add 3 roundings of 2^-24; amplitude one more on each of cos and
  sin; then the rounding to storage u |y|.
  |y - y*| <= u |y| + amplitude * (|x1| + |x2|) * 2^-21.
* attention scores: d products accumulated in float32 (d + 4 roundings of up to 2^-23 each,
  accumulators that truncate included), times scale, relative to the row's largest score
  (bounded by swing = scale * max_t sum |q||k|): delta = (d + 8) * 2^-23 * swing + 2^-20.
  Weights are off by a factor within exp(2 delta) and by ex2's 2^-22; the own factor of
  bf16 is the weights' rounding to bf16 ahead of the P.V product.
  |out - out*| <= (2 delta + 2^-18 [+ u for bf16]) * sum p|v| + u |out| ;
  |mass - mass*| <= (2 delta + 2^-18) * weight + 2^-23 |mass| ; |lse - lse*| <= delta + 2^-19 (1 + |lse|).
* eviction moves bytes and picks by exact comparison: equality.
"""
import numpy as np
import pytest
import torch

from helpers import dev, f64
from oracle import cache_ops
from oracle.numerics import round_to
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


def tables_for(lists, seed, spare=0.25):
    """Scattered block tables of several lists of lengths; (num_blocks, [numpy tables])."""
    rng = np.random.default_rng(seed)
    total = sum(-(-int(n) // 16) for lens in lists for n in lens)
    nb = max(1, total + max(1, int(spare * total)))
    free = list(rng.permutation(nb))
    got = []
    for lens in lists:
        w = max([1] + [-(-int(n) // 16) for n in lens])
        t = np.full((max(len(lens), 1), w), -1, np.int32)
        for i, n in enumerate(lens):
            for j in range(-(-int(n) // 16)):
                t[i, j] = free.pop()
        got.append(t)
    return nb, got


# --------------------------------------------------------------------------- rotary
SCALINGS = {
    "plain": {}, "linear": dict(factor=8.0), "ntk": dict(factor=4.0),
    "ramp": dict(factor=16.0, original_len=4096, amplitude=1.2772588722239782),
    "bands": dict(factor=8.0, original_len=8192, low=1.0, high=4.0, base=500000.0)}


def check_rotary(got, x, pos, dtype, rot, layout, scaling):
    kw = dict(SCALINGS[scaling])
    amp = kw.pop("amplitude", 1.0)
    freq = cache_ops.rotary_frequencies(rot, scaling, **kw)
    x = f64(x)
    want = cache_ops.rotary(x, pos, freq, layout, amp)
    n = rot // 2
    first = np.arange(n) if layout == "half" else 2 * np.arange(n)
    second = first + n if layout == "half" else first + 1
    size = np.abs(x[..., first]) + np.abs(x[..., second])
    tol = np.zeros_like(x)
    tol[..., first] = tol[..., second] = amp * size * 2.0**-21
    tol[..., :rot] += U[dtype] * np.abs(want[..., :rot])
    bad = np.abs(f64(got) - want) > tol
    assert not bad.any(), (np.argwhere(bad)[:3], f64(got)[bad][:3], want[bad][:3])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot,scaling,T,Hq,Hkv", [
    (128, 128, "plain", 1, 8, 2), (128, 128, "ramp", 5, 32, 8), (128, 64, "bands", 305, 4, 1),
    (64, 32, "linear", 33, 3, 3), (64, 16, "ntk", 700, 8, 8), (80, 20, "plain", 17, 5, 1),
    (256, 256, "bands", 3, 2, 2), (8, 2, "linear", 4, 1, 1), (96, 96, "plain", 40, 12, 4)])
def test_rotary_append(dtype, layout, d, rot, scaling, T, Hq, Hkv):
    rng = np.random.default_rng(T + d)
    wide = normal((T, Hq + 2 * Hkv, d), dtype, 7)       # q, k, v as slices of one projection
    q, k, v = wide[:, :Hq], wide[:, Hq:Hq + Hkv], wide[:, Hq + Hkv:]
    pos = rng.integers(-5, 1 << 20, T)
    pos[0] = 2**31 - 1 if T > 1 else 131072
    nb = -(-T // 16) + 2
    slots = rng.permutation(nb * 16)[:T].astype(np.int64)
    slots[-1] = -1 if T > 2 else slots[-1]
    kc, vc = normal((nb, Hkv, 16, d), dtype, 8), normal((nb, Hkv, 16, d), dtype, 9)
    k0, v0 = kc.clone(), vc.clone()
    rot_t = binding.Rotary(d, rot_dim=rot, layout=layout, scaling=scaling, **SCALINGS[scaling])
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    keep = wide.clone()
    qo, ko = binding.rotary_append(rot_t, q, k, v, i32(pos),
                                   torch.from_numpy(slots).to(dev()), kc, vc, err=err)
    torch.cuda.synchronize()
    assert int(err) == 0 and torch.equal(wide, keep)
    check_rotary(qo, q, pos, dtype, rot, layout, scaling)
    check_rotary(ko, k, pos, dtype, rot, layout, scaling)
    assert torch.equal(qo[..., rot:], q[..., rot:])
    for t in range(T):
        if slots[t] >= 0:
            b, r = divmod(int(slots[t]), 16)
            assert torch.equal(kc[b, :, r], ko[t]) and torch.equal(vc[b, :, r], v[t])
            k0[b, :, r], v0[b, :, r] = ko[t], v[t]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)     # nothing else was written
    # in place, and without reporting the keys
    wide2 = wide.clone()
    q2, k2, v2 = wide2[:, :Hq], wide2[:, Hq:Hq + Hkv], wide2[:, Hq + Hkv:]
    binding.rotary_append(rot_t, q2, k2, None, i32(pos), q_out=q2, k_out=k2)
    assert torch.equal(q2, qo) and torch.equal(k2, ko) and torch.equal(v2, v)
    kc2, vc2 = normal((nb, Hkv, 16, d), dtype, 8), normal((nb, Hkv, 16, d), dtype, 9)
    a = binding.make_rotary_args(rot_t, None, k, v, i32(pos), slot_mapping=torch.from_numpy(slots).to(dev()),
                                 k_cache=kc2, v_cache=vc2)
    binding.rotary_append_args(a)
    assert torch.equal(kc2, kc) and torch.equal(vc2, vc)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_plain_rotary_is_the_rope_kernels(dtype):
    q, k, v = normal((9, 8, 64), dtype, 1), normal((9, 2, 64), dtype, 2), normal((9, 2, 64), dtype, 3)
    pos = i32(np.arange(9) * 14563)
    caches = [normal((3, 2, 16, 64), dtype, 4 + i % 2) for i in range(4)]
    slots = torch.arange(9, device=dev()) * 5
    a = binding.rope_append(q, k, v, pos, slots, caches[0], caches[1])
    b = binding.rotary_append(binding.Rotary(64), q, k, v, pos, slots, caches[2], caches[3])
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])


def test_rotary_unaligned_tensors_and_bad_slots():
    """Element-aligned tensors take the narrow path; a slot beyond the pool is flagged."""
    flat = normal((4 * 3 * 64 + 1,), "bf16", 5)
    q = flat[1:].view(4, 3, 64)
    k, v = normal((4, 2, 64), "bf16", 6), normal((4, 2, 64), "bf16", 7)
    pos = i32([0, 1, 2, 1 << 30])
    kc, vc = normal((2, 2, 16, 64), "bf16", 8), normal((2, 2, 16, 64), "bf16", 9)
    k0 = kc.clone()
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    slots = torch.tensor([3, 32, -7, 31], device=dev())
    qo, ko = binding.rotary_append(binding.Rotary(64), q, k, v, pos, slots, kc, vc, err=err)
    check_rotary(qo, q, [0, 1, 2, 1 << 30], "bf16", 64, "half", "plain")
    assert int(err) == binding.DEVERR_BAD_SLOT
    k0[0, :, 3], k0[1, :, 15] = ko[0], ko[3]
    assert torch.equal(kc, k0)


# --------------------------------------------------------------------------- attention
def make_case(B, Hq, Hkv, d, dtype, lens, plens, rows, seed, bias=False, mass=False):
    nb, (tab, ptab) = tables_for([lens, plens], seed)
    c = dict(B=B, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, lens=np.asarray(lens), plens=plens, rows=rows,
             nb=nb, tab=tab, ptab=ptab, q=normal((B, Hq, d), dtype, seed + 1),
             kc=normal((nb, Hkv, 16, d), dtype, seed + 2), vc=normal((nb, Hkv, 16, d), dtype, seed + 3),
             scale=d**-0.5)
    # what lies behind the tokens of a last page belongs to nobody and may hold anything
    for t, ls in ((tab, lens), (ptab, plens)):
        for i, n in enumerate(ls):
            if n % 16:
                for cache in (c["kc"], c["vc"]):
                    cache[int(t[i, n // 16]), :, n % 16:] = float("nan")
    c["bias"] = None
    if bias:
        rng = np.random.default_rng(seed)
        x = rng.normal(size=(B, max(max(lens), 1))).astype(np.float32)
        x[rng.random(x.shape) < 0.3] = -np.inf
        x[0] = -np.inf
        x[B // 2] = np.finfo(np.float32).min      # a mask of the type's lowest value
        c["bias"] = torch.from_numpy(x).to(dev())
    if mass:
        c["mass"] = torch.rand((nb, Hkv, 16), generator=torch.Generator().manual_seed(seed)).to(dev())
        c["mass"][torch.rand(c["mass"].shape, device=dev()) < 0.02] = float("nan")   # stale slots
        c["known"] = np.maximum(np.asarray(lens) - 1 - (np.arange(B) % 3), 0)
        for b in range(B):      # weights that count are finite
            for t in range(c["known"][b]):
                c["mass"][int(tab[b, t // 16]), :, t % 16].nan_to_num_(nan=0.25)
    return c


def run_case(c, out=None, **kw):
    B = c["B"]
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    lse = torch.empty((B, c["Hq"]), device=dev())
    if kw.pop("general", False):   # a stated number of parts: not the form for short contexts
        kw["num_parts"] = binding.shared_default_parts(B, c["Hq"], c["kc"].shape[1], c["d"],
                                                       binding.dtype_code(c["q"]), c["tab"].shape[1])
    out = torch.full_like(c["q"], 7.0) if out is None else out
    if len(c["plens"]):
        plan = binding.shared_plan(c["rows"], c["plens"], c["Hq"], c["Hkv"], c["d"],
                                   binding.dtype_code(c["q"]), kw.pop("num_ctas", 0))
        kw.update(prefix_tables=torch.from_numpy(c["ptab"]).to(dev()),
                  prefix_plan=torch.from_numpy(plan).to(dev()))
    if "mass" in c:
        kw.update(mass=c["mass"], scores=binding.alloc_scores(c["nb"], c["Hq"]),
                  mass_lens=i32(c["known"]), decay=0.75)
    a = binding.make_shared_args(c["q"], c["kc"], c["vc"], torch.from_numpy(c["tab"]).to(dev()),
                                 i32(c["lens"]), c["scale"], out, lse=lse, attn_bias=c["bias"],
                                 err=err, **kw)
    binding.decode_attn_shared_args(a)
    torch.cuda.synchronize()
    return out, lse, int(err), a


def excluded(bias):
    """The bias with what is too low for float32 in base 2 as -inf (as the call states)."""
    if bias is None:
        return None
    x = bias.cpu().numpy().astype(np.float64)
    return np.where(x < -2.35e38, -np.inf, x)


def check_case(c, out, lse, mass0=None, want_err=0, err=0):
    dtype, d = c["dtype"], c["d"]
    assert err == want_err
    kc, vc = np.nan_to_num(f64(c["kc"])), np.nan_to_num(f64(c["vc"]))
    ref = cache_ops.shared_attention(f64(c["q"]), kc, vc, c["tab"], c["lens"], c["scale"], c["ptab"],
                                     c["plens"], c["rows"] if len(c["plens"]) else None,
                                     excluded(c["bias"]))
    got, got_lse = f64(out), f64(lse)
    for b, (o, l, w, absv, swing) in enumerate(ref):
        delta = (d + 8) * 2.0**-23 * swing + 2.0**-20
        tol = (2 * delta + 2.0**-18 + (U[dtype] if dtype == "bf16" else 0))[:, None] * absv
        tol = tol + U[dtype] * np.abs(o)
        bad = ~(np.abs(got[b] - o) <= tol)
        assert not bad.any(), (b, np.argwhere(bad)[:3], got[b][bad][:3], o[bad][:3], tol[bad][:3])
        dead = np.isneginf(l)
        assert np.isneginf(got_lse[b][dead]).all() and (got[b][dead] == 0).all()
        big = np.abs(l[~dead])
        assert (np.abs(got_lse[b][~dead] - l[~dead]) <= delta[~dead] + 2.0**-19 * (1 + big)).all(), b
        if mass0 is not None:
            n = int(c["lens"][b])
            t = np.arange(n)
            blk = c["tab"][b][t // 16]
            m0 = mass0[blk, :, t % 16].T
            want = np.where(t < c["known"][b], 0.75 * np.nan_to_num(m0), 0.0) + w
            gm = f64(c["mass"])[blk, :, t % 16].T
            dg = delta.reshape(c["Hkv"], -1).max(1)[:, None]
            ok = np.abs(gm - want) <= (2 * dg + 2.0**-18) * w + 2.0**-22 * np.abs(want)
            assert ok.all(), (b, np.argwhere(~ok)[:3], gm[~ok][:3], want[~ok][:3])
    if mass0 is not None:     # every other slot is as it was
        own = np.zeros((c["nb"], 16), bool)
        for b in range(c["B"]):
            t = np.arange(int(c["lens"][b]))
            own[c["tab"][b][t // 16], t % 16] = True
        keep = ~own[:, None, :].repeat(c["Hkv"], 1)
        np.testing.assert_array_equal(f64(c["mass"])[keep], mass0[keep])


SHARED = [
    # B, Hq, Hkv, d, lens, plens, rows
    (1, 1, 1, 64, [1], [1], [0]),
    (1, 8, 1, 128, [0], [17], [0]),
    (2, 4, 2, 64, [0, 0], [0, 5], [0, -1]),                       # rows with nothing at all
    (3, 8, 2, 128, [5, 16, 33], [100], [0, 0, 0]),
    (4, 8, 8, 64, [1, 2, 15, 16], [128], [0, -1, 0, 0]),
    (5, 16, 2, 128, [0, 1, 300, 31, 32], [129, 127], [0, 1, 1, 0, -1]),
    (37, 8, 2, 128, list(range(37)), [250, 1, 31], [i % 4 - 1 for i in range(37)]),
    (70, 8, 1, 64, [3] * 70, [400], [0] * 70),                    # several row tiles
    (130, 4, 1, 128, [0] * 65 + [1] * 65, [513], [0] * 130),
    (33, 8, 1, 128, [1] * 33, [2000], [0] * 33),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("general", [False, True])
@pytest.mark.parametrize("i", range(len(SHARED)))
def test_shared_attention(dtype, i, general):
    B, Hq, Hkv, d, lens, plens, rows = SHARED[i]
    c = make_case(B, Hq, Hkv, d, dtype, lens, plens, rows, 11 * i)
    out, lse, err, _ = run_case(c, general=general)
    check_case(c, out, lse, err=err)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("ctas", [1, 3, 40])
@pytest.mark.parametrize("parts", [1, 9])
def test_shared_attention_under_other_partitions(dtype, ctas, parts):
    c = make_case(9, 8, 2, 64, dtype, [40, 0, 7, 100, 16, 1, 33, 64, 2], [700, 129], [0, 1] * 4 + [0], 3)
    out, lse, err, _ = run_case(c, num_ctas=ctas, num_parts=parts)
    check_case(c, out, lse, err=err)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("general", [False, True])
@pytest.mark.parametrize("plens", [[], [90, 300]])
def test_weights_are_accumulated(dtype, G, plens, general):
    B = 7
    rows = [-1, 0, 1, 0, 1, 0, -1] if plens else [-1] * B
    c = make_case(B, 2 * G, 2, 64 if G < 4 else 128, dtype, [0, 1, 2, 17, 64, 200, 33], plens, rows, G,
                  mass=True)
    m0 = f64(c["mass"])
    out, lse, err, a = run_case(c, general=general)
    check_case(c, out, lse, m0, err=err)
    # a second call goes on from there
    m1 = f64(c["mass"])
    binding.decode_attn_shared_args(a)
    torch.cuda.synchronize()
    check_case(c, out, lse, m1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("general", [False, True])
@pytest.mark.parametrize("plens", [[], [64]])
def test_masks_on_own_tokens(dtype, plens, general):
    c = make_case(5, 8, 2, 64, dtype, [20, 33, 16, 1, 50], plens, [0, 0, -1, 0, 0], 5, bias=True, mass=True)
    m0 = f64(c["mass"])
    out, lse, err, _ = run_case(c, general=general)
    check_case(c, out, lse, m0, err=err)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_default_new_token_and_planned_partition(dtype):
    """Without mass_lens the newest token starts from zero; a host plan of the own tokens
    gives the same result."""
    c = make_case(6, 8, 2, 64, dtype, [1, 16, 17, 40, 90, 2], [70], [0, 0, -1, 0, 0, 0], 21, mass=True)
    c["known"] = np.maximum(c["lens"] - 1, 0)
    for b in range(6):
        for t in range(c["known"][b]):
            c["mass"][int(c["tab"][b, t // 16]), :, t % 16].nan_to_num_(nan=0.25)
    m0, first = f64(c["mass"]), c["mass"].clone()
    out, lse, err, _ = run_case(c)
    check_case(c, out, lse, m0, err=err)
    want = c["mass"].clone()
    c["mass"].copy_(first)
    plan = torch.from_numpy(binding.plan_parts(c["lens"], 2, 64, c["tab"], 12)).to(dev())
    a = binding.make_shared_args(
        c["q"], c["kc"], c["vc"], torch.from_numpy(c["tab"]).to(dev()), i32(c["lens"]), c["scale"],
        torch.empty_like(out), prefix_tables=torch.from_numpy(c["ptab"]).to(dev()),
        prefix_plan=torch.from_numpy(binding.shared_plan(c["rows"], c["plens"], 8, 2, 64,
                                                         binding.dtype_code(out))).to(dev()),
        mass=c["mass"], scores=binding.alloc_scores(c["nb"], 8), decay=0.75, plan=plan,
        flags=binding.ATTN_CHECK_PLAN)
    binding.decode_attn_shared_args(a)
    # another split of the own tokens: the same sums in another order
    torch.testing.assert_close(c["mass"], want, rtol=2.0**-16, atol=0, equal_nan=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("general", [False, True])
def test_a_row_alone_equals_the_batch_without_sharing(dtype, general):
    """The same tokens as one long own sequence, through the framework's attention."""
    c = make_case(4, 8, 2, 128, dtype, [33, 1, 16, 70], [160], [0] * 4, 31)
    out, lse, err, _ = run_case(c, general=general)
    joined = np.full((4, 10 + 5), -1, np.int32)
    for b in range(4):
        n = -(-int(c["lens"][b]) // 16)
        joined[b, :10] = c["ptab"][0]
        joined[b, 10:10 + n] = c["tab"][b, :n]
    ref = binding.decode_attention(c["q"], c["kc"], c["vc"], torch.from_numpy(joined).to(dev()),
                                   i32(c["lens"] + 160), c["scale"])
    # weights of each side are rounded to bf16 on their own
    tol = dict(rtol=2 * U[dtype], atol=2e-2 if dtype == "bf16" else 2e-6)
    torch.testing.assert_close(out.float(), ref.float(), **tol)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("general", [False, True])
def test_bad_blocks_and_plans_are_flagged(dtype, general):
    c = make_case(3, 8, 2, 64, dtype, [5, 40, 20], [100, 40], [0, 0, 1], 41)
    good = c["ptab"].copy()
    c["ptab"][0, 3] = c["nb"]          # tokens 48..63 of prefix 0 drop out
    out, lse, err, _ = run_case(c, general=general)
    assert err == binding.DEVERR_BAD_BLOCK
    # the same as a prefix without that page
    c2 = dict(c, ptab=np.full((2, 7), -1, np.int32), plens=[84, 40])
    c2["ptab"][0, :6] = np.delete(good[0], 3)[:6]
    c2["ptab"][1, :3] = good[1][:3]
    check_case(c2, out, lse)
    c["ptab"] = good
    # a plan made for other sizes
    plan = binding.shared_plan([0, 0], c["plens"], 8, 2, 64, binding.dtype_code(c["q"]), 4)
    pad = np.zeros(len(plan) + 64, np.int32)
    pad[:len(plan)] = plan
    e = torch.zeros(1, dtype=torch.int32, device=dev())
    a = binding.make_shared_args(c["q"], c["kc"], c["vc"], torch.from_numpy(c["tab"]).to(dev()),
                                 i32(c["lens"]), c["scale"], out,
                                 prefix_tables=torch.from_numpy(c["ptab"]).to(dev()),
                                 prefix_plan=torch.from_numpy(pad).to(dev()), err=e,
                                 num_parts=4 if general else None)
    binding.decode_attn_shared_args(a)
    torch.cuda.synchronize()
    assert int(e) & binding.DEVERR_BAD_PLAN


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_repeated_calls_are_bit_identical(dtype):
    c = make_case(40, 16, 4, 128, dtype, [i * 7 % 90 for i in range(40)], [1500, 333],
                  [i % 3 - 1 for i in range(40)], 51)
    out, lse, err, a = run_case(c)
    first = out.clone()
    for _ in range(5):
        binding.decode_attn_shared_args(a)
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    check_case(c, out, lse, err=err)


@pytest.mark.parametrize("general", [False, True])
def test_shared_attention_in_a_graph_and_on_another_stream(general):
    c = make_case(6, 8, 2, 64, "bf16", [3, 50, 16, 1, 0, 20], [300], [0, 0, 0, -1, 0, 0], 61, mass=True)
    first = c["mass"].clone()
    out, lse, err, a = run_case(c, general=general)
    want, want_mass = out.clone(), c["mass"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        binding.decode_attn_shared_args(a, side)
    for _ in range(2):
        c["mass"].copy_(first)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        torch.testing.assert_close(c["mass"], want_mass, rtol=0, atol=0, equal_nan=True)
    c["mass"].copy_(first)
    side.wait_stream(torch.cuda.current_stream())
    binding.decode_attn_shared_args(a, side)
    side.synchronize()
    assert torch.equal(out, want)


# --------------------------------------------------------------------------- eviction
def evict_case(B, Hkv, d, dtype, lens, keeps, seed, ties=False):
    nb, (tab,) = tables_for([lens], seed)
    g = torch.Generator().manual_seed(seed)
    mass = torch.randn((nb, Hkv, 16), generator=g).exp()
    if ties:
        mass = (mass * 2).round() - 1.0      # few values, negative ones and both zeros
        mass[torch.rand(mass.shape, generator=g) < 0.2] = -0.0
        mass[torch.rand(mass.shape, generator=g) < 0.05] = float("inf")
        mass[torch.rand(mass.shape, generator=g) < 0.05] = float("nan")
        mass[torch.rand(mass.shape, generator=g) < 0.05] = float("-inf")
    return dict(nb=nb, tab=tab, lens=lens, keeps=keeps, mass=mass.to(dev()),
                kc=normal((nb, Hkv, 16, d), dtype, seed + 1), vc=normal((nb, Hkv, 16, d), dtype, seed + 2))


def bits(t):
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32).cpu().numpy()


def check_evict(c, sink, recent, stride):
    t0 = [bits(c[k]) for k in ("kc", "vc", "mass")]
    mass0 = c["mass"].cpu().numpy()
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    kept = binding.evict(c["kc"], c["vc"], c["mass"], torch.from_numpy(c["tab"]).to(dev()),
                         i32(c["lens"]), i32(c["keeps"]), stride, sink, recent, err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    _, want = cache_ops.evict((t0[0], t0[1], mass0), c["tab"], c["lens"], c["keeps"], sink, recent)
    got = kept.cpu().numpy()
    new = [x.copy() for x in t0]
    for b, heads in enumerate(want):
        for g, src in enumerate(heads):
            assert got[b, g, :len(src)].tolist() == src.tolist(), (b, g)
            assert (got[b, g, len(src):] == -1).all()
            j = np.arange(len(src))
            blk = c["tab"][b]
            for n, o in zip(new, t0):
                n[blk[j // 16], g, j % 16] = o[blk[src // 16], g, src % 16]
    for k, n in zip(("kc", "vc", "mass"), new):
        np.testing.assert_array_equal(bits(c[k]), n)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("lens,keeps,sink,recent", [
    ([1], [1], 0, 0), ([2], [1], 0, 0), ([5, 0, 17], [3, 0, 0], 0, 0), ([33, 16, 40], [16, 16, 39], 4, 8),
    ([200, 64, 3], [64, 64, 64], 4, 16), ([100], [10], 8, 8), ([100], [10], 20, 4), ([100], [10], 4, 20),
    ([1000, 777], [500, 1], 1, 0), ([5000], [4097], 16, 1024)])
def test_evict(dtype, ties, lens, keeps, sink, recent):
    c = evict_case(len(lens), 2, 64, dtype, lens, keeps, len(lens) * 7 + sum(lens), ties)
    check_evict(c, sink, recent, max(keeps) + 3)


@pytest.mark.parametrize("Hkv,d,dtype", [(1, 128, "bf16"), (3, 8, "f32"), (2, 96, "bf16"), (1, 256, "f32"),
                                         (8, 128, "bf16")])
def test_evict_head_shapes(Hkv, d, dtype):
    c = evict_case(3, Hkv, d, dtype, [300, 31, 129], [100, 30, 64], Hkv + d)
    check_evict(c, 2, 10, 100)


@pytest.mark.parametrize("L,K", [(3000, 1500), (9000, 8999), (16400, 3), (50000, 20000)])
def test_evict_long_rows_shared_by_clusters(L, K):
    c = evict_case(1, 1, 64, "bf16", [L], [K], 3, ties=True)
    check_evict(c, 4, 100, K)


def test_evict_a_row_longer_than_the_keys_kept_on_chip():
    c = evict_case(1, 1, 8, "f32", [800001], [5000], 3, ties=True)
    check_evict(c, 4, 100, 5000)


def test_evict_many_rows_walk():
    """Enough (row, head) pairs that each is walked by one CTA."""
    lens = [(37 * i) % 300 for i in range(40)]
    c = evict_case(40, 2, 64, "bf16", lens, [(11 * i) % 200 for i in range(40)], 17, ties=True)
    check_evict(c, 3, 9, 200)


def widened(c, pages):
    """The case behind tables of `pages` entries (the kernels are chosen by their width)."""
    tab = np.full((c["tab"].shape[0], pages), -1, np.int32)
    tab[:, :c["tab"].shape[1]] = c["tab"]
    return dict(c, tab=tab)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pages", [16, 17, 32, 33, 70])
@pytest.mark.parametrize("B", [1, 5, 77])
def test_evict_short_rows_by_every_kernel(dtype, pages, B):
    lens = [(53 * i + 200) % 257 for i in range(B)]
    keeps = [(29 * i + 100) % 200 for i in range(B)]
    c = widened(evict_case(B, 1 + B % 2, 64, dtype, lens, keeps, 7 * B + pages, ties=B != 5), pages)
    check_evict(c, 3, 9, 200)


@pytest.mark.parametrize("L,K,sink,recent", [(256, 255, 0, 0), (256, 1, 0, 0), (256, 128, 128, 0),
                                             (255, 128, 0, 128), (241, 240, 1, 1), (512, 256, 4, 16),
                                             (512, 511, 0, 0), (497, 3, 1, 1)])
def test_evict_at_the_ends_of_a_short_row(L, K, sink, recent):
    check_evict(evict_case(2, 3, 128, "bf16", [L, L - 1], [K, K], L + K, ties=True), sink, recent, K)
    check_evict(evict_case(2, 3, 128, "bf16", [L, 5], [K, K], L + K), sink, recent, K + 1)


@pytest.mark.parametrize("pages,copies", [(3, 1), (40, 1), (40, 20)])   # one CTA, chunks, walks
def test_evict_leaves_bad_rows_alone(pages, copies):
    c = evict_case(5 * copies, 2, 64, "bf16", [40] * 5 * copies, [8, 8, 8, -1, 30] * copies, 9)
    assert c["tab"].shape[1] == 3
    before = [bits(c[k]).copy() for k in ("kc", "vc", "mass")]
    tab = widened(c, pages)["tab"]
    tab[0::5, 1] = c["nb"]                    # a block outside the pool
    tab[1::5, 2] = -1
    lens = np.array([40, 40, 16 * pages + 1, 40, 40] * copies)     # row 2: longer than its table
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    # row 3 keeps a negative number, row 4 more than kept holds
    kept = binding.evict(c["kc"], c["vc"], c["mass"], torch.from_numpy(tab).to(dev()), i32(lens),
                         i32(c["keeps"]), 16, err=err)
    assert int(err) == binding.DEVERR_BAD_BLOCK | binding.DEVERR_BAD_LEN
    assert (kept == -1).all()
    for k, x in zip(("kc", "vc", "mass"), before):
        np.testing.assert_array_equal(bits(c[k]), x)


def test_evict_in_a_graph():
    c = evict_case(4, 2, 64, "bf16", [90, 33, 64, 200], [32, 33, 20, 100], 13)
    saved = [c[k].clone() for k in ("kc", "vc", "mass")]
    kept = torch.empty((4, 2, 100), dtype=torch.int32, device=dev())
    a = binding.make_evict_args(c["kc"], c["vc"], c["mass"], torch.from_numpy(c["tab"]).to(dev()),
                                i32(c["lens"]), i32(c["keeps"]), kept, 2, 8)
    binding.evict_args(a)
    torch.cuda.synchronize()
    want = [c[k].clone() for k in ("kc", "vc", "mass")] + [kept.clone()]
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        binding.evict_args(a, side)
    for k, x in zip(("kc", "vc", "mass"), saved):
        c[k].copy_(x)
    kept.fill_(9)
    g.replay()
    torch.cuda.synchronize()
    for x, y in zip([c[k] for k in ("kc", "vc", "mass")] + [kept], want):
        assert torch.equal(x, y)


def test_evict_behind_tables_for_millions_of_tokens():
    """The launch follows the tables' width, not the rows' lengths."""
    c = evict_case(1, 2, 64, "bf16", [70], [33], 23)
    wide = np.full((1, 1 << 17), -1, np.int32)
    wide[:, :c["tab"].shape[1]] = c["tab"]
    check_evict(dict(c, tab=wide), 2, 5, 40)


# --------------------------------------------------------------------------- where it can go wrong
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("plens", [[], [64]])
@pytest.mark.parametrize("parts", [None, 7])
def test_excluded_tokens_may_hold_anything(dtype, plens, parts):
    lens = [40, 33, 1, 16, 100]
    c = make_case(5, 8, 2, 64, dtype, lens, plens, [0, -1, 0, 0, 0], 71, bias=True, mass=True)
    rng = np.random.default_rng(5)
    mass0 = f64(c["mass"])
    for b, n in enumerate(lens):
        x = excluded(c["bias"])[b, :n]
        for t in np.flatnonzero(np.isneginf(x)):
            for cache in (c["kc"], c["vc"]):
                cache[int(c["tab"][b, t // 16]), :, t % 16] = \
                    float(rng.choice([np.nan, np.inf, -np.inf]))
    out, lse, err, _ = run_case(c, num_parts=parts)
    # (the oracle multiplies what is excluded by zero: it gets zeros there)
    for cache in ("kc", "vc"):
        c[cache] = torch.nan_to_num(c[cache], 0.0, 0.0, 0.0)
    check_case(c, out, lse, mass0, err=err)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows_of", [1, 24])
@pytest.mark.parametrize("parts", [None, 7])
def test_nan_spreads_as_in_the_formula(dtype, rows_of, parts):
    """NaN or infinity in what counts: the rows (heads, columns) that the formula makes NaN
    are NaN, and no others change."""
    B, Hq, Hkv, d, G = 6 * rows_of, 8, 2, 64, 4
    lens, rows = [40, 0, 100, 33, 5, 20] * rows_of, [0, 0, 1, -1, 1, 0] * rows_of
    c = make_case(B, Hq, Hkv, d, dtype, lens, [300, 50], rows, 81, mass=True)
    before = {k: c[k].clone() for k in ("q", "kc", "vc", "mass")}
    want, want_lse, err, _ = run_case(c, num_parts=parts)
    want_mass = c["mass"].clone()
    nan = torch.zeros((B, Hq, d), dtype=torch.bool)
    c["mass"].copy_(before["mass"])
    c["q"][0, 1] = float("nan")                                    # a query head, prefix and own
    nan[0, 1] = True
    c["q"][1, 6, 3] = float("inf")                                 # a row with a prefix alone
    nan[1, 6] = True
    c["kc"][int(c["tab"][3, 1]), 0, 2, 5] = float("nan")           # own key, KV head 0
    nan[3, :G] = True
    c["kc"][int(c["ptab"][1, 2]), 1, 7, 0] = float("nan")          # key of prefix 1, KV head 1
    nan[torch.tensor(rows) == 1, G:] = True
    c["vc"][int(c["ptab"][0, 0]), 0, 0, 9] = float("inf")          # value of prefix 0: no NaN
    c["vc"][int(c["tab"][5, 0]), 1, 3, 8] = float("nan")           # own value: one column
    nan[5, G:, 8] = True
    inf = torch.zeros_like(nan)
    inf[torch.tensor(rows) == 0, :G, 9] = True
    out, lse, err, _ = run_case(c, num_parts=parts)
    assert err == 0
    o, w = out.float().cpu(), want.float().cpu()
    inf &= ~nan
    assert torch.equal(o.isnan(), nan)
    assert (o[inf] == float("inf")).all()
    assert torch.equal(o[~nan & ~inf], w[~nan & ~inf])
    whole = nan.all(-1)
    assert torch.equal(lse.isnan().cpu(), whole)
    assert torch.equal(lse.cpu()[~whole], want_lse.cpu()[~whole])
    # weights: those of a KV head with a NaN query head or key are NaN, the others are as before
    heads = whole.view(B, Hkv, G).any(-1)
    for b in range(B):
        for t in range(0, lens[b]):
            at = (int(c["tab"][b, t // 16]), slice(None), t % 16)
            got, old = c["mass"][at].cpu(), want_mass[at].cpu()
            assert torch.equal(got.isnan(), heads[b]) and torch.equal(got[~heads[b]], old[~heads[b]])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prefix_waits_that_give_up_report_a_timeout(dtype):
    """Waits of 64 clocks end long before a copy lands: the call flags it, ends, and after the
    workspace is zero-filled again the next call is exact."""
    c = make_case(9, 8, 2, 128, dtype, [40, 3, 0, 17, 90, 1, 64, 200, 33], [1000, 130],
                  [i % 3 - 1 for i in range(9)], 91)
    want, want_lse, err, a = run_case(c)
    assert err == 0
    space = torch.zeros(a.workspace_bytes, dtype=torch.uint8, device=dev())
    out, lse, err, b = run_case(c, workspace=space, flags=binding.ATTN_SHORT_WAITS)
    assert err & binding.DEVERR_TIMEOUT and not err & ~binding.DEVERR_TIMEOUT
    space.zero_()
    out, lse, err, _ = run_case(c, workspace=space)
    assert err == 0 and torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("general", [False, True])
def test_a_captured_call_follows_the_plan_in_its_buffer(general):
    """One graph, a plan buffer and a workspace for the largest plan of its sizes: new
    prefixes of the rows and new lengths go in by overwriting the buffers."""
    B, Hq, Hkv, d, P = 12, 8, 2, 64, 3
    c = make_case(B, Hq, Hkv, d, "bf16", [50 - 4 * i for i in range(B)], [700, 90, 300], [0] * B, 95)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    cap, most = binding.shared_plan_cap(B, P, Hq, Hkv, sms)
    buf, lens = torch.zeros(cap, dtype=torch.int32, device=dev()), i32(c["lens"])
    ptab = torch.from_numpy(c["ptab"]).to(dev())
    out, lse = torch.empty_like(c["q"]), torch.empty((B, Hq), device=dev())
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    a = binding.make_shared_args(c["q"], c["kc"], c["vc"], torch.from_numpy(c["tab"]).to(dev()), lens,
                                 c["scale"], out, prefix_tables=ptab, prefix_plan=buf, slots=most,
                                 num_ctas=sms, lse=lse, err=err, num_parts=24 if general else None)

    def put(rows, plens, own):
        plan = binding.shared_plan(rows, plens, Hq, Hkv, d, binding.BF16, sms)
        buf.zero_()
        buf[:len(plan)].copy_(torch.from_numpy(plan))
        lens.copy_(i32(own))
        c.update(rows=rows, plens=plens, lens=np.asarray(own))

    put([0] * B, [700, 90, 300], c["lens"])
    binding.decode_attn_shared_args(a)
    torch.cuda.synchronize()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        binding.decode_attn_shared_args(a, side)
    for rows, plens, own in (([0] * B, [700, 90, 300], c["lens"].tolist()),
                             ([i % 3 for i in range(B)], [700, 90, 300], [0] * B),
                             ([i % 4 - 1 for i in range(B)], [160, 90, 0], [1] * B),
                             ([-1] * B, [700, 90, 300], [3] * B)):
        put(rows, plens, own)
        out.fill_(9.0)
        g.replay()
        torch.cuda.synchronize()
        check_case(c, out, lse, err=int(err))


def test_caches_beyond_32_bit_offsets():
    """Blocks whose elements and bytes lie behind 2^32: append, attention, weights, eviction."""
    Hq, Hkv, d, dtype = 16, 8, 128, "bf16"
    nb = (1 << 32) // (Hkv * 16 * d) + 64                  # 2^32 elements: 8.6 GB a cache
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    rng = np.random.default_rng(7)
    high = list(nb - 1 - rng.permutation(60))
    kc = torch.empty((nb, Hkv, 16, d), dtype=TD[dtype], device=dev())
    vc = torch.empty_like(kc)
    mass = torch.empty((nb, Hkv, 16), device=dev())
    n, plen = 200, 300
    ptab = np.array([[high.pop() for _ in range(19)]], np.int32)
    tab = np.array([[high.pop() for _ in range(13)]], np.int32)
    rot = binding.Rotary(d)
    kv = [normal((n + plen, Hkv, d), dtype, 1), normal((n + plen, Hkv, d), dtype, 2)]
    pos = np.arange(n + plen)
    slots = np.concatenate([ptab[0][np.arange(plen) // 16].astype(np.int64) * 16 + np.arange(plen) % 16,
                            tab[0][np.arange(n) // 16].astype(np.int64) * 16 + np.arange(n) % 16])
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    _, k_rot = binding.rotary_append(rot, None, kv[0], kv[1], i32(pos), torch.from_numpy(slots).to(dev()),
                                     kc, vc, err=err)
    q = normal((1, Hq, d), dtype, 3)
    # the same in small caches
    small = dict(B=1, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, lens=np.array([n]), plens=[plen], rows=[0],
                 nb=32, ptab=np.arange(19, dtype=np.int32)[None],
                 tab=np.arange(19, 32, dtype=np.int32)[None], q=q, scale=d**-0.5, bias=None)
    used = torch.from_numpy(np.concatenate([ptab[0], tab[0]]).astype(np.int64)).to(dev())
    small["kc"], small["vc"] = kc[used], vc[used]
    for x, src in ((small["kc"], k_rot), (small["vc"], kv[1])):
        flat = x.transpose(1, 2).reshape(32 * 16, Hkv, d)
        assert torch.equal(flat[:plen], src[:plen]) and torch.equal(flat[304:304 + n], src[plen:])
    out, lse = torch.empty_like(q), torch.empty((1, Hq), device=dev())
    plan = torch.from_numpy(binding.shared_plan([0], [plen], Hq, Hkv, d, binding.BF16)).to(dev())
    scores = binding.alloc_scores(nb, Hq)
    a = binding.make_shared_args(q, kc, vc, torch.from_numpy(tab).to(dev()), i32([n]), d**-0.5, out,
                                 prefix_tables=torch.from_numpy(ptab).to(dev()), prefix_plan=plan,
                                 mass=mass, scores=scores, mass_lens=i32([0]), lse=lse, err=err)
    binding.decode_attn_shared_args(a)
    torch.cuda.synchronize()
    small["mass"], small["known"] = mass[used], [0]
    unused = np.zeros((32, Hkv, 16))
    m = f64(small["mass"])
    own = np.zeros((32, 16), bool)
    t = np.arange(n)
    own[19 + t // 16, t % 16] = True
    m[~own[:, None, :].repeat(Hkv, 1)] = 0
    small["mass"] = torch.from_numpy(m)
    check_case(small, out, lse, unused, err=int(err))
    big = [bits(x[used]) for x in (kc, vc, mass)]
    kept = binding.evict(kc, vc, mass, torch.from_numpy(tab).to(dev()), i32([n]), i32([90]), 90, 3, 10,
                         err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    src = kept.cpu().numpy()[0]
    new = [x.copy() for x in big]
    j = np.arange(90)
    for g in range(Hkv):
        for x, o in zip(new, big):
            x[19 + j // 16, g, j % 16] = o[19 + src[g] // 16, g, src[g] % 16]
    for x, y in zip(new, (kc, vc, mass)):
        np.testing.assert_array_equal(x, bits(y[used]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("B,pages", [(1, 1), (1, 40), (3, 22), (8, 40), (19, 20), (38, 10), (70, 4)])
def test_short_contexts_in_one_launch(dtype, d, G, B, pages):
    """One CTA or a cluster of up to eight to a (row, KV head), shares that hold no page
    among them, against the oracle."""
    Hkv = 4
    lens = [(37 * b + 16 * pages - 3) % (16 * pages + 1) for b in range(B)]
    lens[-1] = 16 * pages
    plens = [] if pages == 1 else [min(16 * 24, 5 * pages), 1]
    rows = [b % 3 - 1 if plens else -1 for b in range(B)]
    c = make_case(B, Hkv * G, Hkv, d, dtype, lens, plens, rows, 3 * B + G, bias=B == 3, mass=True)
    m0 = f64(c["mass"])
    out, lse, err, a = run_case(c)
    assert a.num_parts == 0 and binding.shared_short(B, Hkv * G, Hkv, d, a.dtype, a.bt_stride,
                                                     a.pt_stride)
    check_case(c, out, lse, m0, err=err)


@pytest.mark.parametrize("general", [False, True])
def test_lengths_that_do_not_fit_are_flagged(general):
    """A row longer than its table, or of negative length, has no own tokens."""
    c = make_case(3, 8, 2, 64, "bf16", [20, 20, 20], [40], [0, -1, 0], 17, mass=True)
    c["known"] = [0, 0, 0]
    before = c["mass"].clone()
    lens = c["lens"].copy()
    c["lens"] = np.array([33, -1, 20])
    out, lse, err, _ = run_case(c, general=general)
    assert err == binding.DEVERR_BAD_LEN
    c["lens"] = np.array([0, 0, 20])
    m0 = f64(before)
    check_case(c, out, lse, m0)
