"""Host side of the cache operators: rotary tables, the shared-prefix planner, position
offsets and eviction in the allocator, and what the calls refuse."""
import ctypes

import numpy as np
import pytest

from oracle.cache_ops import rotary_frequencies


@pytest.fixture(scope="module")
def bind(host_lib):
    from paged_kv_decode_10_gb300 import binding
    return binding


# --------------------------------------------------------------------------- rotary tables
@pytest.mark.parametrize("scaling,kw", [
    ("plain", {}), ("linear", dict(factor=8.0)), ("ntk", dict(factor=4.0)),
    ("ramp", dict(factor=16.0, original_len=4096)),
    ("ramp", dict(factor=2.0, original_len=4096, low=1.0, high=1.0001)),
    ("ramp", dict(factor=3.0, original_len=5, low=1.0, high=32.0)),
    ("bands", dict(factor=8.0, original_len=8192, low=1.0, high=4.0, base=500000.0))])
@pytest.mark.parametrize("rot", [128, 64, 6])
def test_rotary_table_holds_the_frequencies(bind, scaling, kw, rot):
    r = bind.Rotary(128, rot_dim=rot, scaling=scaling, **kw)
    got = np.array(r.table.turns[:rot // 2], np.float64) / 2.0**64 * 2 * np.pi
    want = rotary_frequencies(rot, scaling, **kw)
    # pow, a few multiplications and the truncation to 64 bits, all in double precision
    np.testing.assert_allclose(got, want, rtol=64 * 2.0**-52, atol=2.0**-60)
    assert list(r.table.turns[rot // 2:]) == [0] * (128 - rot // 2)


@pytest.mark.parametrize("kw", [
    dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=130), dict(layout="other"),
    dict(scaling="other"), dict(base=0.5), dict(base=float("nan")), dict(base=float("inf")),
    dict(amplitude=0.0), dict(amplitude=float("nan")), dict(scaling="linear", factor=0.5),
    dict(scaling="linear", factor=float("nan")), dict(scaling="ntk", rot_dim=2, factor=2.0),
    dict(scaling="ramp", factor=2.0), dict(scaling="bands", factor=2.0, original_len=64, low=0.0),
    dict(scaling="bands", factor=2.0, original_len=64, low=4.0, high=4.0),
    dict(scaling="ramp", factor=2.0, original_len=64, base=1.0)])
def test_rotary_refuses(bind, kw):
    with pytest.raises(bind.PkvError):
        bind.Rotary(128, **kw)


@pytest.mark.parametrize("d", [0, 1, 3, 258])
def test_rotary_refuses_head_sizes(bind, d):
    with pytest.raises(bind.PkvError):
        bind.Rotary(d, rot_dim=2)


# --------------------------------------------------------------------------- planner
def read_plan(plan):
    magic, n, B, slots, C, Hkv, G, R = plan[:8]
    rows = plan[16:16 + 4 * B].reshape(B, 4)
    order = plan[16 + 4 * B:16 + 6 * B].reshape(B, 2)
    ctas = plan[16 + 6 * B:16 + 6 * B + C + 1]
    at = (16 + 6 * B + C + 1 + 3) // 4 * 4
    items = plan[at:].reshape(-1, 8)
    assert len(items) == n and ctas[0] == 0 and ctas[-1] == n and (np.diff(ctas) >= 0).all()
    return rows, order, ctas, items, slots, R


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,Hq,Hkv,lens,seed", [
    (1, 8, 8, [1], 0), (1, 8, 1, [5000], 1), (3, 4, 2, [0, 17], 2), (64, 32, 8, [8192], 3),
    (257, 32, 8, [777, 4097, 1, 130], 4), (40, 16, 2, [128, 129, 127, 0, 65536], 5),
    (1000, 8, 8, [31] * 300, 6), (5, 32, 4, [], 7)])
@pytest.mark.parametrize("ctas", [1, 7, 152])
def test_shared_plan_covers_every_token_once(bind, dtype, B, Hq, Hkv, lens, seed, ctas):
    rng = np.random.default_rng(seed)
    prefix = rng.integers(-1, max(len(lens), 1), B) if lens else np.full(B, -1)
    code = bind.BF16 if dtype == "bf16" else bind.F32
    cap, most = bind.shared_plan_cap(B, len(lens), Hq, Hkv, ctas)
    plan = bind.shared_plan(prefix, lens, Hq, Hkv, 128, code, ctas)
    assert len(plan) <= cap
    rows, order, per_cta, items, slots, R = read_plan(plan)
    assert slots <= most and R == (256 if dtype == "bf16" else 64) // (Hq // Hkv)
    taken = set()
    seen = {}
    for p, g, r0, n, t0, t1, split, _ in items:
        assert 0 < n <= R and 0 <= t0 < t1 <= lens[p] and 0 <= g < Hkv
        for b, first in order[r0:r0 + n]:
            assert prefix[b] == p and 0 <= split < rows[b, 1] and first == rows[b, 0]
            slot = (rows[b, 0] + split, g)
            assert slot not in taken and slot[0] < slots
            taken.add(slot)
            seen.setdefault((b, g), []).append((t0, t1))
    for b in range(B):
        has = prefix[b] >= 0 and lens[prefix[b]] > 0
        assert (rows[b, 1] > 0) == has
        assert rows[b, 2:].tolist() == ([prefix[b], lens[prefix[b]]] if has else [-1, 0])
        for g in range(Hkv):
            parts = sorted(seen.get((b, g), []))
            assert len(parts) == rows[b, 1]
            if has:
                assert parts[0][0] == 0 and parts[-1][1] == lens[prefix[b]]
                assert all(x[1] == y[0] for x, y in zip(parts, parts[1:]))
    # the slots of different rows do not meet
    used = [s for b in range(B) for s in range(rows[b, 0], rows[b, 0] + rows[b, 1])]
    assert len(set(used)) == len(used) == slots


def test_shared_plan_fills_the_gpu(bind):
    plan = bind.shared_plan([0] * 64, [8192], 32, 8, 128, bind.BF16, 152)
    _, _, ctas, items, slots, _ = read_plan(plan)
    assert (np.diff(ctas) > 0).sum() >= 100


def test_shared_plan_refuses(bind):
    ok = dict(row_prefix=[0, 0], prefix_lens=[100], Hq=8, Hkv=2, d=64, dtype=bind.BF16, num_ctas=4)
    bind.shared_plan(**ok)
    for bad in (dict(row_prefix=[0, 1]), dict(prefix_lens=[-1]), dict(Hq=6), dict(Hq=12),
                dict(Hq=32), dict(d=96), dict(dtype=7), dict(num_ctas=5000), dict(Hkv=0),
                dict(out=np.empty(16, np.int32)), dict(out=np.empty(30, np.int32)),
                dict(out=np.empty(512, np.int64))):
        with pytest.raises(bind.PkvError):
            bind.shared_plan(**{**ok, **bad})


def test_short_contexts_are_few_rows_of_few_pages(bind):
    def short(B, Hkv, own, pre=0, G=4, d=128, dtype=bind.BF16):
        return bind.shared_short(B, Hkv * G, Hkv, d, dtype, own, pre)
    assert short(1, 1, 1) and short(14, 1, 128) and short(2, 17, 64) and short(76, 1, 32)
    assert short(19, 8, 16) and not short(19, 8, 17) and not short(153, 1, 1)
    assert not short(1, 1, 129) and not short(15, 1, 65) and not short(35, 1, 33)
    # several waves where the other form has more kernels or a costly partition
    assert short(38, 8, 4, 4) and not short(38, 8, 8, 8) and not short(77, 8, 4, 4)
    assert short(76, 8, 8, 8, d=64) and short(152, 8, 4, 4, d=64) and not short(152, 8, 8, 8, d=64)
    assert short(76, 8, 16, dtype=bind.F32) and not short(152, 8, 16, dtype=bind.F32)
    assert not short(65536, 8, 1) and not short(1, 1, (1 << 26) - 1, 1 << 25)
    for bad in ((1, 0, 4), (1, 1, -1), (1, 1, 1, -1), (1, 1, 1, 0, 3), (1, 1, 1, 0, 4, 96)):
        with pytest.raises(bind.PkvError):
            short(*bad)


def test_shared_workspace_grows_with_slots(bind):
    a = bind.shared_workspace_bytes(4, 8, 2, 64, 8, 0)
    b = bind.shared_workspace_bytes(4, 8, 2, 64, 8, 10)
    assert a >= bind.workspace_bytes(4, 8, 2, 64, 8) + 4 * 8 * 4
    assert b - a >= 10 * 8 * 65 * 4
    with pytest.raises(bind.PkvError):
        bind.shared_workspace_bytes(4, 8, 2, 64, 8, -1)


# --------------------------------------------------------------------------- allocator
def test_offsets_move_positions_only(bind):
    a = bind.BlockAllocator(16, 4, 8)
    s, t = a.join(17), a.join(3)
    a.set_offset(s, 1000)
    pos, slots, lens, tables = a.prepare_step([s, t], 8)
    assert pos.tolist() == [1017, 3] and lens.tolist() == [18, 4]
    assert slots[0] == tables[0, 1] * 16 + 1 and a.offset(s) == 1000 and a.offset(t) == 0
    assert a.seq_slots(s, 0, 2)[0].tolist() == [0, 1]      # indices within the sequence
    a.leave(s)
    assert a.join(0) == s and a.offset(s) == 0            # a reused id starts afresh
    with pytest.raises(bind.PkvError):
        a.set_offset(s, -1)
    with pytest.raises(bind.UnknownSequence):
        a.set_offset(3, 1)
    with pytest.raises(bind.UnknownSequence):
        a.offset(3)


def test_position_beyond_32_bits_is_refused(bind):
    a = bind.BlockAllocator(4, 2, 2)
    s = a.join(1)
    a.set_offset(s, 2**31 - 2)
    assert a.prepare_step([s], 2)[0].tolist() == [2**31 - 1]
    free, n = a.num_free(), a.seq_len(s)
    with pytest.raises(bind.PkvError):
        a.prepare_step([s], 2)
    assert a.num_free() == free and a.seq_len(s) == n


def test_evict_many_returns_blocks_and_keeps_positions(bind):
    a = bind.BlockAllocator(32, 4, 16)
    s, t = a.join(100), a.join(40)
    blocks = a.seq_blocks(s)
    free = a.free_stack()
    a.evict_many([s, t], [33, 40])
    assert a.seq_len(s) == 33 and a.seq_blocks(s) == blocks[:3] and a.offset(s) == 67
    assert a.free_stack() == free + blocks[3:]
    assert a.seq_len(t) == 40 and a.offset(t) == 0
    pos, slots, lens, _ = a.prepare_step([s], 16)
    assert pos[0] == 100 and lens[0] == 34 and slots[0] == blocks[2] * 16 + 1
    a.evict_many([s], [0])
    assert a.seq_len(s) == 0 and a.seq_blocks(s) == [] and a.offset(s) == 101


def test_evict_many_is_all_or_nothing(bind):
    a = bind.BlockAllocator(32, 4, 16)
    s, t = a.join(100), a.join(40)
    state = (a.seq_blocks(s), a.seq_blocks(t), a.free_stack())
    for ids, keep, err in (([s, 3], [1, 1], bind.UnknownSequence), ([s, s], [1, 1], bind.PkvError),
                           ([s, t], [1, -1], bind.PkvError), ([s], [1, 2], bind.PkvError)):
        with pytest.raises(err):
            a.evict_many(ids, keep)
        assert (a.seq_blocks(s), a.seq_blocks(t), a.free_stack()) == state
        assert a.offset(s) == a.offset(t) == 0


def test_cached_tables_after_an_eviction(bind):
    """The table buffer of pkv_prepare_step_cached equals a fresh pkv_prepare_step's
    when a sequence shrank and grew again between two steps."""
    def run(cached):
        a = bind.BlockAllocator(64, 4, 16)
        s, t = a.join(100), a.join(31)
        out = (np.empty(2, np.int32), np.empty(2, np.int64), np.empty(2, np.int32),
               np.full((2, 16), 7, np.int32))
        state = np.full(6, -1, np.int32)
        got = []
        for step in range(20):
            if step in (3, 9):
                a.evict_many([s], [17])
            if step == 9:
                a.join(20)     # takes blocks that s returned
            if cached:
                a.prepare_step_cached([s, t], 16, out, state)
            else:
                a.prepare_step([s, t], 16, out)
            got.append([x.copy() for x in out])
        return got
    for x, y in zip(run(True), run(False)):
        for u, v in zip(x, y):
            np.testing.assert_array_equal(u, v)


# --------------------------------------------------------------------------- refusals (nothing is launched)
def fake(n=1 << 20):
    return ctypes.c_void_p(n)


def evict_ok(b):
    a = b.EvictArgs()
    for f in ("k_cache", "v_cache", "mass", "block_tables", "seq_lens", "keep_lens", "kept",
              "workspace"):
        setattr(a, f, fake())
    a.v_cache = fake(1 << 22)
    a.workspace_bytes = 1 << 30
    a.num_blocks, a.bt_stride, a.kept_stride, a.sink, a.recent = 8, 4, 16, 0, 0
    a.B, a.Hkv, a.d, a.dtype = 2, 2, 64, b.BF16
    return a


@pytest.mark.parametrize("field,value", [
    ("k_cache", None), ("v_cache", None), ("mass", None), ("block_tables", None),
    ("seq_lens", None), ("keep_lens", None), ("kept", None), ("k_cache", fake((1 << 20) + 8)),
    ("num_blocks", 0), ("bt_stride", 0), ("kept_stride", 0), ("sink", -1), ("recent", -1),
    ("B", -1), ("B", 70000), ("Hkv", 0), ("d", 0), ("d", 4), ("d", 1024), ("dtype", 5),
    ("mass", fake((1 << 20) + 4)), ("workspace", None), ("workspace", fake((1 << 20) + 16)),
    ("workspace_bytes", 256), ("v_cache", fake()), ("v_cache", fake((1 << 20) + 4096)),
    ("k_cache", fake((1 << 22) + 8 * 2 * 16 * 64 * 2 - 16))])
def test_evict_refuses(bind, field, value):
    a = evict_ok(bind)
    setattr(a, field, value)
    assert bind.load().pkv_evict(ctypes.byref(a), None) in (bind.ERR_INVALID_ARG,
                                                            bind.ERR_UNSUPPORTED)
    assert bind.load().pkv_last_error()


def test_empty_batches_need_nothing(bind):
    lib = bind.load()
    a = evict_ok(bind)
    a.B = 0
    a.k_cache = None
    assert lib.pkv_evict(ctypes.byref(a), None) == bind.OK
    s = shared_ok(bind)
    s.B = 0
    s.q_rot = None
    assert lib.pkv_decode_attn_shared(ctypes.byref(s), None) == bind.OK
    r = rotary_ok(bind)
    r.T = 0
    r.q = None
    assert lib.pkv_rotary_append(ctypes.byref(r), None) == bind.OK
    for f in (lib.pkv_evict, lib.pkv_decode_attn_shared, lib.pkv_rotary_append):
        assert f(None, None) == bind.ERR_INVALID_ARG


def shared_ok(b):
    a = b.SharedArgs()
    for f in ("q_rot", "k_cache", "v_cache", "block_tables", "seq_lens", "prefix_tables",
              "prefix_plan", "mass", "scores", "workspace"):
        setattr(a, f, fake())
    a.out = fake(1 << 21)
    a.workspace_bytes = 1 << 40
    a.num_blocks, a.bt_stride, a.n_prefixes, a.pt_stride = 8, 4, 1, 4
    a.plan_ints, a.slots, a.num_ctas = 4096, 4, 4
    a.B, a.Hq, a.Hkv, a.d, a.dtype, a.num_parts = 2, 8, 2, 64, b.BF16, 8
    a.scale, a.mass_decay = 0.125, 1.0
    return a


@pytest.mark.parametrize("field,value", [
    ("q_rot", None), ("k_cache", None), ("v_cache", None), ("block_tables", None),
    ("seq_lens", None), ("out", None), ("workspace", None), ("out", fake()),
    ("q_rot", fake((1 << 20) + 8)), ("out", fake((1 << 21) + 4)),
    ("workspace", fake((1 << 20) + 16)), ("workspace_bytes", 4096), ("prefix_plan", None),
    ("prefix_plan", fake((1 << 20) + 4)), ("plan_ints", 16), ("slots", -1), ("num_ctas", 5000),
    ("pt_stride", 0), ("bt_stride", 0), ("num_blocks", 0), ("num_blocks", 1 << 27),
    ("scores", None), ("scores", fake((1 << 20) + 4)), ("flags", 1), ("flags", 2), ("flags", 4),
    ("attn_bias", fake()), ("Hq", 7), ("Hq", 6), ("Hkv", 0), ("d", 96), ("dtype", 3), ("B", 70000),
    ("num_parts", 5000), ("out", fake((1 << 20) + 2 * 8 * 64 * 2 - 16)), ("scale", float("nan")),
    ("scale", float("inf")), ("mass_decay", float("nan"))])
def test_shared_attention_refuses(bind, field, value):
    a = shared_ok(bind)
    setattr(a, field, value)
    assert bind.load().pkv_decode_attn_shared(ctypes.byref(a), None) in (bind.ERR_INVALID_ARG,
                                                                         bind.ERR_UNSUPPORTED)
    assert bind.load().pkv_last_error()


KEEP = []


def rotary_ok(b):
    r = b.Rotary(64)
    KEEP.append(r)
    a = b.RotaryArgs()
    a.rotary = ctypes.pointer(r.table)
    for i, f in enumerate(("q", "k", "v", "positions", "slot_mapping", "k_cache", "v_cache")):
        setattr(a, f, fake(1 + i << 20))
    a.q_out, a.k_out = a.q, a.k
    a.q_stride = a.q_out_stride = 8 * 64
    a.k_stride = a.v_stride = a.k_out_stride = 2 * 64
    a.num_blocks, a.T, a.Hq, a.Hkv, a.d, a.dtype = 8, 4, 8, 2, 64, b.BF16
    return a


@pytest.mark.parametrize("field,value", [
    ("rotary", None), ("q", None), ("k", None), ("v", None), ("q_out", None), ("positions", None),
    ("k_cache", None), ("v_cache", None), ("k_cache", fake((1 << 20) + 8)), ("d", 128),
    ("dtype", 9), ("T", -1), ("Hq", -1), ("Hkv", -1), ("q_stride", 64), ("k_stride", 64),
    ("v_stride", 64), ("k_out_stride", 64), ("q_stride", 1024), ("q", fake((1 << 20) + 1)),
    ("num_blocks", -1), ("Hq", 1 << 20),
    # outputs over other tensors, or over their own inputs but not in place
    ("q_out", fake(2 << 20)), ("q_out", fake(3 << 20)), ("k_out", fake(1 << 20)),
    ("k_out", fake(3 << 20)), ("q_out", fake((1 << 20) + 1024)), ("q_out", fake((1 << 20) - 1024)),
    ("k_out", fake((2 << 20) + 16)), ("k", fake((1 << 20) + 4096 - 16)), ("v_cache", fake(6 << 20)),
    ("k_cache", fake((7 << 20) + 16))])
def test_rotary_append_refuses(bind, field, value):
    a = rotary_ok(bind)
    setattr(a, field, value)
    assert bind.load().pkv_rotary_append(ctypes.byref(a), None) in (bind.ERR_INVALID_ARG,
                                                                    bind.ERR_UNSUPPORTED)
    assert bind.load().pkv_last_error()


def test_rotary_append_tells_interleaved_rows_from_overlapping_ones(bind):
    """q, k and v as slices of one projection's output, q rotated where it lies: refused
    only from the step on at which a slice reaches the next (by the argument that is
    checked after the overlaps: there is nothing to launch on)."""
    def why(k_at, T=4, hq=8, row=768):
        a = rotary_ok(bind)
        a.T, a.Hq = T, hq
        a.q = a.q_out = fake(1 << 20)
        a.k, a.v = fake((1 << 20) + 2 * k_at), fake((1 << 20) + 2 * (k_at + 128))
        a.k_out = fake(9 << 20)
        a.q_stride = a.q_out_stride = a.k_stride = a.v_stride = row
        a.d, a.num_blocks = 64, -1
        assert bind.load().pkv_rotary_append(ctypes.byref(a), None) == bind.ERR_INVALID_ARG
        return bind.load().pkv_last_error().decode()
    assert "append" in why(512) and "append" in why(512 + 768) and "append" in why(512, T=1)
    assert "overlap" in why(504) and "overlap" in why(520) and "overlap" in why(504, T=1)
    assert "overlap" in why(512 + 768 - 8)


def test_rotary_append_needs_an_initialised_table(bind):
    a = rotary_ok(bind)
    a.rotary = ctypes.pointer(bind.RotaryTable())
    assert bind.load().pkv_rotary_append(ctypes.byref(a), None) == bind.ERR_INVALID_ARG


def test_binding_checks_tensors(bind):
    import torch
    x = torch.zeros(2, 4, 64)
    rot = bind.Rotary(64)
    with pytest.raises(bind.PkvError):
        bind.make_rotary_args(rot, x, x, x, torch.zeros(2, dtype=torch.int32), x, x)   # host tensors
    cache = torch.zeros(4, 2, 16, 64)
    with pytest.raises(bind.PkvError):
        bind.make_evict_args(cache, cache, torch.zeros(4, 2, 16), torch.zeros(1, 2, dtype=torch.int32),
                             torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                             torch.zeros(1, 2, 4, dtype=torch.int32))
    with pytest.raises(bind.PkvError):
        bind.make_shared_args(x, cache, cache, torch.zeros(2, 2, dtype=torch.int32),
                              torch.zeros(2, dtype=torch.int32), 1.0, x)
    a, b = torch.zeros(8), torch.zeros(4, 4)
    assert bind._overlap(a[:4], a[3:]) and not bind._overlap(a[:4], a[4:])
    assert bind._overlap(b[:, 0], b[:, 1]) and not bind._overlap(b, a) and not bind._overlap(a[:0], a)
