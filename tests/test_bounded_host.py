"""``BoundedDecoder`` on the host: what it makes of its arguments and how it keeps its state,
with the device part of ``PagedDecoder`` replaced by plain attributes."""
import numpy as np
import contextlib

import numpy as np
import pytest
import torch

from paged_kv_decode_10_gb300 import bounded


@pytest.fixture
def bind(host_lib):
    from paged_kv_decode_10_gb300 import binding
    return binding


@pytest.fixture
def make(bind, monkeypatch):
    """``BoundedDecoder`` without a GPU: buffers on the CPU, nothing launched."""
    def paged_init(self, num_blocks, Hq, Hkv, d, dtype, max_seqs, max_blocks_per_seq,
                   initial_free=None, device="cuda", num_parts=None, rope_base=10000.0, scale=None,
                   flags=0, k_cache=None, v_cache=None, metadata="copy", n_layers=1, plan=True,
                   layer_merge_helpers=None):
        self.torch, self.device, self.n_layers = torch, torch.device("cpu"), n_layers
        self.Hq, self.Hkv, self.d, self.dtype = Hq, Hkv, d, dtype
        self.tdtype = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
        self.bt_stride, self.num_parts, self.scale = max_blocks_per_seq, num_parts, scale or d**-0.5
        self.rope_base, self.flags = rope_base, flags
        self.alloc = bind.BlockAllocator(num_blocks, max_seqs, max_blocks_per_seq, initial_free)
    monkeypatch.setattr(bounded.PagedDecoder, "__init__", paged_init)
    monkeypatch.setattr(bind, "shared_default_parts", lambda *a: 4)
    base = dict(num_blocks=64, Hq=8, Hkv=2, d=64, dtype="f32", max_seqs=4, budget=24, slack=8)
    return lambda **kw: bounded.BoundedDecoder(**{**base, **kw})


def test_rope_base_reaches_the_rotary_table(bind, make):
    for kw, base in (({}, 10000.0), (dict(rope_base=500000.0), 500000.0), (dict(rope_base=1.0), 1.0)):
        want = bind.Rotary(64, base=base)
        assert list(make(**kw).rotary.table.turns) == list(want.table.turns)
    own = bind.Rotary(64, rot_dim=32, base=77.0)
    assert make(rotary=own).rotary is own


def test_rope_base_beside_a_rotary_is_refused(bind, make):
    with pytest.raises(ValueError):
        make(rotary=bind.Rotary(64), rope_base=500000.0)


@pytest.fixture
def two_prefixes(bind, make, monkeypatch):
    """A decoder with two prefixes and a sequence behind each."""
    real = bind.shared_plan
    monkeypatch.setattr(bind, "shared_plan", lambda *a: real(*a, num_ctas=8))
    dec = make()
    monkeypatch.setattr(dec, "_write", lambda *a: None)
    prefixes = [dec.add_prefix(*[torch.zeros((n, 2, 64))] * 2) for n in (40, 100)]
    return dec, [dec.join(prefix=p) for p in prefixes]


@pytest.mark.parametrize("what", ["plan", "tables", "workspace bytes", "workspace"])
def test_a_plan_that_cannot_be_made_leaves_the_last_one(bind, two_prefixes, monkeypatch, what):
    dec, (a, b) = two_prefixes
    dec._prefix_state([a])
    dec._calls["buffer"] = "calls"
    state = {k: getattr(dec, k) for k in ("_prefix_args", "_space", "_calls", "_plan_key", "_rows_now")}
    args = dict(dec._prefix_args)
    assert args["prefix_tables"].shape == (1, 3)

    def fail(*a, **kw):
        raise RuntimeError("out of memory")

    with monkeypatch.context() as m:
        if what == "plan":
            m.setattr(bind, "shared_plan", fail)
        elif what == "tables":
            m.setattr(dec.alloc, "seq_blocks", fail)
        elif what == "workspace bytes":
            m.setattr(bind, "shared_workspace_bytes", fail)
        else:
            m.setattr(torch, "zeros", fail)
        with pytest.raises(RuntimeError):
            dec._prefix_state([b])
    assert all(getattr(dec, k) is v for k, v in state.items())
    assert dec._prefix_args.keys() == args.keys()
    assert all(dec._prefix_args[k] is v for k, v in args.items())
    assert dec._calls == {"buffer": "calls"}
    dec._prefix_state([a])                    # the last batch again: nothing was lost
    assert dec._prefix_args is state["_prefix_args"] and dec._calls == {"buffer": "calls"}
    dec._prefix_state([b])
    assert dec._prefix_args["prefix_tables"].shape == (1, 7) and dec._calls == {}
    assert dec._rows_now == [b]


def test_arguments_that_do_not_reach_the_step_are_refused(bind, make):
    for flags in (bind.ATTN_SIMT, bind.ATTN_SEPARATE_MERGE, bind.STEP_FUSED,
                  bind.ATTN_CHECK_PLAN | bind.ATTN_SIMT, 1 << 20):
        with pytest.raises(ValueError):
            make(flags=flags)
    for helpers in (True, False):
        with pytest.raises(ValueError):
            make(layer_merge_helpers=helpers)
    make(flags=bind.ATTN_CHECK_PLAN, layer_merge_helpers=None)


@pytest.mark.parametrize("kw,short", [(dict(), True), (dict(num_parts=0), True),
                                      (dict(num_parts=5), False), (dict(flags=16), False)])
def test_flags_and_partition_reach_the_calls(bind, make, monkeypatch, kw, short):
    """A stated partition and flags exclude the form for short contexts, as in the call."""
    assert bind.ATTN_CHECK_PLAN == 16
    dec = make(**kw)
    seen = []
    monkeypatch.setattr(bind, "make_rotary_args", lambda *a, **k: None)
    monkeypatch.setattr(bind, "make_shared_args", lambda *a, **k: seen.append(k))
    x = torch.zeros(1, 4, 8, 64)
    dec.q_rots = dec.k_rots = dec.outs = x
    dec.k_caches = dec.v_caches = dec.masses
    dec.positions = dec.slots = dec.tables = dec.seq_lens = torch.zeros(4)
    dec.plan, dec.err = "plan", None
    dec._prepared(1, x[:, :1], x[:, :1], x[:, :1])
    assert len(seen) == 1 and seen[0]["flags"] == kw.get("flags", 0)
    if short:
        assert "num_parts" not in seen[0] and "plan" not in seen[0]
    else:
        assert seen[0]["plan"] == "plan" and seen[0]["num_parts"] == kw.get("num_parts", 4)


def test_sequences_to_evict_may_come_from_an_iterator(make, monkeypatch):
    dec = make()
    ids = [dec.join(20), dec.join(30)]
    seen = []
    monkeypatch.setattr(dec, "_on", lambda stream: contextlib.nullcontext())
    monkeypatch.setattr(dec, "_evict", lambda s, keep: seen.append((s, keep)))
    dec.evict(iter(ids), 5)
    dec.evict(np.array(ids))
    assert seen == [(ids, 5), (ids, 24)]
    with pytest.raises(ValueError):
        dec.evict(iter([ids[0], ids[0]]))


def test_an_eviction_that_cannot_be_prepared_moves_nothing(bind, make, monkeypatch):
    """Every layer's call is made before the first is launched."""
    dec = make(n_layers=3)
    dec.k_caches = dec.v_caches = torch.zeros(3, 1)
    dec.err, sid, launched, made = None, dec.join(20), [], []
    monkeypatch.setattr(dec, "_on", lambda stream: contextlib.nullcontext())
    monkeypatch.setattr(bind, "evict_args", launched.append)

    def prepare(*a, **kw):
        if len(made) == fail_at:
            raise RuntimeError("out of memory")
        made.append(kw["workspace"])
        return len(made)

    monkeypatch.setattr(bind, "make_evict_args", prepare)
    fail_at = 2
    with pytest.raises(RuntimeError):
        dec.evict([sid], 5)
    assert launched == [] and dec.alloc.seq_len(sid) == 20 and dec._held[sid] == 20
    fail_at, made[:] = None, []
    dec.evict([sid], 5)
    assert launched == [1, 2, 3] and dec.alloc.seq_len(sid) == 5 and dec._held[sid] == 5
    assert all(w is made[0] for w in made)        # one layer after the other in one workspace
