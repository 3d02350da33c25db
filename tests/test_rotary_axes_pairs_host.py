"""A rotary table with axes and its axes belong together: neither works without the other."""
import ctypes

import pytest


@pytest.fixture
def bind(host_lib):
    from paged_kv_decode_10_gb300 import binding
    return binding


def call(bind, table, axes):
    a = bind.RotaryArgs()
    a.rotary = ctypes.pointer(table)
    a.T, a.Hkv, a.d, a.dtype = 4, 1, 64, bind.F32
    a.k = a.k_out = a.positions = 1 << 20
    a.k_stride = a.k_out_stride = 64
    lib = bind.load()
    if axes is None:
        return lib.pkv_rotary_append(ctypes.byref(a), None)
    return lib.pkv_rotary_axes_append(ctypes.byref(a), ctypes.byref(axes), 4, None)


KINDS = [dict(ladder="shared"), dict(ladder="own"), dict(order="cyclic"), dict(layout="interleaved"),
         dict(ladder="own", base=500000.0)]


@pytest.mark.parametrize("kind", KINDS)
def test_a_table_with_axes_is_no_plain_one(bind, kind):
    rot = bind.Rotary(64, sections=(12, 20), **kind)
    assert call(bind, rot.table, None) == bind.ERR_INVALID_ARG
    assert call(bind, bind.Rotary(64).table, rot.axes) == bind.ERR_INVALID_ARG


def test_table_and_axes_of_two_makings_are_refused(bind):
    made = [bind.Rotary(64, sections=(12, 20), **kind) for kind in KINDS]
    made += [bind.Rotary(64, sections=(20, 12)), bind.Rotary(64, sections=(12, 10, 10))]
    for x in made:
        for y in made:
            if x is not y:
                assert call(bind, x.table, y.axes) == bind.ERR_INVALID_ARG
    twin = bind.Rotary(64, sections=(12, 20), **KINDS[0])      # (equal ones are as good as the same)
    assert twin.table.check ^ twin.axes.check == made[0].table.check ^ made[0].axes.check
    assert twin.table.check == made[0].table.check


def test_what_no_call_filled_is_refused(bind):
    rot = bind.Rotary(64, sections=(12, 20))
    assert call(bind, bind.RotaryTable(d=64, rot_dim=64), None) == bind.ERR_INVALID_ARG
    assert call(bind, bind.RotaryTable(d=64, rot_dim=64), bind.RotaryAxes(n_axes=2, pairs=32)) == bind.ERR_INVALID_ARG
    assert call(bind, rot.table, bind.RotaryAxes(n_axes=2, pairs=32)) == bind.ERR_INVALID_ARG
    assert call(bind, bind.RotaryTable(d=64, rot_dim=64), rot.axes) == bind.ERR_INVALID_ARG
