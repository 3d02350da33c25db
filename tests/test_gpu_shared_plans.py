"""Prefix plans that do not fit the call, and prefix kernels that gave up: what the call
returns then, whatever an earlier call left in the workspace.

A plan made for another call is dropped whole (the rows have their own tokens alone); a row
whose record names a prefix or a length outside the call's tables loses its prefix.  The
expected results are those of the call without these prefixes, within the tolerances that
test_gpu_cache_ops derives."""
import numpy as np
import pytest
import torch

from helpers import dev
from paged_kv_decode_10_gb300 import binding
from test_gpu_cache_ops import check_case, i32, make_case

pytestmark = pytest.mark.gpu

B, HQ, HKV, D = 5, 8, 2, 64
LENS, PLENS, ROWS = [5, 40, 20, 0, 33], [100, 40], [0, 0, 1, 1, -1]
CTAS = 12


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def case(dtype):
    return make_case(B, HQ, HKV, D, dtype, LENS, PLENS, ROWS, 43)


def good_plan(c):
    return binding.shared_plan(ROWS, PLENS, HQ, HKV, D, binding.dtype_code(c["q"]), CTAS)


def run(c, plan, general, space=None, ptab=None, own_plan=None, **kw):
    """The call with this plan, for the sizes of the good one."""
    good = good_plan(c)
    buf = np.zeros(max(len(plan), len(good)) + 512, np.int32)
    buf[:len(plan)] = plan
    parts = 6
    if space is None:
        n = binding.shared_workspace_bytes(B, HQ, HKV, D, 304, int(good[3]))
        space = torch.zeros(n, dtype=torch.uint8, device=dev())
    out, lse = torch.full_like(c["q"], 7.0), torch.full((B, HQ), 7.0, device=dev())
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    kw = {**dict(slots=int(good[3]), num_ctas=CTAS), **kw}
    a = binding.make_shared_args(
        c["q"], c["kc"], c["vc"], torch.from_numpy(c["tab"]).to(dev()), i32(LENS), c["scale"], out,
        prefix_tables=torch.from_numpy(c["ptab"] if ptab is None else ptab).to(dev()),
        prefix_plan=torch.from_numpy(buf).to(dev()), workspace=space, lse=lse, err=err,
        num_parts=parts if general else None, plan=own_plan, **kw)
    binding.decode_attn_shared_args(a)
    torch.cuda.synchronize()
    return out, lse, int(err), space


def without(c, rows):
    """The case with other prefixes of the rows."""
    if all(r < 0 for r in rows):
        return dict(c, plens=[], rows=rows)
    return dict(c, rows=rows)


def after_a_good_call(c, general):
    out, lse, err, space = run(c, good_plan(c), general)
    check_case(c, out, lse, err=err)
    return space


def other_plan(c, what):
    code = binding.dtype_code(c["q"])
    sizes = dict(rows=ROWS, Hq=HQ, Hkv=HKV, dtype=code, ctas=CTAS)
    sizes.update({"fewer rows": dict(rows=ROWS[:2]), "more rows": dict(rows=ROWS + [0, 1]),
                  "KV heads": dict(Hkv=4), "group": dict(Hq=16),
                  "CTAs": dict(ctas=CTAS - 1)}[what])
    return binding.shared_plan(sizes["rows"], PLENS, sizes["Hq"], sizes["Hkv"], D, sizes["dtype"],
                               sizes["ctas"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("general", [False, True])
@pytest.mark.parametrize("what", ["fewer rows", "more rows", "KV heads", "group", "CTAs"])
def test_a_plan_made_for_another_call_is_dropped(dtype, general, what):
    c = case(dtype)
    space = after_a_good_call(c, general)
    out, lse, err, _ = run(c, other_plan(c, what), general, space)
    check_case(without(c, [-1] * B), out, lse, want_err=binding.DEVERR_BAD_PLAN, err=err)
    out, lse, err, _ = run(c, good_plan(c), general, space)
    check_case(c, out, lse, err=err)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("general", [False, True])
def test_a_plan_of_more_partials_than_the_call_has_is_dropped(dtype, general):
    """Where partials are kept; the form for short contexts keeps none."""
    c = case(dtype)
    space = after_a_good_call(c, general)
    out, lse, err, _ = run(c, good_plan(c), general, space, slots=int(good_plan(c)[3]) - 1)
    if general:
        check_case(without(c, [-1] * B), out, lse, want_err=binding.DEVERR_BAD_PLAN, err=err)
    else:
        check_case(c, out, lse, err=err)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("general", [False, True])
@pytest.mark.parametrize("cut", ["prefixes", "width"])
def test_rows_whose_prefix_lies_outside_the_tables_lose_it(dtype, general, cut):
    """A table of one prefix, or too narrow for the longer one."""
    c = case(dtype)
    space = after_a_good_call(c, general)
    ptab = c["ptab"][:1] if cut == "prefixes" else np.ascontiguousarray(c["ptab"][:, :5])
    out, lse, err, _ = run(c, good_plan(c), general, space, ptab=ptab)
    lost = 1 if cut == "prefixes" else 0
    rows = [-1 if r == lost else r for r in ROWS]
    check_case(without(c, rows), out, lse, want_err=binding.DEVERR_BAD_PLAN, err=err)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("what", ["rows", "head", "split", "first", "missing", "no row"])
def test_a_plan_that_leaves_partials_out_is_dropped(dtype, what):
    """Records of items that fit nothing, or an item that no CTA works off."""
    c = case(dtype)
    space = after_a_good_call(c, True)
    plan = good_plan(c)
    ctas = plan[16 + 6 * B:16 + 6 * B + CTAS + 1]
    items = plan[(16 + 6 * B + CTAS + 1 + 3) // 4 * 4:].reshape(-1, 8)
    if what == "missing":
        last = int(np.flatnonzero(np.diff(ctas))[-1])
        ctas[last + 1:] -= 1
    elif what == "no row":
        order = plan[16 + 4 * B:16 + 6 * B].reshape(B, 2)
        order[0, 0] = B
    else:
        field, value = {"rows": (3, 1000), "head": (1, HKV), "split": (6, -1), "first": (2, B)}[what]
        items[0, field] = value
    out, lse, err, _ = run(c, plan, True, space)
    check_case(without(c, [-1] * B), out, lse, want_err=binding.DEVERR_BAD_PLAN, err=err)


@pytest.mark.parametrize("batch", [9, 70])
def test_rows_behind_a_prefix_kernel_that_gave_up_are_nan(batch):
    """Waits of 64 clocks end before the first copy lands: no partial of an earlier call
    passes for this one's."""
    rows = [i % 3 - 1 for i in range(batch)]
    c = make_case(batch, 8, 2, 128, "bf16", [17 + i % 40 for i in range(batch)], [1000, 130], rows, 47)
    code = binding.dtype_code(c["q"])
    plan = binding.shared_plan(rows, [1000, 130], 8, 2, 128, code)
    space = torch.zeros(binding.shared_workspace_bytes(batch, 8, 2, 128, 16, int(plan[3])),
                        dtype=torch.uint8, device=dev())
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    out, lse = torch.empty_like(c["q"]), torch.empty((batch, 8), device=dev())

    def call(flags):
        a = binding.make_shared_args(
            c["q"], c["kc"], c["vc"], torch.from_numpy(c["tab"]).to(dev()), i32(c["lens"]),
            c["scale"], out, prefix_tables=torch.from_numpy(c["ptab"]).to(dev()),
            prefix_plan=torch.from_numpy(plan).to(dev()), workspace=space, lse=lse, err=err,
            num_parts=16, flags=flags)
        binding.decode_attn_shared_args(a)
        torch.cuda.synchronize()

    call(0)
    check_case(c, out, lse, err=int(err))
    call(binding.ATTN_SHORT_WAITS)
    behind = torch.tensor(rows) >= 0
    assert int(err) & binding.DEVERR_TIMEOUT
    assert out[behind.to(dev())].isnan().all() and lse[behind.to(dev())].isnan().all()
    space.zero_()
    err.zero_()
    call(0)
    check_case(c, out, lse, err=int(err))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_records_of_the_own_plan_that_name_no_row(dtype):
    """The own tokens' CTAs skip such records, behind a prefix kernel too, and leave the
    workspace as the next call expects it."""
    c = case(dtype)
    space = after_a_good_call(c, True)
    plan = torch.from_numpy(binding.plan_parts(c["lens"], HKV, D, c["tab"], 6))
    bad = plan.clone()
    bad[:, 0] = B
    out, lse, err, _ = run(c, good_plan(c), True, space, own_plan=bad.to(dev()))
    assert err == binding.DEVERR_BAD_PLAN
    out, lse, err, _ = run(c, good_plan(c), True, space, own_plan=plan.to(dev()))
    check_case(c, out, lse, err=err)
