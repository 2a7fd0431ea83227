"""A clipping table that is only partly its plan's, beside gradients that are
not finite: nothing is scaled, in the one-launch and the two-launch form."""

import math

import pytest

from tests import ffn_util as fu
from tests.gpu_util import say
from tests.test_gpu_clip import check, tensors

pytestmark = pytest.mark.gpu


def ovl():
    from communication_overlap_amd import ovl as _o
    return _o


def same_bits(a, b):
    t = fu.torch()
    kind = t.int16 if a.element_size() == 2 else t.int32
    return t.equal(a.view(kind), b.view(kind))


@pytest.mark.parametrize("sizes", [[50, 7, 33], [70000, 31, 40000], [300000, 9, 5]])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("how", ["another plan's first entries", "a count"])
@pytest.mark.parametrize("max_norm", [0.25, math.inf])
def test_a_partly_foreign_table_beside_gradients_that_are_not_finite(sizes, bad, how, max_norm):
    """The foreign entries name live tensors of their own, so that scaling them
    would show; the Inf or NaN lies behind an entry of the plan's own."""
    o, t = ovl(), fu.torch()
    src, guard = tensors(sizes), tensors(sizes, seed=40)
    src[2][sizes[2] // 2] = bad
    kept, kept_guard = [v.clone() for v in src], [v.clone() for v in guard]
    plan = o.grad_clip_plan(src)
    ws = fu.workspace(plan.workspace_bytes)
    o.grad_clip_upload(plan, ws)
    if how == "a count":  # one element less in the first entry: src, dst, first, end, count
        words = ws[:plan.workspace_bytes // 8 * 8].view(t.int64)
        at = (words == src[0].data_ptr()).nonzero()
        assert at.shape[0] == 2  # src and dst of the entry
        words[int(at[0]) + 4] -= 2
    else:
        o.grad_clip_upload(o.grad_clip_plan(guard[:2]), ws)
    norm = t.full((1,), -1.0, device="cuda")
    say(f"  grad_norm_clip_run on a partly foreign table: {how}, {bad}, {sizes}")
    o.grad_norm_clip_run(plan, max_norm, norm, ws)
    st, _ = o.ovl_check(ws, raise_on_error=False)
    assert st == o.OVL_EINVAL
    assert math.isnan(float(norm))
    assert all(same_bits(a, b) for a, b in zip(src + guard, kept + kept_guard))


@pytest.mark.parametrize("sizes", [[50, 7, 33], [70000, 31, 40000]])
def test_the_sound_table_still_clips(sizes):
    o, t = ovl(), fu.torch()
    src = tensors(sizes)
    kept = [fu.f64(v) for v in src]
    plan = o.grad_clip_plan(src)
    ws = fu.workspace(plan.workspace_bytes)
    o.grad_clip_upload(plan, ws)
    norm = t.full((1,), -1.0, device="cuda")
    o.grad_norm_clip_run(plan, 0.25, norm, ws)
    assert o.ovl_check(ws, raise_on_error=False)[0] == o.OVL_OK
    check(kept, src, float(norm), 0.25)
