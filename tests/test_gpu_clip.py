"""Global gradient norm and clipping against the float64 oracle: lengths from
0, any alignment, thousands of tensors, both types, in place and not."""

import math

import numpy as np
import pytest

import oracle
from tests import ffn_util as fu
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


def ovl():
    from communication_overlap_amd import ovl as _o
    return _o


def run(src, dst, max_norm, plan=None, ws=None):
    o, t = ovl(), fu.torch()
    plan = plan or o.grad_clip_plan(src, dst)
    if ws is None:
        ws = fu.workspace(plan.workspace_bytes)
        o.grad_clip_upload(plan, ws)
    norm = t.full((1,), -1.0, device="cuda")
    say(f"  grad_norm_clip_run {len(src)} tensors, max_norm {max_norm}")
    o.grad_norm_clip_run(plan, max_norm, norm, ws)
    return float(norm), plan, ws


def check(src64, dst, norm, max_norm):
    """norm rounded once from 64 bits; coef and the product one float32
    rounding each, then the type's."""
    want, out = oracle.grad_norm_clip(src64, max_norm)
    assert abs(norm - want) <= (fu.U + 1e-12) * want
    for i, (d, w) in enumerate(zip(dst, out)):
        if d is None:
            continue
        name = "bf16" if d.dtype == fu.torch().bfloat16 else "f32"
        # below the normal range a step is absolute: 2^-149 for float32, 2^-133 for bf16
        fu.within(d, w, 3 * fu.U * np.abs(w) + fu.HALF[name] * np.abs(w) + (2.0 ** -133 if name == "bf16" else 2.0 ** -149),
                  f"tensor {i}")


def tensors(sizes, kinds=("f32", "bf16"), sigma=1.0, seed=0):
    return [fu.normal(seed + i, n, sigma=sigma, dtype=kinds[i % len(kinds)]) for i, n in enumerate(sizes)]


@pytest.mark.parametrize("sizes", [
    [1], [2, 1], [3, 5, 7, 9, 1, 15, 17], [0, 1, 0, 0, 33, 0], [8191, 4097, 1], [65536 * 3 + 5], [1 << 20, 3, 1 << 18, 7],
    [17] * 500, [1] * 3001, [0, 0], [],
])
@pytest.mark.parametrize("kinds", [("f32",), ("bf16",), ("bf16", "f32", "f32")])
@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_sizes_and_types(sizes, kinds, max_norm):
    t = fu.torch()
    src = tensors(sizes, kinds)
    dst = [t.full_like(v, 7.0) for v in src]
    norm, _, _ = run(src, dst, max_norm)
    check([fu.f64(v) for v in src], dst, norm, max_norm)


@pytest.mark.parametrize("max_norm", [0.25, 1e9, math.inf])
@pytest.mark.parametrize("n", [5, 100, 40000, 700001])
def test_in_place(n, max_norm):
    src = tensors([n, 3, n // 2 + 1])
    before = [fu.f64(v) for v in src]
    norm, _, _ = run(src, None, max_norm)
    check(before, src, norm, max_norm)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 2, 3, 9, 31, 1000, 50001, 300007])
def test_every_alignment_and_nothing_beside(n, kind):
    """Views into one buffer at every element offset, source and output
    offsets alike and different; the elements beside keep their values."""
    t = fu.torch()
    per = 4 if kind == "f32" else 8
    src, dst, bufs = [], [], []
    for so in range(per):
        for do in {so, (so + 1) % per}:
            sb, db = fu.normal(so, n + 2 * per, dtype=kind), t.full((n + 2 * per,), 7.0, dtype=fu.ttype(kind), device="cuda")
            src.append(sb[so + 1:so + 1 + n])
            dst.append(db[do + 1:do + 1 + n])
            bufs.append((db, do + 1))
    norm, _, _ = run(src, dst, 0.5)
    check([fu.f64(v) for v in src], dst, norm, 0.5)
    for db, at in bufs:
        assert bool((db[:at] == 7).all()) and bool((db[at + n:] == 7).all())


def test_norm_only_entries_and_repeated_sources():
    src = tensors([100, 200, 31])
    norm, _, _ = run(src + [src[1]], [None, src[1].clone(), None, None], 0.5)
    want = math.sqrt(sum(float((fu.f64(v) ** 2).sum()) for v in src + [src[1]]))
    assert abs(norm - want) <= (fu.U + 1e-12) * want


@pytest.mark.parametrize("n", [50, 200000])
@pytest.mark.parametrize("sigma", [1e-30, 1e30])
def test_squares_beyond_float32(n, sigma):
    t = fu.torch()
    src = tensors([n, n // 2], sigma=sigma)
    dst = [t.empty_like(v) for v in src]
    norm, _, _ = run(src, dst, 1.0)
    check([fu.f64(v) for v in src], dst, norm, 1.0)


@pytest.mark.parametrize("n", [50, 200000])
def test_not_finite(n):
    t = fu.torch()
    for bad, in_norm in ((float("inf"), math.inf), (float("nan"), math.nan)):
        src = tensors([n, 9])
        src[0][n // 2] = bad
        dst = [t.full_like(v, 7.0) for v in src]
        norm, _, _ = run(src, dst, 1.0)
        assert norm == in_norm or (math.isnan(norm) and math.isnan(in_norm))
        if math.isinf(in_norm):  # coef 0: inf * 0 is NaN, the rest is zero
            assert bool(dst[0][n // 2].isnan()) and not bool(dst[1].any())
        else:
            assert all(bool(d.isnan().all()) for d in dst)


def test_zero_gradients_and_max_norm_zero():
    t = fu.torch()
    src = [t.zeros(1000, device="cuda")]
    norm, _, _ = run(src, None, 1.0)
    assert norm == 0 and not bool(src[0].any())
    src = tensors([1000])
    run(src, None, 0.0)
    assert not bool(src[0].any())


def test_past_two_to_the_31_elements():
    t = fu.torch()
    n = (1 << 31) + 5
    big = t.full((n,), 0.5, dtype=t.bfloat16, device="cuda")
    big[-1] = 2.0
    norm, _, _ = run([big], None, 1.0)
    want = math.sqrt(0.25 * (n - 1) + 4.0)
    assert abs(norm - want) <= (fu.U + 1e-12) * want
    coef = np.float32(1.0 / (want + 1e-6))
    lo, hi = float(t.tensor(0.5 * float(coef)).bfloat16()), float(t.tensor(2.0 * float(coef)).bfloat16())
    assert float(big[0]) == lo and float(big[-2]) == lo and float(big[-1]) == hi
    assert bool((big[:-1] == lo).all())


def test_one_plan_many_runs_capture_and_new_values():
    """Captured and replayed on new values between eager runs of another plan
    whose table lies in another workspace."""
    t = fu.torch()
    src = tensors([70000, 31, 4097])
    dst = [t.empty_like(v) for v in src]
    other = tensors([123456], ("f32",), seed=50)
    _, plan, ws = run(src, dst, 0.5)
    norm = t.empty(1, device="cuda")
    o = ovl()
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g, stream=s):
        o.grad_norm_clip_run(plan, 0.5, norm, ws)
    for i in range(3):
        for j, v in enumerate(src):
            v.copy_(fu.normal(100 + 10 * i + j, v.numel(), dtype="bf16" if v.dtype == t.bfloat16 else "f32"))
        run(other, None, 0.25)
        g.replay()
        t.cuda.synchronize()
        check([fu.f64(v) for v in src], dst, float(norm), 0.5)
        first = [d.clone() for d in dst]
        o.grad_norm_clip_run(plan, 0.5, norm, ws)
        assert all(t.equal(a, b) for a, b in zip(first, dst))


@pytest.mark.parametrize("sizes", [[50, 7], [70000, 31, 0, 40000]])
@pytest.mark.parametrize("how", ["never uploaded", "another plan's", "another call's", "one entry"])
def test_a_table_that_is_not_the_plan_s_is_refused(sizes, how):
    """Nothing that such a table names is read or written: EINVAL, a NaN norm,
    gradients as they were; after an upload the run is whole."""
    o, t = ovl(), fu.torch()
    src = tensors(sizes)
    kept = [v.clone() for v in src]
    plan = o.grad_clip_plan(src)
    d = o.gemm_epilogue_desc(8, 4096, 4096)
    ws = fu.workspace(max(plan.workspace_bytes, o.gemm_epilogue_workspace_bytes(d)))
    if how == "another plan's":
        other = [v.clone() for v in src]
        o.grad_clip_upload(o.grad_clip_plan(other), ws)
    elif how != "never uploaded":
        o.grad_clip_upload(plan, ws)
        if how == "another call's":
            out = t.empty(8, 4096, dtype=t.bfloat16, device="cuda")
            o.gemm_epilogue_run(d, fu.normal(1, 8, 4096), fu.normal(2, 4096, 4096), None, None, out, None, ws)
        else:  # the first entry's number of elements
            words = ws[:plan.workspace_bytes // 8 * 8].view(t.int64)
            at = (words == src[0].data_ptr()).nonzero()
            assert at.shape[0] == 2  # src and dst of the entry
            words[int(at[0]) + 4] += 2
    norm = t.full((1,), -1.0, device="cuda")
    say(f"  grad_norm_clip_run on a table: {how}")
    o.grad_norm_clip_run(plan, 0.25, norm, ws)
    st, detail = o.ovl_check(ws, raise_on_error=False)
    assert st == o.OVL_EINVAL
    assert math.isnan(float(norm))
    assert all(t.equal(a, b) for a, b in zip(src, kept))
    o.ovl_flags_reset(None, 0, ws, ws.numel())
    o.grad_clip_upload(plan, ws)
    o.grad_norm_clip_run(plan, 0.25, norm, ws)
    assert o.ovl_check(ws, raise_on_error=False)[0] == o.OVL_OK
    check([fu.f64(v) for v in kept], src, float(norm), 0.25)
