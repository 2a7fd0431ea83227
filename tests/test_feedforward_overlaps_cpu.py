"""Buffers that begin where an output does: refused on the host, but for the
pairs that each call names.  The addresses are never dereferenced."""

import ctypes
import itertools

import pytest

Q = [4096 * i for i in range(2, 20)]  # distinct aligned addresses


def ovl():
    from communication_overlap_amd import ovl as _o
    return _o


def no_gpu():
    """What is accepted here would launch on these addresses with a GPU."""
    import torch
    return not torch.cuda.is_available()


LINEAR = ("a", "b", "bias", "residual", "out", "z", "ws")
GRAD = ("dy", "z", "dz", "a", "b", "z_in", "da", "db", "db_in", "dbias", "dbias_in", "ws")
MOE = ("x", "router", "topk", "gates", "w1", "s1", "w2", "s2", "out", "ws")


def pairs(names, written, named):
    for x, y in itertools.combinations(names, 2):
        if (x in written or y in written) and {x, y} not in named:
            yield x, y


def addresses(names, **same):
    at = dict(zip(names, Q))
    at.update({k: at[v] for k, v in same.items()})
    return [at[n] for n in names]


def linear(o, at, **kw):
    d = o.gemm_epilogue_desc(kw.pop("m", 8), 16, 24, "silu", "bf16", "bf16", **kw)
    return o.lib().gemm_epilogue_run(ctypes.byref(d), *at, None)


def grad(o, at, m=8, **kw):
    d = o.gemm_epilogue_grad_desc(m, 16, 24, **{**dict(act="silu", act_in="relu", da_type="bf16", db_type="f32"), **kw})
    dy, z, dz, a, b, z_in, da, db, db_in, dbias, dbias_in, ws = at
    return o.lib().gemm_epilogue_grad_run(ctypes.byref(d), dy, z, dz, a, b, z_in, da, db, db_in, dbias, dbias_in, ws, None)


def moe(o, at, tokens=4):
    d = o.moe_layer_desc(tokens, 64, 32, 8, 2, w_type="fp8")
    return o.lib().moe_layer_run(ctypes.byref(d), *at, None)


NAMED_LINEAR = [{"residual", "out"}]
NAMED_GRAD = [{"dy", "dz"}, {"z", "dz"}, {"z_in", "da"}, {"db_in", "db"}, {"dbias_in", "dbias"}]


@pytest.mark.parametrize("x,y", pairs(LINEAR, {"out", "z", "ws"}, NAMED_LINEAR))
@pytest.mark.parametrize("m", [8, 100])
def test_gemm_epilogue(x, y, m):
    o = ovl()
    assert linear(o, addresses(LINEAR, **{y: x}), m=m) == o.OVL_EINVAL


@pytest.mark.parametrize("x,y", pairs(GRAD, {"dz", "da", "db", "dbias", "ws"}, NAMED_GRAD))
def test_gemm_epilogue_grad(x, y):
    o = ovl()
    assert grad(o, addresses(GRAD, **{y: x})) == o.OVL_EINVAL


@pytest.mark.parametrize("x,y", pairs(("db", "db_in", "dbias", "dbias_in", "ws"), {"db", "dbias", "ws"}, NAMED_GRAD))
def test_gemm_epilogue_grad_without_rows(x, y):
    """db and dbias are written without rows, too."""
    o = ovl()
    assert grad(o, addresses(GRAD, **{y: x}), m=0) == o.OVL_EINVAL


@pytest.mark.parametrize("x,y", pairs(MOE, {"topk", "gates", "out", "ws"}, []))
def test_moe_layer(x, y):
    o = ovl()
    assert moe(o, addresses(MOE, **{y: x})) == o.OVL_EINVAL


@pytest.mark.parametrize("x,y", pairs(MOE, {"out", "ws"}, []))
def test_moe_layer_with_the_caller_s_routing(x, y):
    o = ovl()
    at = addresses(MOE, **{y: x})
    if "router" not in (x, y):
        at[MOE.index("router")] = None
        assert moe(o, at) == o.OVL_EINVAL


@pytest.mark.skipif("not no_gpu()", reason="accepted calls would run on these addresses")
def test_named_and_harmless_pairs_pass():
    """Without a device an accepted call ends with EHIP."""
    o = ovl()
    for x, y in [("residual", "out"), ("a", "b"), ("a", "residual"), ("a", "bias")]:
        assert linear(o, addresses(LINEAR, **{y: x})) == o.OVL_EHIP
    for x, y in [("dy", "dz"), ("z", "dz"), ("z_in", "da"), ("db", "db_in"), ("dbias", "dbias_in"), ("a", "b"),
                 ("z", "z_in"), ("a", "z_in"), ("dy", "z")]:
        assert grad(o, addresses(GRAD, **{y: x})) == o.OVL_EHIP
    at = addresses(GRAD)  # dz is an input without act, and may be `a`
    at[0] = at[1] = None
    at[2] = at[3]
    assert grad(o, at, act="none") == o.OVL_EHIP
    at = addresses(GRAD, dz="z_in")  # z_in is not read without da
    at[GRAD.index("da")] = None
    assert grad(o, at) == o.OVL_EHIP
    for x, y in [("x", "router"), ("w1", "w2"), ("s1", "s2")]:
        assert moe(o, addresses(MOE, **{y: x})) == o.OVL_EHIP


def plan(o, *tensors):
    arr = (o.GradClipTensor * max(1, len(tensors)))(*[o.GradClipTensor(*t) for t in tensors])
    h = ctypes.c_void_p()
    assert o.lib().grad_clip_plan(arr, len(tensors), ctypes.byref(h)) == o.OVL_OK
    return h


def test_clipping_refuses_a_norm_or_workspace_over_a_tensor():
    """src at 1 MiB of 256 float32, dst at 2 MiB; a counted one at 3 MiB within a longer one."""
    o, mib = ovl(), 1 << 20
    h = plan(o, (mib, 2 * mib, 256, 1, 0), (3 * mib, None, 1 << 16, 1, 0), (3 * mib + 64, None, 4, 1, 0))
    size = o.lib().grad_clip_workspace_bytes(h)
    run = lambda norm, ws: o.lib().grad_norm_clip_run(h, 1.0, norm, ws, None)  # noqa: E731
    far, ws = 64 * mib, 128 * mib
    for norm in (mib, mib + 1020, 2 * mib, 2 * mib + 512, 3 * mib + 4, 3 * mib + (1 << 18) - 4, ws, ws + size - 4):
        assert run(norm, ws) == o.OVL_EINVAL
    for base in (mib, 2 * mib, 3 * mib):
        for w in (base, base - size + 16, base + 1008):
            assert run(far, w // 16 * 16) == o.OVL_EINVAL
            assert o.lib().grad_clip_upload(h, w // 16 * 16, None) == o.OVL_EINVAL
    if no_gpu():
        for norm in (mib - 4, mib + 1024, 3 * mib - 4, 3 * mib + (1 << 18), ws - 4, ws + size):
            assert run(norm, ws) == o.OVL_EHIP
        assert o.lib().grad_clip_upload(h, 2 * mib + 1024, None) == o.OVL_EHIP
        assert run(far, 3 * mib + (1 << 18)) == o.OVL_EHIP
    o.lib().grad_clip_plan_destroy(h)
    h = plan(o)
    if no_gpu():
        assert o.lib().grad_norm_clip_run(h, 1.0, far, ws, None) == o.OVL_EHIP
    o.lib().grad_clip_plan_destroy(h)
