"""Host side of the feed-forward calls on the CPU: every refusal comes before
any device work, and the size queries answer 0 for what is refused."""

import ctypes

import pytest


def ovl():
    from communication_overlap_amd import ovl as _o
    return _o


P = 4096  # an aligned address that nothing dereferences: the refusals come first


def linear(o, desc=None, a=P, b=P, bias=None, residual=None, out=P, z=None, ws=P, **kw):
    d = desc or o.gemm_epilogue_desc(*kw.pop("mnk", (8, 16, 24)), **kw)
    return o.lib().gemm_epilogue_run(ctypes.byref(d), a, b, bias, residual, out, z, ws, None), d


@pytest.mark.parametrize("kw,status", [
    (dict(mnk=(-1, 16, 24)), "OVL_ESHAPE"),
    (dict(mnk=(8, 0, 24)), "OVL_ESHAPE"),
    (dict(mnk=(8, 16, 0)), "OVL_ESHAPE"),
    (dict(mnk=(8, 20, 24)), "OVL_EALIGN"),
    (dict(mnk=(8, 16, 20)), "OVL_EALIGN"),
    (dict(mnk=((1 << 20) + 8, 16, 24)), "OVL_EUNSUPPORTED"),
    (dict(mnk=(8, (1 << 20) + 8, 24)), "OVL_EUNSUPPORTED"),
    (dict(mnk=(1 << 18, 16, 4096)), "OVL_EUNSUPPORTED"),       # a of 2 GiB
    (dict(mnk=(8, 1 << 18, 4096)), "OVL_EUNSUPPORTED"),        # b of 2 GiB
    (dict(lda=16), "OVL_ESHAPE"), (dict(ldb=8), "OVL_ESHAPE"), (dict(ldo=8), "OVL_ESHAPE"),
    (dict(ldz=8), "OVL_ESHAPE"), (dict(ldr=8), "OVL_ESHAPE"), (dict(lda=-8), "OVL_ESHAPE"),
    (dict(lda=28), "OVL_EALIGN"), (dict(ldo=20), "OVL_EALIGN"),
    (dict(lda=(1 << 20) + 8), "OVL_EUNSUPPORTED"),
    (dict(act=5), "OVL_EINVAL"), (dict(act=-1), "OVL_EINVAL"), (dict(out_type=2), "OVL_EINVAL"),
    (dict(res_type=7), "OVL_EINVAL"),
    (dict(a=None), "OVL_EINVAL"), (dict(b=None), "OVL_EINVAL"), (dict(out=None), "OVL_EINVAL"),
    (dict(ws=None), "OVL_EINVAL"),
    (dict(a=P + 2), "OVL_EALIGN"), (dict(b=P + 8), "OVL_EALIGN"), (dict(bias=P + 4), "OVL_EALIGN"),
    (dict(residual=P + 8), "OVL_EALIGN"), (dict(out=P + 8), "OVL_EALIGN"), (dict(z=P + 8), "OVL_EALIGN"),
    (dict(ws=P + 8), "OVL_EALIGN"),
])
def test_gemm_epilogue_refuses(kw, status):
    o = ovl()
    st, d = linear(o, **kw)
    assert st == getattr(o, status)
    if not set(kw) & {"a", "b", "bias", "residual", "out", "z", "ws"}:
        assert o.gemm_epilogue_workspace_bytes(d) == 0


def test_gemm_epilogue_reserved_and_null_desc():
    o = ovl()
    d = o.gemm_epilogue_desc(8, 16, 24)
    d.reserved = 1
    assert linear(o, d)[0] == o.OVL_EINVAL
    assert o.lib().gemm_epilogue_run(None, P, P, None, None, P, None, P, None) == o.OVL_EINVAL
    assert o.lib().gemm_epilogue_workspace_bytes(None) == 0


def test_gemm_epilogue_without_rows_touches_nothing():
    o = ovl()
    d = o.gemm_epilogue_desc(0, 16, 24)
    assert linear(o, d, a=None, b=None, out=None)[0] == o.OVL_OK


def grad(o, desc=None, dy=None, z=None, dz=P, a=P, b=P, z_in=None, da=P, db=P, db_in=None, dbias=P, dbias_in=None,
         ws=P, **kw):
    d = desc or o.gemm_epilogue_grad_desc(*kw.pop("mnk", (8, 16, 24)), **kw)
    return o.lib().gemm_epilogue_grad_run(ctypes.byref(d), dy, z, dz, a, b, z_in, da, db, db_in, dbias, dbias_in, ws,
                                          None), d


@pytest.mark.parametrize("kw,status", [
    (dict(mnk=(-1, 16, 24)), "OVL_ESHAPE"), (dict(mnk=(8, 20, 24)), "OVL_EALIGN"),
    (dict(mnk=(8, 16, 4)), "OVL_ESHAPE"), (dict(mnk=((1 << 20) + 8, 16, 24)), "OVL_EUNSUPPORTED"),
    (dict(mnk=(1 << 18, 4096, 8)), "OVL_EUNSUPPORTED"),  # dz of 2 GiB
    (dict(lda=16), "OVL_ESHAPE"), (dict(ldb=8), "OVL_ESHAPE"), (dict(lddz=8), "OVL_ESHAPE"),
    (dict(lddy=8), "OVL_ESHAPE"), (dict(ldz=8), "OVL_ESHAPE"), (dict(ldz_in=16), "OVL_ESHAPE"),
    (dict(ldda=16), "OVL_ESHAPE"), (dict(lddb=8), "OVL_ESHAPE"), (dict(ldda=28), "OVL_EALIGN"),
    (dict(act=9), "OVL_EINVAL"), (dict(act_in=9), "OVL_EINVAL"), (dict(da_type=2), "OVL_EINVAL"),
    (dict(db_type=2), "OVL_EINVAL"), (dict(dy_type=3), "OVL_EINVAL"),
    (dict(dz=None), "OVL_EINVAL"), (dict(a=None), "OVL_EINVAL"), (dict(b=None), "OVL_EINVAL"),
    (dict(ws=None), "OVL_EINVAL"),
    (dict(db=None, db_in=P), "OVL_EINVAL"), (dict(dbias=None, dbias_in=P), "OVL_EINVAL"),
    (dict(z_in=P), "OVL_EINVAL"),                     # act_in is NONE
    (dict(act_in="silu"), "OVL_EINVAL"),              # act_in without z_in
    (dict(act="silu"), "OVL_EINVAL"), (dict(act="silu", dy=P), "OVL_EINVAL"),
    (dict(dy=P), "OVL_EINVAL"), (dict(z=P), "OVL_EINVAL"),  # act is NONE
    (dict(dz=P + 8), "OVL_EALIGN"), (dict(a=P + 8), "OVL_EALIGN"), (dict(b=P + 8), "OVL_EALIGN"),
    (dict(da=P + 8), "OVL_EALIGN"), (dict(db=P + 8), "OVL_EALIGN"), (dict(db_in=P + 8), "OVL_EALIGN"),
    (dict(dbias=P + 4), "OVL_EALIGN"), (dict(dbias_in=P + 4), "OVL_EALIGN"), (dict(ws=P + 4), "OVL_EALIGN"),
])
def test_gemm_epilogue_grad_refuses(kw, status):
    o = ovl()
    st, d = grad(o, **kw)
    assert st == getattr(o, status)
    assert o.lib().gemm_epilogue_grad_run(None, *[P] * 12, None) == o.OVL_EINVAL
    assert o.lib().gemm_epilogue_grad_workspace_bytes(None) == 0


def moe(o, desc=None, x=P, router=P, topk=P, gates=P, w1=P, s1=None, w2=P, s2=None, out=P, ws=P, **kw):
    d = desc or o.moe_layer_desc(*kw.pop("size", (4, 64, 32, 8, 2)), **kw)
    return o.lib().moe_layer_run(ctypes.byref(d), x, router, topk, gates, w1, s1, w2, s2, out, ws, None), d


@pytest.mark.parametrize("kw,status", [
    (dict(size=(-1, 64, 32, 8, 2)), "OVL_ESHAPE"), (dict(size=(4, 0, 32, 8, 2)), "OVL_ESHAPE"),
    (dict(size=(4, 64, 0, 8, 2)), "OVL_ESHAPE"), (dict(size=(4, 64, 32, 0, 1)), "OVL_ESHAPE"),
    (dict(size=(4, 64, 32, 8, 0)), "OVL_ESHAPE"), (dict(size=(4, 64, 32, 2, 3)), "OVL_ESHAPE"),
    (dict(size=(4, 60, 32, 8, 2)), "OVL_EALIGN"), (dict(size=(4, 64, 36, 8, 2)), "OVL_EALIGN"),
    (dict(size=(4, 72, 32, 8, 2), w_type="fp8", s1=P, s2=P), "OVL_EALIGN"),
    (dict(size=(129, 64, 32, 8, 2)), "OVL_EUNSUPPORTED"), (dict(size=(4, 64, 32, 257, 2)), "OVL_EUNSUPPORTED"),
    (dict(size=(4, 64, 32, 16, 9)), "OVL_EUNSUPPORTED"), (dict(size=(4, 65544, 32, 8, 2)), "OVL_EUNSUPPORTED"),
    (dict(size=(4, 65536, 8192, 8, 2)), "OVL_EUNSUPPORTED"),  # an expert of 2 GiB
    (dict(act=7), "OVL_EINVAL"), (dict(gated=2), "OVL_EINVAL"), (dict(norm_topk=3), "OVL_EINVAL"),
    (dict(w_type=1), "OVL_EINVAL"), (dict(out_type=2), "OVL_EINVAL"),
    (dict(x=None), "OVL_EINVAL"), (dict(topk=None), "OVL_EINVAL"), (dict(gates=None), "OVL_EINVAL"),
    (dict(w1=None), "OVL_EINVAL"), (dict(w2=None), "OVL_EINVAL"), (dict(out=None), "OVL_EINVAL"),
    (dict(ws=None), "OVL_EINVAL"), (dict(s1=P), "OVL_EINVAL"), (dict(s1=P, s2=P), "OVL_EINVAL"),
    (dict(w_type="fp8"), "OVL_EINVAL"), (dict(w_type="fp8", s1=P), "OVL_EINVAL"),
    (dict(x=P + 8), "OVL_EALIGN"), (dict(w1=P + 8), "OVL_EALIGN"), (dict(w2=P + 8), "OVL_EALIGN"),
    (dict(out=P + 8), "OVL_EALIGN"), (dict(topk=P + 2), "OVL_EALIGN"), (dict(gates=P + 2), "OVL_EALIGN"),
    (dict(router=P + 2), "OVL_EALIGN"), (dict(ws=P + 8), "OVL_EALIGN"),
])
def test_moe_layer_refuses(kw, status):
    o = ovl()
    st, d = moe(o, **kw)
    assert st == getattr(o, status)
    assert o.lib().moe_layer_run(None, *[P] * 10, None) == o.OVL_EINVAL
    assert o.lib().moe_layer_workspace_bytes(None) == 0


def test_moe_layer_without_tokens_touches_nothing():
    o = ovl()
    d = o.moe_layer_desc(0, 64, 32, 8, 2)
    assert moe(o, d, x=None, router=None, topk=None, gates=None, w1=None, w2=None, out=None)[0] == o.OVL_OK


def plan(o, *tensors):
    arr = (o.GradClipTensor * max(1, len(tensors)))(*[o.GradClipTensor(*t) for t in tensors])
    h = ctypes.c_void_p()
    st = o.lib().grad_clip_plan(arr, len(tensors), ctypes.byref(h))
    return st, h


@pytest.mark.parametrize("tensors,status", [
    ([(P, P, 4, 2, 0)], "OVL_EINVAL"),                           # type
    ([(P, P, 4, 1, 5)], "OVL_EINVAL"),                           # reserved
    ([(P, P, -1, 1, 0)], "OVL_ESHAPE"),
    ([(P, P, (1 << 40) + 1, 1, 0)], "OVL_EUNSUPPORTED"),
    ([(None, P, 4, 1, 0)], "OVL_EINVAL"),
    ([(P + 2, P + 2, 4, 1, 0)], "OVL_EALIGN"), ([(P, P + 64 + 1, 4, 0, 0)], "OVL_EALIGN"),
    ([(P, P + 8, 4, 1, 0)], "OVL_EINVAL"),                       # dst shifted within src
    ([(P, P, 4, 1, 0), (P + 8, P + 8, 4, 1, 0)], "OVL_EINVAL"),  # two overlapping tensors in place
    ([(P, P, 4, 1, 0), (P, P, 4, 1, 0)], "OVL_EINVAL"),          # the same tensor twice
    ([(P, None, 4, 1, 0), (P, P, 4, 1, 0)], "OVL_EINVAL"),       # one counted, one written
    ([(P, P + 64, 16, 1, 0), (P + 256, P + 96, 4, 1, 0)], "OVL_EINVAL"),  # overlapping outputs
])
def test_grad_clip_plan_refuses(tensors, status):
    o = ovl()
    st, h = plan(o, *tensors)
    assert st == getattr(o, status) and not h.value


def test_grad_clip_plan_accepts():
    o = ovl()
    for tensors in ([], [(None, None, 0, 1, 0)], [(P, None, 4, 1, 0), (P, None, 4, 1, 0)],
                    [(P, P, 4, 1, 0), (P + 16, P + 16, 3, 0, 0)], [(P + 2, P + 64, 7, 0, 0)],
                    [(P, P + 16, 4, 1, 0)]):
        st, h = plan(o, *tensors)
        assert st == o.OVL_OK
        assert o.lib().grad_clip_workspace_bytes(h) > o.ERROR_RECORD_BYTES
        assert o.lib().grad_norm_clip_run(h, -1.0, P, P, None) == o.OVL_EINVAL
        assert o.lib().grad_norm_clip_run(h, float("nan"), P, P, None) == o.OVL_EINVAL
        assert o.lib().grad_norm_clip_run(h, 1.0, None, P, None) == o.OVL_EINVAL
        assert o.lib().grad_norm_clip_run(h, 1.0, P, None, None) == o.OVL_EINVAL
        assert o.lib().grad_norm_clip_run(h, 1.0, P + 2, P, None) == o.OVL_EALIGN
        assert o.lib().grad_norm_clip_run(h, 1.0, P, P + 8, None) == o.OVL_EALIGN
        assert o.lib().grad_clip_upload(h, None, None) == o.OVL_EINVAL
        assert o.lib().grad_clip_upload(h, P + 8, None) == o.OVL_EALIGN
        o.lib().grad_clip_plan_destroy(h)
    assert o.lib().grad_clip_plan(None, 1, ctypes.byref(ctypes.c_void_p())) == o.OVL_EINVAL
    assert o.lib().grad_clip_plan(None, 0, None) == o.OVL_EINVAL
    assert o.lib().grad_clip_workspace_bytes(None) == 0
    assert o.lib().grad_norm_clip_run(None, 1.0, P, P, None) == o.OVL_EINVAL


def test_binding_refuses_host_and_short_tensors():
    """Tensors off the current device are refused before the library is called."""
    import torch
    o = ovl()
    d = o.gemm_epilogue_desc(8, 16, 24)
    t = torch.zeros(8, 24, dtype=torch.bfloat16)
    with pytest.raises(o.OvlError) as e:
        o.gemm_epilogue_run(d, t, P, None, None, P, None, P, stream=0)
    assert e.value.status == o.OVL_EINVAL
    with pytest.raises(o.OvlError):
        o.grad_clip_plan([torch.zeros(4)])
    with pytest.raises(o.OvlError):
        o.grad_clip_plan([torch.zeros(4)], [])


def test_binding_refuses_a_plan_of_another_device():
    o = ovl()
    p = o.grad_clip_plan([])
    p.device = 5
    for call in (lambda: o.grad_clip_upload(p, P, stream=0), lambda: o.grad_norm_clip_run(p, 1.0, P, P, stream=0)):
        with pytest.raises(o.OvlError) as e:
            call()
        assert e.value.status == o.OVL_EINVAL


Q = [4096 * i for i in range(2, 16)]  # distinct aligned addresses that nothing dereferences


@pytest.mark.parametrize("kw", [
    dict(out=Q[0]), dict(out=Q[1]), dict(z=Q[0]), dict(z=Q[1]), dict(z=Q[3]),      # over an input or another output
    dict(residual=Q[5], z=Q[5]),
    dict(residual=Q[3], res_type="f32"), dict(residual=Q[3], ldr=24),               # in place of another type or stride
])
def test_gemm_epilogue_refuses_overlaps(kw):
    o = ovl()
    assert linear(o, **{**dict(a=Q[0], b=Q[1], out=Q[3], ws=Q[4]), **kw})[0] == o.OVL_EINVAL


@pytest.mark.parametrize("kw", [
    dict(dz=Q[1], lddy=24), dict(dz=Q[1], dy_type="f32"), dict(dz=Q[2], ldz=24),    # dz over dy or z
    dict(da=Q[6], da_type="f32"), dict(da=Q[6], ldda=32),                           # da over z_in
    dict(da=Q[3]), dict(da=Q[4]), dict(da=Q[5]), dict(db=Q[3]), dict(db=Q[4]), dict(dbias=Q[4]),
    dict(dz=Q[4]), dict(dz=Q[5]), dict(da=Q[8]), dict(da=Q[9], db_in=Q[9]),
])
def test_gemm_epilogue_grad_refuses_overlaps(kw):
    o = ovl()
    base = dict(dy=Q[1], z=Q[2], dz=Q[3], a=Q[4], b=Q[5], z_in=Q[6], da=Q[7], db=Q[8], dbias=Q[10], ws=Q[11],
                act="silu", act_in="relu")
    assert grad(o, **{**base, **kw})[0] == o.OVL_EINVAL


def test_moe_layer_refuses_overlaps():
    o = ovl()
    for out in Q[:3]:
        assert moe(o, x=Q[0], w1=Q[1], w2=Q[2], out=out, router=Q[4], topk=Q[5], gates=Q[6], ws=Q[7])[0] == o.OVL_EINVAL


def test_grad_clip_plan_takes_a_generator():
    """Host tensors are refused for where they lie, not for the iterable's kind."""
    import torch
    o = ovl()
    assert len(o.grad_clip_plan(iter([])).tensors[0]) == 0
    with pytest.raises(o.OvlError, match="current device"):
        o.grad_clip_plan(torch.zeros(4) for _ in range(2))
