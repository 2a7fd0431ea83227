"""The feed-forward calls' binding on the CPU: buffers of another type than the
call's are refused, whatever their element size."""

import pytest

P = 4096  # an aligned address that nothing dereferences


def ovl():
    from communication_overlap_amd import ovl as _o
    return _o


def tensor(dtype, *shape):
    import torch
    return torch.empty(shape, dtype=getattr(torch, dtype))


def linear(o, **kw):
    d = o.gemm_epilogue_desc(8, 16, 24, out_type="bf16", res_type="f32")
    args = {**dict(a=P, b=P, bias=P, residual=P, out=P, z=P, workspace=P), **kw}
    return o.gemm_epilogue_run(d, stream=0, **args)


def grad(o, **kw):
    d = o.gemm_epilogue_grad_desc(8, 16, 24, "silu", "relu", "f32", "bf16", "f32")
    names = ("dz", "a", "b", "z_in", "da", "db", "db_in", "dbias", "dbias_in", "workspace", "dy", "z")
    return o.gemm_epilogue_grad_run(d, stream=0, **{**dict.fromkeys(names, P), **kw})


def moe(o, w_type="fp8", **kw):
    d = o.moe_layer_desc(4, 64, 32, 8, 2, w_type=w_type, out_type="f32")
    names = ("x", "router", "topk_idx", "gates", "w1", "w1_scale", "w2", "w2_scale", "out", "workspace")
    return o.moe_layer_run(d, stream=0, **{**dict.fromkeys(names, P), **kw})


HALVES, WORDS, BYTES = ("float16",), ("int32", "bfloat16"), ("int8", "float8_e5m2", "float8_e4m3fnuz")


@pytest.mark.parametrize("call,name,shape,wrong,right", [
    (linear, "a", (8, 24), HALVES, ("bfloat16", "int16")), (linear, "b", (24, 16), HALVES, ("bfloat16", "int16")),
    (linear, "bias", (16,), WORDS, ("float32",)), (linear, "residual", (8, 16), WORDS, ("float32",)),
    (linear, "out", (8, 16), HALVES, ("bfloat16",)), (linear, "z", (8, 16), HALVES, ("bfloat16",)),
    (linear, "workspace", (1 << 20,), ("float32", "int16"), ("uint8", "int8", "bool")),
    (grad, "dz", (8, 16), HALVES, ("bfloat16",)), (grad, "a", (8, 24), HALVES, ("bfloat16",)),
    (grad, "b", (24, 16), HALVES, ("bfloat16",)), (grad, "z_in", (8, 24), HALVES, ("bfloat16",)),
    (grad, "da", (8, 24), HALVES, ("bfloat16",)), (grad, "db", (24, 16), WORDS, ("float32",)),
    (grad, "db_in", (24, 16), WORDS, ("float32",)), (grad, "dbias", (16,), WORDS, ("float32",)),
    (grad, "dbias_in", (16,), WORDS, ("float32",)), (grad, "dy", (8, 16), WORDS, ("float32",)),
    (grad, "z", (8, 16), HALVES, ("bfloat16",)),
    (moe, "x", (4, 64), HALVES, ("bfloat16",)), (moe, "router", (64, 8), HALVES, ("bfloat16",)),
    (moe, "topk_idx", (4, 2), ("float32", "int64"), ("int32",)), (moe, "gates", (4, 2), WORDS, ("float32",)),
    (moe, "w1", (8, 64, 64), BYTES, ("uint8", "float8_e4m3fn")), (moe, "w2", (8, 64, 32), BYTES, ("uint8", "float8_e4m3fn")),
    (moe, "w1_scale", (8, 64), WORDS, ("float32",)), (moe, "w2_scale", (8, 64), WORDS, ("float32",)),
    (moe, "out", (4, 64), WORDS, ("float32",)),
])
def test_binding_refuses_other_types(call, name, shape, wrong, right):
    """The right types pass this check: they are host tensors here, and refused as such."""
    o = ovl()
    for dtypes, why in ((wrong, "elements of type"), (right, "current device")):
        for dtype in dtypes:
            with pytest.raises(o.OvlError, match=why) as e:
                call(o, **{name: tensor(dtype, *shape)})
            assert e.value.status == o.OVL_EINVAL and name in str(e.value)


def test_binding_refuses_bf16_weights_of_another_type():
    o = ovl()
    for name, shape in (("w1", (8, 64, 64)), ("w2", (8, 32, 64))):
        with pytest.raises(o.OvlError, match="elements of type"):
            moe(o, "bf16", w1_scale=None, w2_scale=None, **{name: tensor("float16", *shape)})


def test_binding_refuses_a_norm_of_another_type():
    o = ovl()
    with pytest.raises(o.OvlError, match="elements of type"):
        o.grad_norm_clip_run(o.grad_clip_plan([]), 1.0, tensor("int32", 1), P, stream=0)
