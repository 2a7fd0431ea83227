"""Values of the feed-forward calls that bounds over random data do not see:
inputs of which one bit, one tail or one infinity decides the output."""

import numpy as np
import pytest

import oracle
from tests import ffn_util as fu
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


def ovl():
    from communication_overlap_amd import ovl as _o
    return _o


def set_values(w, fp8, *values):
    """Sets elements of a weight, given as (index, value), each 1, -1 or 0."""
    code = {1.0: 0x38, -1.0: 0xB8, 0.0: 0}
    for at, v in values:
        w[at] = code[v] if fp8 else v


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("w", ["bf16", "fp8"])
@pytest.mark.parametrize("T,E", [(1, 4), (12, 16), (60, 4)])
def test_h_keeps_the_bits_of_float32(T, E, w, out):
    """h of two columns that differ by their last terms alone, subtracted by the
    second weight: 1 + 2^-9 + 2^-b less 1 + 2^-9 is 2^-b, exact in both types."""
    from tests.test_gpu_moe_layer import Moe
    t = fu.torch()
    c = Moe(T, 64, 32, E, 1, w, out, "none", False, route=False, seed=1)
    c.x.zero_()
    c.w1.zero_()
    c.w2.zero_()
    if w == "fp8":
        c.s1.fill_(1.0)
        c.s2.fill_(1.0)
    c.gates.fill_(1.0)
    last = t.tensor([2.0 ** -(16 + i % 8) for i in range(T)], dtype=t.float64, device="cuda")  # 2^-b of a token
    c.x[:, 0] = 1.0
    c.x[:, 1] = 2.0 ** -9
    c.x[:, 2] = last.to(t.bfloat16)
    for e in range(E):
        at1 = (lambda k, n: (e, n, k)) if w == "fp8" else (lambda k, n: (e, k, n))  # noqa: E731
        set_values(c.w1, w == "fp8", *((at1(k, 7), 1.0) for k in range(3)), *((at1(k, 9), 1.0) for k in range(2)))
        set_values(c.w2, w == "fp8", (at1(7, 5), 1.0), (at1(9, 5), -1.0))
    c.run()
    want = t.zeros(T, 64, dtype=t.float64, device="cuda")
    want[:, 5] = last
    assert t.equal(c.out[:T].double(), want)


@pytest.mark.parametrize("T", [1, 5, 128])
@pytest.mark.parametrize("E,K", [(8, 2), (64, 8), (200, 4)])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("sigma", [1.0, 40.0])
def test_gates_are_rounded_once(T, E, K, norm, sigma):
    """A gate is the float64 softmax rounded to float32: half a step, and 2^-30
    of it for the float64 sums (a logit of size 300 is off by 2^-44 of it)."""
    from tests.test_gpu_moe_layer import Moe
    c = Moe(T, 256, 16, E, K, norm=norm, seed=T)
    c.router = fu.normal(7, 256, E, sigma=sigma / 16)
    c.run()
    ids, gates = oracle.route(fu.f64(c.x) @ fu.f64(c.router), K, norm)
    assert np.array_equal(c.ids.cpu().numpy(), ids)
    # below the normal range a float32 step is 2^-149
    fu.within(c.gates, gates, (fu.U + 2.0 ** -30) * gates + 2.0 ** -149, "gates")
