"""Values of the feed-forward calls that bounds over random data do not see:
inputs of which one bit, one tail or one infinity decides the output."""

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


@pytest.mark.parametrize("w", ["bf16"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 9])
def test_an_infinite_second_weight_gives_what_the_product_gives(T, out, w):
    """h times an infinite weight is the infinity of h's sign, whether h has one
    significant bit or 24; zero times it is NaN, and so are two opposite ones."""
    from tests.test_gpu_moe_layer import Moe
    t = fu.torch()
    inf = float("inf")
    c = Moe(T, 64, 32, 4, 1, w, out, "none", False, route=False, seed=1)
    c.x.zero_()
    c.w1.zero_()
    c.w2.zero_()
    c.gates.fill_(0.5)
    # h of columns 0..5: 1, -3 * 2^-5, 1 + 2^-9, -(1 + 2^-9 + 2^-20), 0, the largest bf16
    c.x[:, :3] = t.tensor([1.0, 2.0 ** -9, 2.0 ** -20], device="cuda")
    big = float(t.finfo(t.bfloat16).max)
    for e in range(4):
        c.w1[e, :3, :6] = t.tensor([[1.0, -3 / 32, 1.0, -1.0, 0.0, big], [0, 0, 1.0, -1.0, 0, 0], [0, 0, 0, -1.0, 0, 0]])
        for i in range(6):
            c.w2[e, i, i] = inf
            c.w2[e, i, 8 + i] = -inf
        c.w2[e, 0, 16], c.w2[e, 3, 16] = inf, inf   # opposite infinities
        c.w2[e, 0, 17], c.w2[e, 1, 17] = inf, 1.0   # beside a finite term
        c.w2[e, 2, 18] = 2.0                        # no infinity
    c.run()
    got = c.out[:T].float().cpu()
    nan = float("nan")
    want = t.zeros(64)
    want[:6] = t.tensor([inf, -inf, inf, -inf, nan, inf])
    want[8:14] = t.tensor([-inf, inf, -inf, inf, nan, -inf])
    want[16], want[17], want[18] = nan, inf, 1.0 + 2.0 ** -9
    want = want.to(fu.ttype(out)).float()
    # zero weights of finite h add nothing: every other column is exactly zero
    for i in range(T):
        assert t.equal(got[i].isnan(), want.isnan())
        assert t.equal(got[i].nan_to_num(7.0, inf, -inf), want.nan_to_num(7.0, inf, -inf))


def test_an_infinite_h_stays_one():
    """An infinite activation times finite weights: infinities, NaN at zero weights."""
    from tests.test_gpu_moe_layer import Moe
    t = fu.torch()
    c = Moe(2, 64, 32, 2, 1, "bf16", "f32", "none", False, route=False, seed=1)
    c.x.zero_()
    c.x[:, 0] = 1.0
    c.w1.zero_()
    c.w1[:, 0, 4] = float("inf")
    c.w2.fill_(1.0)
    c.w2[:, 4, 1] = -2.0
    c.w2[:, 4, 2] = 0.0
    c.gates.fill_(1.0)
    c.run()
    assert bool((c.out[:2, 0] == float("inf")).all()) and bool((c.out[:2, 1] == -float("inf")).all())
    assert bool(c.out[:2, 2].isnan().all()) and bool((c.out[:2, 3:] == float("inf")).all())


# ------------------------------------------------------------------ activations' tails

def activation(act, z):
    """act at the float32 values z: a product of zeros with z as its bias."""
    o, t = ovl(), fu.torch()
    n = -(-len(z) // 8) * 8
    bias = t.zeros(n, device="cuda")
    bias[:len(z)] = t.from_numpy(z).cuda()
    a, b = (t.zeros(*s, dtype=t.bfloat16, device="cuda") for s in ((3, 8), (8, n)))
    out = t.empty(3, n, device="cuda")
    d = o.gemm_epilogue_desc(3, n, 8, act, "f32")
    say(f"  gemm_epilogue_run of {n} pre-activations, {act}")
    o.gemm_epilogue_run(d, a, b, bias, None, out, None, fu.workspace(o.gemm_epilogue_workspace_bytes(d)))
    assert t.equal(out[0], out[2])
    return fu.f64(out[0, :len(z)])


def derivative(act, z):
    """act' at the bf16 values z: the factor of a product of ones."""
    o, t = ovl(), fu.torch()
    k = -(-len(z) // 8) * 8
    z_in = t.zeros(2, k, dtype=t.bfloat16, device="cuda")
    z_in[:, :len(z)] = t.from_numpy(z).cuda()
    dz, b = (t.zeros(r, 8, dtype=t.bfloat16, device="cuda") for r in (2, k))
    dz[:, 0], b[:, 0] = 1.0, 1.0
    da = t.empty(2, k, device="cuda")
    d = o.gemm_epilogue_grad_desc(2, 8, k, "none", act, "bf16", "f32", "f32")
    say(f"  gemm_epilogue_grad_run of {k} pre-activations, {act}")
    o.gemm_epilogue_grad_run(d, dz, None, b, z_in, da, None, None, None, None,
                             fu.workspace(o.gemm_epilogue_grad_workspace_bytes(d)))
    assert t.equal(da[0], da[1])
    return fu.f64(da[0, :len(z)])


def bf16_points(lo, hi):
    """Every bf16 value of [lo, hi] from 2^-20 up in size."""
    v = (np.arange(1 << 16, dtype=np.uint32) << 16).view(np.float32)
    return np.sort(v[np.isfinite(v) & (v >= lo) & (v <= hi) & (np.abs(v) >= 2.0 ** -20)])


def closest(got, want, bound, z):
    bad = ~(np.abs(got - want) <= bound)
    i = int(np.argmax(bad))
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} off; at z = {z[i]}: {got[i]} against {want[i]}, bound {bound[i]}"


def test_gelu_keeps_its_tail():
    """0.5 z erfc(-z / sqrt 2), relative to itself down to 1e-35.  By way of the
    error function's argument, off by 2 U of itself (U = 2^-24), erfc(x) moves
    by 2 x^2 + 1 = z^2 + 1 times as much of itself, and by way of exp(-z^2 / 2)
    by 1.5 z^2 U, three roundings of the exponent; 34 U are left for the
    polynomial or erfc's own steps, the exponential and the products."""
    z = np.linspace(-12.4, 6, 6001).astype(np.float32)
    want = np.array([0.5 * v * math.erfc(-v / math.sqrt(2.0)) for v in z.astype(np.float64)])
    closest(activation("gelu", z), want, (2 * (z.astype(np.float64) ** 2 + 1) + 34) * fu.U * np.abs(want), z)


def test_gelu_derivative_keeps_its_tail():
    """cdf + z pdf: the cdf as above; in the pdf the exponent z^2 / 2 is off by 3 U
    of itself (a constant and two products), the exponential by 2 U more and its
    two factors by 3 U; one sum."""
    z = bf16_points(-12.4, 6.0)
    v = z.astype(np.float64)
    cdf = np.array([0.5 * math.erfc(-x / math.sqrt(2.0)) for x in v])
    pdf = np.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    bound = ((2 * (v * v + 1) + 34) * cdf + (1.5 * v * v + 6) * np.abs(v) * pdf) * fu.U
    closest(derivative("gelu", z), cdf + v * pdf, bound * (1 + 2.0 ** -10) + fu.U * np.abs(cdf + v * pdf), z)


def sigmoid(v):
    """To a few steps of itself on either side: exp(-|v|) is exact to 2^-53 of itself."""
    e = np.exp(-np.abs(v))
    return np.where(v > 0, 1.0, e) / (1.0 + e)


# sigma(x)'s relative error: the exponent |x| log2(e) / 2 is off by 2 U of itself
# (constant and product) and taken twice, 2 |x| U; two exponentials 4 U, the
# reciprocal 2 U, its sum 1 U and three products 3 U.  Results below float32's
# normal range are rounded to multiples of 2^-149, twice at most.
def sigma_bound(x):
    return (2 * np.abs(x) + 12) * fu.U


LEAST = 2.0 ** -148


def test_silu_and_its_derivative_keep_their_tails():
    """z sigma(z) down to where it leaves float32, near z = -106, and its
    derivative s + z s (1 - s): the first term is off by sigma's error, the
    second, h r squared, by no more of itself, and their sum by U."""
    z = np.linspace(-120, 20, 14001).astype(np.float32)
    v = z.astype(np.float64)
    want = v * sigmoid(v)
    closest(activation("silu", z), want, sigma_bound(v) * np.abs(want) + LEAST, z)
    z = bf16_points(-300.0, 300.0)
    v = z.astype(np.float64)
    s, t = sigmoid(v), sigmoid(-v)
    want = s * (1 + v * t)
    bound = s * (1 + np.abs(v) * t) * sigma_bound(v) + fu.U * np.abs(want) + LEAST
    got = derivative("silu", z)
    closest(got, want, bound, z)
    assert np.abs(got[(z < -80) & (z > -100)]).min() > 0


def test_gelu_tanh_and_its_derivative_keep_their_tails():
    """z sigma(w), w = 2 sqrt(2 / pi) (z + c z^3), off by 6 U of itself (two
    constants, four products and a sum, of terms of one sign)."""
    r = 2 * math.sqrt(2 / math.pi)
    z = np.linspace(-10.5, 6, 6001).astype(np.float32)
    v = z.astype(np.float64)
    w = r * (v + 0.044715 * v ** 3)
    want = v * sigmoid(w)
    err = sigma_bound(w) + 7 * np.abs(w) * fu.U
    closest(activation("gelu_tanh", z), want, err * np.abs(want) + LEAST, z)
    z = bf16_points(-40.0, 40.0)
    v = z.astype(np.float64)
    w, d = r * (v + 0.044715 * v ** 3), r * (1 + 3 * 0.044715 * v * v)
    s, t = sigmoid(w), sigmoid(-w)
    want = s * (1 + v * t * d)
    err = sigma_bound(w) + 7 * np.abs(w) * fu.U
    bound = s * (err + np.abs(v) * t * d * (err + 8 * fu.U)) + fu.U * np.abs(want) + LEAST
    closest(derivative("gelu_tanh", z), want, bound, z)


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dy", ["bf16", "f32"])
def test_own_derivative_far_out(act, dy):
    """dz at pre-activations up to infinity: no 0 * inf on the way, NaN stays
    NaN, and at -40 SiLU's derivative is exp(-40) (1 - 40), a bf16 number."""
    t, o = fu.torch(), ovl()
    z = t.tensor([[3e38, -3e38, math.inf, -math.inf, 40.0, -40.0, math.nan, -300.0]] * 8, device="cuda").bfloat16()
    dz, ones = t.empty_like(z), t.ones(8, 8, device="cuda", dtype=fu.ttype(dy))
    d = o.gemm_epilogue_grad_desc(8, 8, 8, act, "none", dy)
    o.gemm_epilogue_grad_run(d, dz, None, None, None, None, None, None, None, None,
                             fu.workspace(o.gemm_epilogue_grad_workspace_bytes(d)), ones, z)
    got = fu.f64(dz[3])
    assert got[:5].tolist() == [1, 0, 1, 0, 1] and math.isnan(got[6]) and got[7] == 0
    want = math.exp(-40.0) * (1 - 40.0) if act == "silu" else 0.0
    assert abs(got[5] - want) <= (fu.HALF["bf16"] + 200 * fu.U) * abs(want)
