"""The product with bias, activation and residual, and its gradient, against
the float64 oracle: row counts around every tile and variant border, ragged
sizes, row strides with NaN between rows, each activation and type, in place,
captured, on another stream, and with workspaces that other calls used."""

import numpy as np
import pytest

import oracle
from tests import ffn_util as fu
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


def ovl():
    from communication_overlap_amd import ovl as _o
    return _o


KINDS = ("none", "relu", "gelu", "gelu_tanh", "silu")


class Linear:
    def __init__(self, m, n, k, act="none", out="bf16", bias=True, res="", z=False, pad=0, seed=0):
        o, t = ovl(), fu.torch()
        self.m, self.n, self.k, self.act, self.out_t = m, n, k, act, out
        ld = lambda w: w + pad if pad else 0  # noqa: E731
        self.desc = o.gemm_epilogue_desc(m, n, k, act, out, res or "bf16", ld(k), ld(n), ld(n), ld(n), ld(n))
        wide = lambda x: fu.strided(x, x.shape[1] + pad)[0] if pad else x  # noqa: E731
        self.a, self.b = wide(fu.normal(seed, m, k)), wide(fu.normal(seed + 1, k, n, sigma=0.25))
        self.bias = fu.normal(seed + 2, n, dtype="f32") if bias else None
        self.res = wide(fu.normal(seed + 3, m, n, dtype=res)) if res else None
        # outputs with a guard row and, strided, guarded row ends
        self.out_buf = t.full((m + 1, n + pad), 7.0, dtype=fu.ttype(out), device="cuda")
        self.z_buf = t.full((m + 1, n + pad), 7.0, dtype=t.bfloat16, device="cuda") if z else None
        self.out = self.out_buf[:m, :n]
        self.z = self.z_buf[:m, :n] if z else None
        self.ws = fu.workspace(o.gemm_epilogue_workspace_bytes(self.desc))

    def run(self, stream=None):
        say(f"  gemm_epilogue_run m={self.m} n={self.n} k={self.k} act={self.act} out={self.out_t}")
        ovl().gemm_epilogue_run(self.desc, self.a, self.b, self.bias, self.res, self.out, self.z, self.ws, stream)

    def check(self):
        a, b = fu.f64(self.a), fu.f64(self.b)
        out, z = oracle.gemm_epilogue(a, b, fu.f64(self.bias), fu.f64(self.res), self.act)
        zb = fu.sum_bound(a, b, self.k) + 2 * fu.U * (np.abs(z) + 1)
        act = oracle.act(z, self.act)
        ob = fu.SLOPE * zb + 16 * fu.U * (np.abs(act) + np.abs(z)) + fu.U * np.abs(out)
        fu.within(self.out, out, ob + fu.HALF[self.out_t] * (np.abs(out) + ob), "out")
        if self.z is not None:
            fu.within(self.z, z, zb + fu.HALF["bf16"] * (np.abs(z) + zb), "z")
        for buf in (self.out_buf, self.z_buf):
            if buf is not None:
                g = buf.float()
                assert bool((g[self.m:] == 7).all()) and bool((g[:, self.n:] == 7).all()), "wrote past the output"


# The row counts stand on both sides of each variant's border (few rows: 16
# and 32; 128- and 256-row tiles), the widths and lengths off every multiple.
@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 31, 32, 33, 64, 129, 257])
@pytest.mark.parametrize("n,k", [(8, 8), (72, 40), (200, 264), (264, 1000)])
def test_rows_and_ragged_sizes(m, n, k):
    c = Linear(m, n, k, "silu", "f32", res="bf16", z=True, seed=m)
    c.run()
    c.check()


@pytest.mark.parametrize("act", KINDS)
@pytest.mark.parametrize("out,res", [("bf16", ""), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("m", [5, 140])
def test_activations_and_types(act, out, res, m):
    c = Linear(m, 136, 200, act, out, bias=res != "f32", res=res, z=res == "", seed=11)
    c.run()
    c.check()


@pytest.mark.parametrize("m,n,k", [(3, 72, 104), (30, 264, 72), (70, 136, 72), (300, 520, 200)])
def test_strided_rows_never_touch_the_gaps(m, n, k):
    c = Linear(m, n, k, "gelu_tanh", "bf16", res="f32", z=True, pad=24, seed=5)
    c.run()
    c.check()


@pytest.mark.parametrize("m,n,k", [(1, 7168, 2048), (20, 4096, 1024), (128, 1024, 4096), (2056, 4104, 136)])
def test_long_split_and_large(m, n, k):
    c = Linear(m, n, k, "gelu", "f32", z=True, seed=9)
    c.run()
    c.check()


@pytest.mark.parametrize("m", [4, 200])
def test_residual_in_place(m):
    c = Linear(m, 72, 64, "relu", "bf16", res="bf16", seed=3)
    want = Linear(m, 72, 64, "relu", "bf16", res="bf16", seed=3)
    want.run()
    c.out.copy_(c.res)
    ovl().gemm_epilogue_run(c.desc, c.a, c.b, c.bias, c.out, c.out, None, c.ws)
    assert fu.torch().equal(c.out, want.out)


@pytest.mark.parametrize("m", [6, 150])
def test_not_finite_values_stay_in_their_rows_and_columns(m):
    t = fu.torch()
    c = Linear(m, 80, 72, "none", "f32", seed=4)
    c.a[2, 5] = float("nan")
    c.b[7, 9] = float("inf")
    c.run()
    ok = t.isfinite(c.out)
    assert bool(t.isnan(c.out[2]).all())
    assert not bool(ok[:, 9].any())
    ok[2] = True
    ok[:, 9] = True
    assert bool(ok.all())


@pytest.mark.parametrize("m,n,k", [(1, 4096, 4096), (128, 1024, 4096), (1000, 2056, 520)])
def test_same_bits_every_time(m, n, k):
    t = fu.torch()
    c = Linear(m, n, k, "silu", "f32", z=True, seed=6)
    c.run()
    first = c.out.clone()
    for _ in range(3):
        c.out.zero_()
        c.run()
        assert t.equal(c.out, first)


def test_output_past_four_gib():
    """Rows whose output lies past 32-bit byte offsets (m = 262147 rows of 4104 float32)."""
    t, o = fu.torch(), ovl()
    m, n, k = 262147, 4104, 8
    a = t.randint(-4, 5, (m, k), device="cuda").to(t.bfloat16)
    b = t.randint(-4, 5, (k, n), device="cuda").to(t.bfloat16)
    out = t.empty(m, n, device="cuda")
    d = o.gemm_epilogue_desc(m, n, k, "relu", "f32")
    say("  gemm_epilogue_run with 4.3 GB of output")
    o.gemm_epilogue_run(d, a, b, None, None, out, None, fu.workspace(o.gemm_epilogue_workspace_bytes(d)))
    for r in range(0, m, 65536):  # small integers: exact
        assert t.equal(out[r:r + 65536], t.relu(a[r:r + 65536].float() @ b.float()))


@pytest.mark.parametrize("m", [3, 100, 300])
def test_another_stream_and_capture(m):
    """A captured call replayed between eager calls of another size on the same workspace."""
    t, o = fu.torch(), ovl()
    c = Linear(m, 264, 1000, "silu", "f32", seed=8)
    e = Linear(m + 1, 520, 2048, "none", "f32", seed=20)
    ws = fu.workspace(max(c.ws.numel(), e.ws.numel()))
    c.ws = e.ws = ws
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(s):
        c.run()
    s.synchronize()
    c.check()
    want = c.out.clone()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        c.run()
    for _ in range(3):
        c.out.zero_()
        e.run()
        g.replay()
        t.cuda.synchronize()
        assert t.equal(c.out, want)
        e.check()


# ------------------------------------------------------------------ gradient

class Grad:
    def __init__(self, m, n, k, act_in="none", da="bf16", db="f32", acc=False, pad=0, act="none", dy="bf16", seed=0):
        o, t = ovl(), fu.torch()
        self.m, self.n, self.k, self.act, self.act_in = m, n, k, act, act_in
        self.da_t, self.db_t = da, db
        ld = lambda w: w + pad if pad else 0  # noqa: E731
        self.desc = o.gemm_epilogue_grad_desc(m, n, k, act, act_in, dy, da, db, ld(k), ld(n), ld(n), ld(n), ld(n),
                                              ld(k), ld(k), ld(n))
        wide = lambda x: fu.strided(x, x.shape[1] + pad)[0] if pad else x  # noqa: E731
        self.a, self.b = wide(fu.normal(seed, m, k)), wide(fu.normal(seed + 1, k, n, sigma=0.25))
        self.dz = wide(fu.normal(seed + 2, m, n))
        self.z_in = wide(fu.normal(seed + 3, m, k, sigma=2.0)) if act_in != "none" else None
        self.dy = wide(fu.normal(seed + 6, m, n, dtype=dy)) if act != "none" else None
        self.z = wide(fu.normal(seed + 7, m, n, sigma=2.0)) if act != "none" else None
        self.db_in = wide(fu.normal(seed + 4, k, n, dtype=db)) if acc else None
        self.dbias_in = fu.normal(seed + 5, n, dtype="f32") if acc else None
        self.da_buf = t.full((m + 1, k + pad), 7.0, dtype=fu.ttype(da), device="cuda")
        self.db_buf = t.full((k + 1, n + pad), 7.0, dtype=fu.ttype(db), device="cuda")
        self.da, self.db = self.da_buf[:m, :k], self.db_buf[:k, :n]
        self.dbias = t.full((n,), 7.0, device="cuda")
        self.ws = fu.workspace(o.gemm_epilogue_grad_workspace_bytes(self.desc))

    def run(self, da=True, db=True, dbias=True, stream=None):
        say(f"  gemm_epilogue_grad_run m={self.m} n={self.n} k={self.k} act={self.act} act_in={self.act_in}")
        ovl().gemm_epilogue_grad_run(self.desc, self.dz, self.a, self.b, self.z_in if da else None,
                                     self.da if da else None, self.db if db else None, self.db_in if db else None,
                                     self.dbias if dbias else None, self.dbias_in if dbias else None, self.ws,
                                     self.dy, self.z, stream)

    def check(self):
        dz, a, b = fu.f64(self.dz), fu.f64(self.a), fu.f64(self.b)
        if self.act != "none":
            dy, z = fu.f64(self.dy), fu.f64(self.z)
            want = dy * oracle.act_grad(z, self.act)
            fu.within(self.dz, want, (fu.HALF["bf16"] + 2 * fu.U) * np.abs(want)
                      + 32 * fu.U * np.abs(dy) * (1 + np.abs(z)), "dz")
        da, db, dbias = oracle.gemm_epilogue_grad(dz, a, b, fu.f64(self.z_in), self.act_in, fu.f64(self.db_in),
                                                  fu.f64(self.dbias_in))
        sb = fu.sum_bound(dz, b.T, self.n)
        if self.z_in is not None:
            z = fu.f64(self.z_in)
            sb = fu.SLOPE * sb + 32 * fu.U * np.abs(dz @ b.T) * (1 + np.abs(z)) + fu.U * np.abs(da)
        fu.within(self.da, da, sb + fu.HALF[self.da_t] * (np.abs(da) + sb), "da")
        sb = fu.sum_bound(a.T, dz, self.m) + fu.U * np.abs(db)
        fu.within(self.db, db, sb + fu.HALF[self.db_t] * (np.abs(db) + sb), "db")
        sb = (self.m + 2) * fu.U * np.abs(dz).sum(axis=0) + 2 * fu.U * np.abs(dbias)
        fu.within(self.dbias, dbias, sb, "dbias")
        for buf, rows, cols in ((self.da_buf, self.m, self.k), (self.db_buf, self.k, self.n)):
            g = buf.float()
            assert bool((g[rows:] == 7).all()) and bool((g[:, cols:] == 7).all()), "wrote past the output"


@pytest.mark.parametrize("m", [0, 1, 7, 64, 65, 200])
@pytest.mark.parametrize("n,k", [(8, 8), (72, 136), (264, 40)])
def test_grad_rows_and_ragged_sizes(m, n, k):
    c = Grad(m, n, k, acc=True, seed=m)
    c.run()
    c.check()


@pytest.mark.parametrize("act_in", KINDS[1:])
@pytest.mark.parametrize("da,db", [("bf16", "bf16"), ("f32", "f32")])
def test_grad_activation_before(act_in, da, db):
    c = Grad(140, 136, 200, act_in, da, db, acc=da == "f32", seed=2)
    c.run()
    c.check()


@pytest.mark.parametrize("act", KINDS[1:])
@pytest.mark.parametrize("dy", ["bf16", "f32"])
def test_grad_own_activation(act, dy):
    c = Grad(70, 72, 104, "relu", act=act, dy=dy, seed=3)
    c.dz.fill_(float("nan"))
    c.run()
    c.check()


@pytest.mark.parametrize("m,n,k", [(70, 136, 72), (600, 264, 520)])
def test_grad_strided_rows_never_touch_the_gaps(m, n, k):
    c = Grad(m, n, k, "silu", acc=True, pad=24, act="gelu", seed=5)
    c.run()
    c.check()


@pytest.mark.parametrize("m,n,k", [(128, 256, 256), (20000, 72, 40), (2056, 4104, 1032), (4096, 64, 64)])
def test_grad_split_and_large(m, n, k):
    c = Grad(m, n, k, "gelu_tanh", seed=7)
    c.run()
    c.check()


@pytest.mark.parametrize("da,db,dbias", [(True, False, False), (False, True, False), (False, False, True),
                                         (True, False, True), (False, False, False)])
def test_grad_parts_alone_are_the_whole_call_s(da, db, dbias):
    t = fu.torch()
    c, w = Grad(130, 200, 72, "silu", seed=8), Grad(130, 200, 72, "silu", seed=8)
    w.run()
    c.run(da, db, dbias)
    for on, got, want in ((da, c.da, w.da), (db, c.db, w.db), (dbias, c.dbias, w.dbias)):
        assert t.equal(got, want) if on else bool((got == 7).all())


def test_grad_accumulates_in_place():
    t = fu.torch()
    c = Grad(100, 72, 64, acc=True, seed=9)
    c.run()
    d = Grad(100, 72, 64, acc=True, seed=9)
    d.db.copy_(d.db_in)
    d.dbias.copy_(d.dbias_in)
    d.db_in, d.dbias_in = d.db, d.dbias
    d.run()
    assert t.equal(c.db, d.db) and t.equal(c.dbias, d.dbias)


def test_grad_da_over_z_in_and_dz_over_dy():
    t = fu.torch()
    w, c = (Grad(90, 72, 64, "silu", act="relu", seed=10) for _ in range(2))
    w.run()
    c.dz, c.da = c.dy, c.z_in
    c.run()
    assert t.equal(c.dz, w.dz) and t.equal(c.da, w.da) and t.equal(c.db, w.db)


def test_grad_derivatives_far_out_are_zero_or_one():
    """Pre-activations up to infinity: no 0 * inf on the way, NaN stays NaN."""
    t = fu.torch()
    for act in KINDS[1:]:
        c = Grad(8, 8, 8, act=act, seed=1)
        c.dy.fill_(1.0)
        c.z[0, :7] = t.tensor([3e38, -3e38, float("inf"), float("-inf"), 40.0, -40.0, float("nan")], device="cuda")
        c.run(False, False, False)
        assert c.dz[0, :6].tolist() == [1, 0, 1, 0, 1, 0] and bool(c.dz[0, 6].isnan()), act


@pytest.mark.parametrize("m,n,k", [(128, 256, 256), (3000, 264, 136)])
def test_grad_same_bits_and_capture(m, n, k):
    t = fu.torch()
    c = Grad(m, n, k, "silu", act="gelu", seed=12)
    c.run()
    c.check()
    first = [x.clone() for x in (c.dz, c.da, c.db, c.dbias)]
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g, stream=s):
        c.run()
    for _ in range(3):
        for x in (c.dz, c.da, c.db, c.dbias):
            x.zero_()
        g.replay()
        t.cuda.synchronize()
        for x, y in zip((c.dz, c.da, c.db, c.dbias), first):
            assert t.equal(x, y)


@pytest.mark.parametrize("act", KINDS)
def test_grad_against_differences(act):
    """The whole layer's gradient along random directions against central
    differences of the float64 loss sum(c * out): the difference is off by
    h^2 / 6 of a third derivative and 2^-53 / h of the loss; the kernel by its
    dz, rounded to bf16 (2^-8 of each term)."""
    r = np.random.RandomState(5)
    m, n, k = 9, 24, 16
    o, t = ovl(), fu.torch()
    a, b, bias = fu.normal(1, m, k), fu.normal(2, k, n, sigma=0.3), fu.normal(3, n, dtype="f32")
    out, z = t.empty(m, n, device="cuda"), t.empty(m, n, dtype=t.bfloat16, device="cuda")
    fd = o.gemm_epilogue_desc(m, n, k, act, "f32")
    o.gemm_epilogue_run(fd, a, b, bias, None, out, z, fu.workspace(o.gemm_epilogue_workspace_bytes(fd)))
    cc = fu.normal(4, m, n, dtype="f32")
    gd = o.gemm_epilogue_grad_desc(m, n, k, act, "none", "f32", "f32", "f32")
    da, db, dbias = t.empty(m, k, device="cuda"), t.empty(k, n, device="cuda"), t.empty(n, device="cuda")
    dz = cc.bfloat16() if act == "none" else t.empty(m, n, dtype=t.bfloat16, device="cuda")
    o.gemm_epilogue_grad_run(gd, dz, a, b, None, da, db, None, dbias, None,
                             fu.workspace(o.gemm_epilogue_grad_workspace_bytes(gd)),
                             None if act == "none" else cc, None if act == "none" else z)
    x = [fu.f64(v) for v in (a, b, bias)]
    c = fu.f64(cc)
    h = 1e-5

    def loss(args):
        return float((c * oracle.gemm_epilogue(*args, None, act)[0]).sum())

    # the kernel reads z rounded to bf16: its derivative moves by at most 2^-8 |z| times the second derivative (< 1.2)
    zf = fu.f64(z)
    slack = (2.0 ** -8) * np.abs(c) * fu.SLOPE + (2.0 ** -8) * np.abs(c) * np.abs(zf) * 1.2
    if act == "relu":
        assert np.abs(oracle.gemm_epilogue(*x, None, act)[1]).min() > 1e-3  # no difference steps over the corner
    for at, g in ((0, da), (1, db), (2, dbias)):
        d = r.standard_normal(x[at].shape)
        up, dn = list(x), list(x)
        up[at], dn[at] = x[at] + h * d, x[at] - h * d
        step = np.abs(x[0]) @ np.abs(d) if at == 1 else (np.abs(d) @ np.abs(x[1]) if at == 0 else np.abs(d)[None, :])
        assert abs((loss(up) - loss(dn)) / (2 * h) - float((fu.f64(g) * d).sum())) <= float((slack * step).sum()) + 1e-4


def test_grad_dz_over_z():
    t = fu.torch()
    w, c = (Grad(90, 72, 64, "silu", act="relu", seed=12) for _ in range(2))
    w.run()
    c.dz = c.z
    c.run()
    assert t.equal(c.dz, w.dz) and t.equal(c.da, w.da) and t.equal(c.db, w.db)
