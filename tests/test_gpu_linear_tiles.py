"""The products' 128 x 128 tiles (over 512 tiles of 64 x 128 and under 128 of
256 x 256), whole and with K cut, 256 x 256 tiles with K cut, and the row
stream over more column tiles than compute units."""

import pytest

from tests import ffn_util as fu
from tests.test_gpu_linear import Grad, Linear, ovl

pytestmark = pytest.mark.gpu


def ceil(a, b):
    return -(-a // b)


def tiles(mn, tm, tn):
    return sum(ceil(m, tm) * ceil(n, tn) for m, n in mn)


def tier(*mnk):
    """(tile rows, whether K is cut) for a launch's products."""
    mn = [x[:2] for x in mnk]
    if tiles(mn, 256, 256) >= 128:
        edge, slots = 256, 256
    elif tiles(mn, 64, 128) <= 512:
        return 64, None  # cut by a model of costs
    else:
        edge, slots = 128, 512
    steps = [ceil(k, 64) for _, _, k in mnk]
    work = sum(tiles([x], edge, edge) * s for x, s in zip(mn, steps))
    share = max(8, ceil(work, slots), ceil(max(steps), 16))
    return edge, 2 * max(steps) > 3 * share


@pytest.mark.parametrize("m,n,k,where", [(2056, 2184, 136, (128, False)), (2056, 2184, 2056, (128, True)),
                                         (1416, 3080, 72, (128, False)), (2056, 4104, 4104, (256, True))])
@pytest.mark.parametrize("pad", [0, 24])
def test_forward(m, n, k, where, pad):
    assert tier((m, n, k)) == where
    c = Linear(m, n, k, "gelu", "f32" if pad else "bf16", res="bf16" if pad else "f32", z=True, pad=pad, seed=3)
    c.run()
    c.check()


GRADS = [(520, 520, 4104, (128, False)), (1304, 2568, 1032, (128, True)), (2056, 4104, 1032, (256, True))]


@pytest.mark.parametrize("m,n,k,where", GRADS)
@pytest.mark.parametrize("pad", [0, 24])
def test_grad(m, n, k, where, pad):
    assert tier((k, n, m), (m, k, n)) == where
    c = Grad(m, n, k, "silu", "f32" if pad else "bf16", "bf16" if pad else "f32", acc=True, pad=pad,
             act="gelu_tanh" if pad else "none", seed=4)
    c.run()
    c.check()


@pytest.mark.parametrize("m,n,k,where", GRADS[:2])
def test_grad_parts_alone(m, n, k, where):
    t = fu.torch()
    w, c = (Grad(m, n, k, "relu", seed=5) for _ in range(2))
    w.run()
    for on in range(3):
        c.run(on == 0, on == 1, on == 2)
    assert t.equal(c.da, w.da) and t.equal(c.db, w.db) and t.equal(c.dbias, w.dbias)


@pytest.mark.parametrize("make", [lambda: Linear(2056, 2184, 136, "silu", "f32", z=True, seed=6),
                                  lambda: Linear(2056, 2184, 2056, "silu", "f32", z=True, seed=6),
                                  lambda: Linear(1416, 3080, 72, "relu", "bf16", res="bf16", seed=6),
                                  lambda: Grad(520, 520, 4104, "silu", acc=True, seed=7),
                                  lambda: Grad(1304, 2568, 1032, "silu", act="gelu", seed=7)])
def test_same_bits_captured_and_replayed(make):
    """Replayed between eager calls of another size on the same workspace."""
    t, o = fu.torch(), ovl()
    c, e = make(), Linear(300, 520, 4096, seed=8)
    ws = fu.workspace(max(c.ws.numel(), e.ws.numel()))
    c.ws = e.ws = ws
    outs = [x for x in (getattr(c, n, None) for n in ("out", "z", "dz", "da", "db", "dbias")) if t.is_tensor(x)]
    if isinstance(c, Grad) and c.act == "none":
        outs = [x for x in outs if x is not c.dz]
    if isinstance(c, Grad) and c.act != "none":
        outs = [x for x in outs if x is not c.z]
    c.run()
    t.cuda.synchronize()
    want = [x.clone() for x in outs]
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        c.run()
    for _ in range(3):
        for x in outs:
            x.zero_()
        e.run()
        g.replay()
        t.cuda.synchronize()
        assert all(t.equal(x, y) for x, y in zip(outs, want))
    c.check()


@pytest.mark.parametrize("m", [1, 16, 20, 32])
@pytest.mark.parametrize("n,k", [(33032, 264), (50304, 72)])
def test_more_column_tiles_than_compute_units(m, n, k):
    c = Linear(m, n, k, "none", "f32", z=m == 20, res="bf16" if m == 32 else "", seed=m)
    c.run()
    c.check()
