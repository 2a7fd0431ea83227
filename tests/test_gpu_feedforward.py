"""The feed-forward calls used together, as a training step and as a decoding
step use them, beside the framework's own reduction and quantizer."""

import numpy as np
import pytest

import oracle
from tests import ffn_util as fu
from tests.gpu_util import say, zeros_bytes

pytestmark = pytest.mark.gpu


def ovl():
    from communication_overlap_amd import ovl as _o
    return _o


def test_training_step_of_a_block_on_two_ranks():
    """x -> act(x W1 + b1) W2 + b2 + x on two emulated ranks' batches: forward,
    backward, ring all-reduce of the weight gradients, clipping; against
    float64 with the bf16 roundings of the stored tensors (h, z and dz) put in
    where the calls put them."""
    o, t = ovl(), fu.torch()
    m, h, f = 200, 136, 264
    w1, b1 = fu.normal(1, h, f, sigma=0.1), fu.normal(2, f, dtype="f32")
    w2, b2 = fu.normal(3, f, h, sigma=0.1), fu.normal(4, h, dtype="f32")
    sizes = [h * f, f, f * h, h]
    total = -(-sum(sizes) // 2) * 2
    buckets, want = [], np.zeros(sum(sizes))
    up = o.gemm_epilogue_desc(m, f, h, "gelu_tanh", "bf16")
    down = o.gemm_epilogue_desc(m, h, f, "none", "f32", "bf16")
    gdown = o.gemm_epilogue_grad_desc(m, h, f, "none", "gelu_tanh", "bf16", "bf16", "f32")
    gup = o.gemm_epilogue_grad_desc(m, f, h, da_type="f32")
    ws = fu.workspace(max(o.gemm_epilogue_workspace_bytes(up), o.gemm_epilogue_workspace_bytes(down),
                          o.gemm_epilogue_grad_workspace_bytes(gdown), o.gemm_epilogue_grad_workspace_bytes(gup)))
    for rank in range(2):
        x, dy = fu.normal(10 + rank, m, h), fu.normal(20 + rank, m, h)
        z, hid = (t.empty(m, f, dtype=t.bfloat16, device="cuda") for _ in range(2))
        y = t.empty(m, h, device="cuda")
        say(f"  block, rank {rank}")
        o.gemm_epilogue_run(up, x, w1, b1, None, hid, z, ws)
        o.gemm_epilogue_run(down, hid, w2, b2, x, y, None, ws)
        bucket = t.zeros(total, device="cuda")
        parts = bucket.split(sizes + [total - sum(sizes)])
        dz, dx = t.empty(m, f, dtype=t.bfloat16, device="cuda"), t.empty(m, h, device="cuda")
        dw1, db1, dw2, db2 = parts[0].view(h, f), parts[1].clone(), parts[2].view(f, h), parts[3].clone()
        # the bucket's matrices start at multiples of 16 bytes here; the gradient's pointers must
        assert dw2.data_ptr() % 16 == 0
        o.gemm_epilogue_grad_run(gdown, dy, hid, w2, z, dz, dw2, None, db2, None, ws)
        o.gemm_epilogue_grad_run(gup, dz, x, w1, None, dx, dw1, None, db1, None, ws)
        parts[1].copy_(db1)
        parts[3].copy_(db2)
        # forward and gradients of this rank in float64, from the stored bf16 tensors
        out, _ = oracle.gemm_epilogue(fu.f64(hid), fu.f64(w2), fu.f64(b2), fu.f64(x))
        tol = fu.sum_bound(fu.f64(hid), fu.f64(w2), f) + 4 * fu.U * (np.abs(out) + 1)
        fu.within(y, out, tol, "y")
        _, dw2_r, db2_r = oracle.gemm_epilogue_grad(fu.f64(dy), fu.f64(hid), fu.f64(w2))
        dx_r, dw1_r, db1_r = oracle.gemm_epilogue_grad(fu.f64(dz), fu.f64(x), fu.f64(w1))
        fu.within(dx, dx_r, fu.sum_bound(fu.f64(dz), fu.f64(w1).T, f), "dx")
        want += np.concatenate([v.ravel() for v in (dw1_r, db1_r, dw2_r, db2_r)])
        buckets.append(bucket)
    # reduce the buckets of the two ranks, then clip the summed gradient in place
    rd = o.ring_desc(2, total, 64)
    fb = o.ring_allreduce_flags_bytes(rd)
    flags, rws = zeros_bytes(fb), zeros_bytes(o.ring_allreduce_workspace_bytes(rd))
    o.ovl_flags_reset(flags, fb, rws, rws.numel())
    summed = [t.zeros(total, device="cuda") for _ in range(2)]
    o.ring_allreduce_run(rd, buckets, summed, flags, rws, 1)
    o.ovl_check(rws)
    grads = list(summed[0].split(sizes + [total - sum(sizes)])[:4])
    plan = o.grad_clip_plan(grads)
    cws = fu.workspace(plan.workspace_bytes)
    o.grad_clip_upload(plan, cws)
    norm = t.empty(1, device="cuda")
    o.grad_norm_clip_run(plan, 1.0, norm, cws)
    n64, clipped = oracle.grad_norm_clip([want], 1.0)
    # every gradient is within (m + 2) U of its absolute sum, at most sqrt(m) times the values' size here
    assert abs(float(norm) - n64) <= 1e-4 * n64
    got = np.concatenate([fu.f64(g).ravel() for g in grads])
    assert np.linalg.norm(got - clipped[0]) <= 1e-4 * np.linalg.norm(clipped[0])


def test_decoding_step_experts_then_projection():
    """A few tokens through the experts and on through a projection with a
    residual, all captured in one graph on one workspace and replayed on new
    tokens."""
    o, t = ovl(), fu.torch()
    T, H, I, E, K, N = 3, 256, 128, 8, 2, 264
    md = o.moe_layer_desc(T, H, I, E, K, "silu", True, "bf16", "bf16")
    ld = o.gemm_epilogue_desc(T, N, H, "none", "f32", "bf16")
    ws = fu.workspace(max(o.moe_layer_workspace_bytes(md), o.gemm_epilogue_workspace_bytes(ld)))
    x, router = fu.normal(1, T, H), fu.normal(2, H, E, sigma=H ** -0.5)
    w1, w2 = fu.normal(3, E, H, 2 * I, sigma=0.1), fu.normal(4, E, I, H, sigma=0.1)
    wp, res = fu.normal(5, H, N, sigma=0.1), fu.normal(6, T, N)
    ids, gates = t.empty(T, K, dtype=t.int32, device="cuda"), t.empty(T, K, device="cuda")
    mid, out = t.empty(T, H, dtype=t.bfloat16, device="cuda"), t.empty(T, N, device="cuda")

    def step():
        o.moe_layer_run(md, x, router, ids, gates, w1, None, w2, None, mid, ws)
        o.gemm_epilogue_run(ld, mid, wp, None, res, out, None, ws)

    step()
    t.cuda.synchronize()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        step()
    for seed in range(3):
        x.copy_(fu.normal(30 + seed, T, H))
        g.replay()
        t.cuda.synchronize()
        got = out.clone()
        want_ids, _ = oracle.route(fu.f64(x) @ fu.f64(router), K, True)
        assert np.array_equal(ids.cpu().numpy(), want_ids)
        ref, _ = oracle.gemm_epilogue(fu.f64(mid), fu.f64(wp), None, fu.f64(res))
        fu.within(got, ref, fu.sum_bound(fu.f64(mid), fu.f64(wp), H) + 4 * fu.U * np.abs(ref), "out")
        moe = oracle.moe_layer(fu.f64(x), want_ids, fu.f64(gates), fu.f64(w1), fu.f64(w2))
        assert np.linalg.norm(fu.f64(mid) - moe) <= (2.0 ** -8 + 1e-4) * np.linalg.norm(moe)
        step()
        t.cuda.synchronize()
        assert t.equal(out, got)


def test_fp8_experts_share_the_dispatch_s_quantizer():
    """E4M3 weights made by fp8_quantize_rows in the dispatch's layout give the
    layer of the decoded weights."""
    from tests.test_gpu_moe_layer import Moe
    c = Moe(6, 256, 128, 4, 2, "fp8", "bf16", seed=40)
    c.run()
    c.check()


def test_calls_at_once_on_two_streams():
    """Calls that overlap in time on workspaces of their own: each one's bits are
    those of the call alone."""
    from tests.test_gpu_clip import tensors
    from tests.test_gpu_linear import Grad, Linear
    from tests.test_gpu_moe_layer import Moe
    o, t = ovl(), fu.torch()
    src = tensors([70000, 31, 30000])

    class Clip:
        def __init__(self):
            self.out = [t.empty_like(v) for v in src]
            self.plan = o.grad_clip_plan(src, self.out)
            self.ws, self.norm = fu.workspace(self.plan.workspace_bytes), t.zeros(1, device="cuda")
            o.grad_clip_upload(self.plan, self.ws)

        def run(self):
            o.grad_norm_clip_run(self.plan, 0.5, self.norm, self.ws)

    def results(c):
        return [getattr(c, n) for n in ("out", "z", "da", "db", "dbias", "norm", "gates") if t.is_tensor(getattr(c, n, None))] \
            + (c.out if isinstance(c, Clip) else [])

    def calls():
        return [Linear(300, 264, 520), Linear(1, 2048, 4096), Grad(700, 264, 136), Moe(1, 1024, 512, 16, 2),
                Moe(9, 512, 256, 8, 2, "fp8"), Clip()]

    alone, left, right = calls(), calls(), calls()
    for c in alone:
        c.run()
    t.cuda.synchronize()
    streams = t.cuda.Stream(), t.cuda.Stream()
    for _ in range(3):
        for s, cs in zip(streams, (left, right[::-1])):
            s.wait_stream(t.cuda.current_stream())
            with t.cuda.stream(s):
                for c in cs:
                    c.run()
        t.cuda.synchronize()
        for want, a, b in zip(alone, left, right):
            for x, y, z in zip(results(want), results(a), results(b)):
                assert t.equal(x, y) and t.equal(x, z)
