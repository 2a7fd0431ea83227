"""The few-token mixture-of-experts layer against the float64 oracle."""

import numpy as np
import pytest

import oracle
from tests import ffn_util as fu
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


def ovl():
    from communication_overlap_amd import ovl as _o
    return _o


class Moe:
    def __init__(self, T, H, I, E, K, w="bf16", out="f32", act="silu", gated=True, norm=True, route=True, seed=0):
        o, t = ovl(), fu.torch()
        self.T, self.H, self.I, self.E, self.K = T, H, I, E, K
        self.w, self.out_t, self.act, self.gated, self.norm = w, out, act, gated, norm
        n1 = 2 * I if gated else I
        self.desc = o.moe_layer_desc(T, H, I, E, K, act, gated, w, out, norm)
        self.x = fu.normal(seed, T, H)
        self.router = fu.normal(seed + 1, H, E, sigma=H ** -0.5) if route else None
        self.w1, self.w2 = fu.normal(seed + 2, E, H, n1, sigma=0.1), fu.normal(seed + 3, E, I, H, sigma=0.1)
        self.s1 = self.s2 = None
        if w == "fp8":  # the quantizer of the FP8 dispatch, on the transposed weights
            self.w1, self.s1 = self.quantize(self.w1)
            self.w2, self.s2 = self.quantize(self.w2)
        r = np.random.RandomState(seed)
        self.ids = t.full((T, K), 99, dtype=t.int32, device="cuda")
        self.gates = t.full((T, K), 99.0, device="cuda")
        if not route:
            ids = np.stack([r.permutation(E)[:K] for _ in range(T)]).astype(np.int32).reshape(T, K)
            self.ids.copy_(t.from_numpy(ids))
            self.gates.copy_(t.from_numpy(r.rand(T, K).astype(np.float32)))
        self.out = t.full((T + 1, H), 7.0, dtype=fu.ttype(out), device="cuda")
        self.ws = fu.workspace(o.moe_layer_workspace_bytes(self.desc))

    @staticmethod
    def quantize(w):
        o, t = ovl(), fu.torch()
        rows = w.transpose(1, 2).contiguous()
        codes = t.empty(rows.shape, dtype=t.uint8, device="cuda")
        scale = t.empty(rows.shape[:2], device="cuda")
        o.fp8_quantize_rows(rows, codes, scale, rows.shape[0] * rows.shape[1], rows.shape[2])
        return codes, scale

    def weights(self):
        if self.w == "bf16":
            return fu.f64(self.w1), fu.f64(self.w2)
        dec = lambda c, s: (oracle.e4m3_decode(c.cpu().numpy()) * fu.f64(s)[..., None]).transpose(0, 2, 1)  # noqa: E731
        return dec(self.w1, self.s1), dec(self.w2, self.s2)

    def run(self, stream=None):
        say(f"  moe_layer_run T={self.T} H={self.H} I={self.I} E={self.E} K={self.K} {self.w} out={self.out_t}")
        ovl().moe_layer_run(self.desc, self.x, self.router, self.ids, self.gates, self.w1, self.s1, self.w2, self.s2,
                            self.out, self.ws, stream)

    def check(self):
        x = fu.f64(self.x)
        w1, w2 = self.weights()
        if self.router is not None:
            ids, gates = oracle.route(x @ fu.f64(self.router), self.K, self.norm)
            assert np.array_equal(self.ids.cpu().numpy(), ids)
            fu.within(self.gates, gates, 4 * fu.U * gates, "gates")
        ids, gates = self.ids.cpu().numpy(), fu.f64(self.gates)
        ref = oracle.moe_layer(x, ids, gates, w1, w2, self.act, self.gated)
        planes = 2.0 ** -17 if self.out_t == "bf16" else 2.0 ** -25
        bound = np.zeros_like(ref)
        size = np.zeros_like(ref)
        for t in range(self.T):
            for j in range(self.K):
                e = int(ids[t, j])
                if not 0 <= e < self.E:
                    continue
                u = x[t] @ w1[e]
                ub = (self.H + 4) * fu.U * (np.abs(x[t]) @ np.abs(w1[e])) + 2 * fu.U * np.abs(u)
                g, gb = oracle.act(u[:self.I], self.act), ub[:self.I]
                gb = fu.SLOPE * gb + 16 * fu.U * (np.abs(g) + np.abs(u[:self.I]))
                h, hb = g, gb
                if self.gated:
                    h = g * u[self.I:]
                    hb = gb * np.abs(u[self.I:]) + (np.abs(g) + gb) * ub[self.I:]
                hb = hb + (2 * fu.U + planes) * np.abs(h)
                a2 = np.abs(w2[e])
                bound[t] += gates[t, j] * (hb @ a2 + (3 * self.I + 8) * fu.U * (np.abs(h) @ a2))
                size[t] += gates[t, j] * np.abs(h @ w2[e])
        bound += (2 * self.K + 2) * fu.U * size
        fu.within(self.out[:self.T], ref, bound + fu.HALF[self.out_t] * (np.abs(ref) + bound), "out")
        assert bool((self.out[self.T] == 7).all()), "wrote past the last token"


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 33, 64, 128])
@pytest.mark.parametrize("w", ["bf16", "fp8"])
def test_token_counts(T, w):
    c = Moe(T, 144, 80, 12, 3, w, seed=T)
    c.run()
    c.check()


@pytest.mark.parametrize("H,I,E,K", [(8, 8, 1, 1), (72, 40, 5, 5), (1032, 264, 8, 2), (64, 512, 256, 8),
                                     (200, 72, 60, 4), (136, 8, 130, 2)])
def test_ragged_sizes(H, I, E, K):
    c = Moe(7, H, I, E, K, seed=3)
    c.run()
    c.check()


@pytest.mark.parametrize("H,I", [(16, 16), (80, 208), (1040, 272)])
def test_ragged_sizes_fp8(H, I):
    c = Moe(5, H, I, 6, 2, "fp8", "bf16", seed=4)
    c.run()
    c.check()


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("out,w", [("bf16", "bf16"), ("f32", "fp8")])
def test_activations_and_types(act, gated, out, w):
    c = Moe(4, 96, 80, 6, 2, w, out, act, gated, norm=gated, seed=5)
    c.run()
    c.check()


@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("w", ["bf16", "fp8"])
def test_caller_s_routing_with_absent_and_repeated_experts(T, w):
    t = fu.torch()
    c = Moe(T, 96, 48, 6, 4, w, route=False, seed=6)
    c.ids[0] = -1                                   # a token without experts here
    c.ids[1] = t.tensor([6, 2, -7, 2 ** 31 - 1])    # one of four here
    c.ids[2] = 5                                    # the same expert four times
    c.run()
    c.check()
    assert not bool(c.out[0].any())


def test_every_pair_on_one_expert():
    """128 tokens x 8 choices of one expert: the row groups go round."""
    c = Moe(128, 64, 48, 8, 8, route=False, seed=7)
    c.ids.fill_(3)
    c.run()
    c.check()


@pytest.mark.parametrize("T", [1, 5])
def test_no_expert_of_this_rank_gives_zeros(T):
    c = Moe(T, 200, 48, 6, 2, route=False, seed=8)
    c.ids.fill_(-1)
    c.run()
    assert not bool(c.out[:T].any()) and bool((c.out[T] == 7).all())


def test_ties_go_to_the_lower_id_and_nan_comes_last():
    t = fu.torch()
    c = Moe(2, 64, 32, 9, 4, seed=9)
    c.router.zero_()
    c.router[:, 7] = 0.5
    c.x[:, :] = 1.0
    c.x[1] = -1.0
    c.run()
    assert c.ids.cpu().tolist() == [[7, 0, 1, 2], [0, 1, 2, 3]]
    c.router[0, 0] = float("nan")
    c.run()
    assert c.ids.cpu().tolist() == [[7, 1, 2, 3], [1, 2, 3, 4]]
    assert bool(t.isfinite(c.gates).all())  # norm_topk: over the chosen ones only


def test_not_finite_weights_of_other_experts_do_not_leak():
    t = fu.torch()
    c = Moe(3, 72, 40, 4, 2, route=False, seed=10)
    c.ids[:] = t.tensor([0, 2])
    for e in (1, 3):
        c.w1[e] = float("nan")
        c.w2[e] = float("inf")
    c.run()
    assert bool(t.isfinite(c.out).all())
    w1, w2 = fu.f64(c.w1), fu.f64(c.w2)
    w1[[1, 3]], w2[[1, 3]] = 0, 0
    c.weights = lambda: (w1, w2)
    c.check()


def test_every_e4m3_code_is_widened_exactly():
    """x picks one code a token, the second weight copies it out: the output is
    the code's value, over all 254 finite codes (subnormals and both zeros)."""
    t = fu.torch()
    c = Moe(128, 256, 16, 1, 1, "fp8", "f32", "none", False, route=False, seed=1)
    codes = np.arange(256, dtype=np.uint8)
    codes[[0x7F, 0xFF]] = 0  # the NaN codes: zero times NaN would reach every token
    c.w1.zero_()
    c.w1[0, 3] = t.from_numpy(codes).cuda()
    c.w2.zero_()
    c.w2[0, 5, 3] = 0x38  # 1.0
    c.s1.fill_(1.0)
    c.s2.fill_(1.0)
    c.ids.zero_()
    c.gates.fill_(1.0)
    for half in range(2):
        c.x.zero_()
        c.x[t.arange(128), t.arange(128) + 128 * half] = 1.0
        c.run()
        want = oracle.e4m3_decode(codes[128 * half:128 * (half + 1)])
        assert np.array_equal(fu.f64(c.out[:128, 5]), want)
        rest = c.out[:128].clone()
        rest[:, 5] = 0
        assert not bool(rest.any())


@pytest.mark.parametrize("w,out", [("bf16", "f32"), ("fp8", "f32"), ("fp8", "bf16")])
@pytest.mark.parametrize("E,T,K", [(2, 128, 2), (16, 100, 8)])
def test_many_units_a_workgroup(w, out, E, T, K):
    """Many short units in turn: few steps each, rows over several groups."""
    c = Moe(T, 2048, 48, E, K, w, out, seed=21)
    c.run()
    c.check()
    d = Moe(T, 48, 4096, E, K, w, out, seed=22)
    d.run()
    d.check()


def test_weights_past_four_gib():
    """Experts whose weights lie past 32-bit offsets."""
    t, o = fu.torch(), ovl()
    T, H, I, E = 3, 2048, 2048, 200
    d = o.moe_layer_desc(T, H, I, E, 2, "relu", False, "bf16", "f32")
    w1 = t.zeros(E, H, I, dtype=t.bfloat16, device="cuda")
    w2 = t.zeros(E, I, H, dtype=t.bfloat16, device="cuda")
    assert w1.numel() > 1 << 29
    r = np.random.RandomState(1)
    for e in (0, 197, 199):
        w1[e] = t.from_numpy(r.randint(-1, 2, (H, I)).astype(np.float32)).cuda().bfloat16()
        w2[e] = t.from_numpy(r.randint(-1, 2, (I, H)).astype(np.float32)).cuda().bfloat16()
    x = t.from_numpy(r.randint(-1, 2, (T, H)).astype(np.float32)).cuda().bfloat16()
    ids = t.tensor([[199, 0], [197, 199], [0, 197]], dtype=t.int32, device="cuda")
    gates = t.tensor([[1.0, 2.0], [0.5, 1.0], [1.0, 4.0]], device="cuda")
    out = t.empty(T, H, device="cuda")
    say("  moe_layer_run with 1.7 GB a weight")
    o.moe_layer_run(d, x, None, ids, gates, w1, None, w2, None, out, fu.workspace(o.moe_layer_workspace_bytes(d)))
    for i in range(T):  # small integers: exact in float32 up to 2^24
        want = sum(float(gates[i, j]) * (np.maximum(fu.f64(x[i]) @ fu.f64(w1[int(ids[i, j])]), 0)
                                         @ fu.f64(w2[int(ids[i, j])])) for j in range(2))
        assert np.abs(want).max() < 2 ** 24 and np.array_equal(fu.f64(out[i]), want)


@pytest.mark.parametrize("T,w", [(1, "bf16"), (20, "bf16"), (9, "fp8")])
def test_same_bits_capture_and_a_shared_workspace(T, w):
    t, o = fu.torch(), ovl()
    c = Moe(T, 1024, 512, 16, 2, w, seed=11)
    e = Moe(T + 3, 208, 304, 5, 3, "bf16", "bf16", seed=12)
    c.ws = e.ws = fu.workspace(max(c.ws.numel(), e.ws.numel()))
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
    for _ in range(4):
        c.out[:T].zero_()
        e.run()
        g.replay()
        t.cuda.synchronize()
        assert t.equal(c.out, want)
        e.check()


@pytest.mark.parametrize("H,E,K", [(64, 1, 1), (64, 9, 4), (4096, 64, 8), (4104, 64, 2), (72, 65, 3), (200, 256, 8)])
@pytest.mark.parametrize("norm", [True, False])
def test_one_token_picks_as_a_row_of_many_does(H, E, K, norm):
    """A token alone has a routing of its own; its choices and gates are those it
    has beside others, ties and NaN among the logits included."""
    t = fu.torch()
    many, one = Moe(3, H, 16, E, K, norm=norm, seed=20), Moe(1, H, 16, E, K, norm=norm, seed=20)
    for x in (many, one):
        x.router = fu.normal(21, H, E, sigma=H ** -0.5)
    one.x = many.x[1:2].clone()
    for i in range(3):
        if i == 1 and E > 4:     # ties, between near and far ids
            for x in (many, one):
                x.router[:, E - 1] = x.router[:, 0]
                x.router[:, 3] = x.router[:, 2]
        if i == 2 and E > 4:     # fewer numbers than choices
            for x in (many, one):
                x.router[0, 1:E - K + 2] = float("nan")
        many.run()
        one.run()
        assert t.equal(one.ids[0], many.ids[1])
        assert t.equal(one.gates[0], many.gates[1]) or (
            bool((one.gates[0].isnan() == many.gates[1].isnan()).all())
            and t.equal(one.gates[0].nan_to_num(7.0), many.gates[1].nan_to_num(7.0)))
        if i == 0:
            one.check()
