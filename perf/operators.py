"""The operators of the feed-forward path as measured cases: the product with
bias, activation and residual in its epilogue, its gradient, a whole
mixture-of-experts layer for a few tokens, and the global gradient norm with
clipping.

`run` computes a case in plain torch operations (float32 throughout, rounded
once into the output's type) or, where `own` is true, through the library's
entry points; `exact` gives the same outputs from the definitions in float64.
"""

import math

import torch

own = False

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # Feed-forward up projection of a training step at the AG-GEMM headline size: bias,
        # activation, and the pre-activation kept for the backward pass.
        linear("linear_train", 8192, 3584, 4096, "gelu_tanh", "bf16", bias=True, residual="", keep_z=True),
        # One decoded token through an output projection of the skinny AG-GEMM's weight: latency.
        linear("linear_token", 1, 7168, 8192, "none", "bf16", bias=True, residual="bf16", keep_z=False),
        # A ragged batch: no size a multiple of a tile, float32 residual stream.
        linear("linear_ragged", 1000, 2056, 520, "silu", "f32", bias=True, residual="f32", keep_z=False),
        # Gradient of the feed-forward down projection at the GEMM-RS size: the derivative of the
        # activation before it folded in, float32 weight gradients accumulated over micro-batches.
        grad("grad_train", 8192, 4096, 1792, "gelu_tanh", "bf16", "f32", accumulate=True, dbias=True),
        # Gradient of a ragged batch, bf16 gradients throughout.
        grad("grad_ragged", 700, 2056, 520, "silu", "bf16", "bf16", accumulate=False, dbias=True),
        # Gradient of the smallest AG-GEMM's product: latency.
        grad("grad_small", 128, 256, 256, "none", "f32", "f32", accumulate=False, dbias=True),
        # One decoded token through the MoE layer of the dispatch workload, routing included.
        moe("moe_token", 1, 4096, 1408, 64, 2, "bf16", "silu", gated=True, route=True, out="bf16"),
        # A small decode batch with FP8 weights, routed by the caller (experts held elsewhere left out).
        moe("moe_fp8", 9, 4096, 1408, 64, 4, "fp8", "silu", gated=True, route=False, out="f32"),
        # The largest decode batch: most experts are read.
        moe("moe_batch", 64, 4096, 1408, 64, 2, "bf16", "silu", gated=True, route=True, out="bf16"),
        # A few small tensors (biases and norms of a small module): latency.
        clip("clip_small", "small", 8, 4099, "f32", max_norm=0.25),
        # One reduced gradient bucket of the ring all-reduce (8M float32).
        clip("clip_bucket", "even", 1, 8 << 20, "f32", max_norm=1.0),
        # The gradients of a whole model: large matrices beside many short vectors, both types.
        clip("clip_model", "model", 60, 384 << 20, "mixed", max_norm=1.0),
    ]


def draw(rng):
    def log(lo, hi, step=1):
        return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))) // step * step))

    kind = rng.choice(("linear", "linear", "grad", "moe", "clip"))
    if kind in ("linear", "grad"):
        while True:
            m, n, k = log(1, 8192), log(8, 8192, 8), log(8, 8192, 8)
            if m * n * k <= 8192 * 4096 * 1792:
                break
        if kind == "linear":
            return linear(None, m, n, k, rng.choice(ACTS), rng.choice(("bf16", "f32")), bias=rng.random() < 0.7,
                          residual=rng.choice(("", "bf16", "f32")), keep_z=rng.random() < 0.5)
        return grad(None, m, n, k, rng.choice(ACTS), rng.choice(("bf16", "f32")), rng.choice(("bf16", "f32")),
                    accumulate=rng.random() < 0.5, dbias=rng.random() < 0.7)
    if kind == "moe":
        experts = rng.choice((4, 8, 16, 32, 60, 64))
        return moe(None, log(1, 64), log(64, 4096, 16), log(32, 1408, 16), experts, rng.randint(1, 4),
                   rng.choice(("bf16", "fp8")), rng.choice(("relu", "gelu", "gelu_tanh", "silu")),
                   gated=rng.random() < 0.7, route=rng.random() < 0.5, out=rng.choice(("bf16", "f32")))
    count = log(1, 60)
    return clip(None, rng.choice(("small", "even", "model")), count, log(count, 256 << 20),
                rng.choice(("f32", "bf16", "mixed")), max_norm=rng.choice((0.5, 1.0, 1e9)))


def linear(name, m, n, k, act, out, bias, residual, keep_z):
    return named(name, kind="linear", m=m, n=n, k=k, act=act, out=out, bias=bias, residual=residual, keep_z=keep_z)


def grad(name, m, n, k, act_in, da, db, accumulate, dbias):
    return named(name, kind="grad", m=m, n=n, k=k, act=act_in, da=da, db=db, accumulate=accumulate, dbias=dbias)


def moe(name, tokens, hidden, inter, experts, topk, weights, act, gated, route, out):
    return named(name, kind="moe", tokens=tokens, hidden=hidden, inter=inter, experts=experts, topk=topk,
                 weights=weights, act=act, gated=gated, route=route, out=out)


def clip(name, shape, count, total, types, max_norm):
    return named(name, kind="clip", shape=shape, count=count, total=total, types=types, max_norm=max_norm)


def named(name, **case):
    return {"name": name, **case} if name else case


def work(case):
    size = {"bf16": 2, "f32": 4, "": 0}
    if case["kind"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": 2 * (m * k + k * n) + 4 * n * case["bias"]
                + m * n * (size[case["residual"]] + size[case["out"]] + 2 * case["keep_z"]),
                "flops": 2 * m * n * k}
    if case["kind"] == "grad":
        m, n, k = case["m"], case["n"], case["k"]
        z_in = 0 if case["act"] == "none" else 2 * m * k
        return {"bytes": 2 * (m * n + m * k + k * n) + z_in + m * k * size[case["da"]]
                + k * n * size[case["db"]] * (2 if case["accumulate"] else 1)
                + 4 * n * case["dbias"] * (2 if case["accumulate"] else 1),
                "flops": 4 * m * n * k}
    if case["kind"] == "moe":
        t, h, i, e, j = case["tokens"], case["hidden"], case["inter"], case["experts"], min(case["topk"], case["experts"])
        per = h * i * (3 if case["gated"] else 2)
        read = e * (1.0 - (1.0 - j / e) ** t)  # experts that t tokens' choices reach
        return {"bytes": int(per * (1 if case["weights"] == "fp8" else 2) * read) + 2 * h * e * case["route"]
                + t * h * (2 + size[case["out"]]) + 8 * t * j,
                "flops": 2 * t * j * per + 2 * t * h * e * case["route"]}
    nbytes = sum(n * size[t] for n, t in tensors_of(case))
    return {"bytes": 2 * nbytes + 4, "flops": 3 * sum(n for n, _ in tensors_of(case))}


def tensors_of(case):
    """(length, type) of each gradient of a clip case, fixed by the case."""
    count, total = case["count"], case["total"]
    if case["shape"] == "even":
        sizes = [total // count] * count
    elif case["shape"] == "small":
        sizes = [1 + (total // count) * (2 * i + 1) // count for i in range(count)]
    else:  # a model: one matrix in six holds nearly everything, the rest are vectors
        big = (count + 5) // 6
        sizes = [(total // big) - 13 * (i % 7) if i % 6 == 0 else 1 + 97 * (i % 43) for i in range(count)]
    kinds = {"f32": ("f32",), "bf16": ("bf16",), "mixed": ("bf16", "bf16", "bf16", "f32")}[case["types"]]
    return [(max(0, n), kinds[(i // 6) % len(kinds)]) for i, n in enumerate(sizes)]


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, sigma=1.0, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(sigma)

    def empty(*shape, dtype):
        return torch.empty(shape, device="cuda", dtype=dtype)

    s = {"case": case}
    if case["kind"] in ("linear", "grad"):
        m, n, k = case["m"], case["n"], case["k"]
        s["a"], s["b"] = normal(m, k), normal(k, n, sigma=0.02)
        if case["kind"] == "linear":
            s["bias"] = normal(n, sigma=0.1, dtype=torch.float32) if case["bias"] else None
            s["residual"] = normal(m, n, dtype=TYPES[case["residual"]]) if case["residual"] else None
            s["out"] = empty(m, n, dtype=TYPES[case["out"]])
            s["z"] = empty(m, n, dtype=torch.bfloat16) if case["keep_z"] else None
        else:
            s["dz"] = normal(m, n, sigma=0.1)
            s["z_in"] = normal(m, k) if case["act"] != "none" else None
            s["db_in"] = normal(k, n, dtype=TYPES[case["db"]]) if case["accumulate"] else None
            s["dbias_in"] = normal(n, dtype=torch.float32) if case["accumulate"] and case["dbias"] else None
            s["da"] = empty(m, k, dtype=TYPES[case["da"]])
            s["db"] = empty(k, n, dtype=TYPES[case["db"]])
            s["dbias"] = empty(n, dtype=torch.float32) if case["dbias"] else None
    elif case["kind"] == "moe":
        t, h, i, e, j = case["tokens"], case["hidden"], case["inter"], case["experts"], min(case["topk"], case["experts"])
        n1 = 2 * i if case["gated"] else i
        s["x"] = normal(t, h)
        if case["weights"] == "bf16":
            s["w1"], s["w2"] = normal(e, h, n1, sigma=0.02), normal(e, i, h, sigma=0.02)
            s["s1"] = s["s2"] = None
        else:
            # E4M3 codes of rows scaled to the format's range, and the float32 scale of each row.
            s["w1"], s["s1"] = fp8_rows(normal(e, n1, h, sigma=0.02))
            s["w2"], s["s2"] = fp8_rows(normal(e, h, i, sigma=0.02))
        if case["route"]:
            s["router"] = normal(h, e, sigma=1.0 / math.sqrt(h))
            s["topk"], s["gates"] = empty(t, j, dtype=torch.int32), empty(t, j, dtype=torch.float32)
        else:
            keys = torch.rand(t, e, generator=g, device="cuda")
            s["router"] = None
            s["topk"] = keys.argsort(dim=1)[:, :j].to(torch.int32).contiguous()
            s["topk"][torch.rand(t, j, generator=g, device="cuda") < 0.1] = -1  # an expert of another rank
            s["gates"] = torch.rand(t, j, generator=g, device="cuda")
        s["out"] = empty(t, h, dtype=TYPES[case["out"]])
    else:
        s["src"] = [normal(n, sigma=0.01, dtype=TYPES[t]) for n, t in tensors_of(case)]
        s["dst"] = [torch.empty_like(v) for v in s["src"]]
        s["norm"] = empty(1, dtype=torch.float32)
    return s


def fp8_rows(w):
    amax = w.abs().amax(dim=-1).float()
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    codes = torch.empty(w.shape, device=w.device, dtype=torch.uint8)
    for e in range(w.shape[0]):  # expert by expert: the float32 copy stays small
        q = (w[e].float() / scale[e].unsqueeze(-1)).clamp(-448.0, 448.0)
        codes[e] = q.to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, scale


# ------------------------------------------------------------------ plain forms

def act(z, kind):
    if kind == "relu":
        return torch.clamp(z, min=0.0)
    if kind == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if kind == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if kind == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def act_grad(z, kind):
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    if kind == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * z * z)
    if kind == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    return torch.ones_like(z)


def run(state):
    kind = state["case"]["kind"]
    if own:
        return {"linear": own_linear, "grad": own_grad, "moe": own_moe, "clip": own_clip}[kind](state)
    return {"linear": plain_linear, "grad": plain_grad, "moe": plain_moe, "clip": plain_clip}[kind](state)


def plain_linear(s):
    c = s["case"]
    z = s["a"].float() @ s["b"].float()
    if s["bias"] is not None:
        z = z + s["bias"]
    out = act(z, c["act"])
    if s["residual"] is not None:
        out = out + s["residual"].float()
    result = {"out": out.to(TYPES[c["out"]])}
    if c["keep_z"]:
        result["z"] = z.to(torch.bfloat16)
    return result


def plain_grad(s):
    c = s["case"]
    dz = s["dz"].float()
    da = dz @ s["b"].float().t()
    if s["z_in"] is not None:
        da = da * act_grad(s["z_in"].float(), c["act"])
    db = s["a"].float().t() @ dz
    if s["db_in"] is not None:
        db = db + s["db_in"].float()
    result = {"da": da.to(TYPES[c["da"]]), "db": db.to(TYPES[c["db"]])}
    if c["dbias"]:
        dbias = dz.sum(dim=0)
        result["dbias"] = dbias + s["dbias_in"] if s["dbias_in"] is not None else dbias
    return result


def choose(logits, topk):
    """The topk largest of each row, ties to the lower id, and their softmax weights."""
    order = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :topk]
    e = torch.exp(logits - logits.amax(dim=1, keepdim=True))
    p = e / e.sum(dim=1, keepdim=True)
    picked = p.gather(1, order)
    return order.to(torch.int32), (picked / picked.sum(dim=1, keepdim=True)).float()


def plain_moe(s):
    c = s["case"]
    j = s["topk"].shape[1]
    x = s["x"].float()
    if c["route"]:
        # 64 bits: a choice between two near logits must not hang on the order of a sum.
        topk, gates = choose(s["x"].double() @ s["router"].double(), j)
    else:
        topk, gates = s["topk"], s["gates"]
    ids = topk.flatten().long()
    here = (ids >= 0) & (ids < c["experts"])
    ids = torch.where(here, ids, torch.zeros_like(ids))
    xs = x.repeat_interleave(j, dim=0)
    if c["weights"] == "bf16":
        u = torch.bmm(xs.unsqueeze(1), s["w1"][ids].float()).squeeze(1)
    else:
        u = torch.bmm(s["w1"][ids].view(torch.float8_e4m3fn).float(), xs.unsqueeze(2)).squeeze(2) * s["s1"][ids]
    h = act(u[:, :c["inter"]], c["act"])
    if c["gated"]:
        h = h * u[:, c["inter"]:]
    if c["weights"] == "bf16":
        y = torch.bmm(h.unsqueeze(1), s["w2"][ids].float()).squeeze(1)
    else:
        y = torch.bmm(s["w2"][ids].view(torch.float8_e4m3fn).float(), h.unsqueeze(2)).squeeze(2) * s["s2"][ids]
    y = torch.where(here.unsqueeze(1), y * gates.flatten().unsqueeze(1), torch.zeros_like(y))
    result = {"out": y.view(c["tokens"], j, c["hidden"]).sum(dim=1).to(TYPES[c["out"]])}
    if c["route"]:
        result["topk"], result["gates"] = topk, gates
    return result


def plain_clip(s):
    norms = torch.stack([(v.float() * v.float()).sum(dtype=torch.float64) for v in s["src"]])
    norm = norms.sum().sqrt().float()
    coef = torch.clamp(s["case"]["max_norm"] / (norm + 1e-6), max=1.0)
    return {"norm": norm.reshape(1), "dst": [(v.float() * coef).to(v.dtype) for v in s["src"]]}


# ------------------------------------------------------------------ the library's calls

def workspace(nbytes):
    """A program's workspace, zeroed once."""
    from communication_overlap_amd import ovl
    ws = torch.empty(max(16, nbytes), device="cuda", dtype=torch.uint8)
    ovl.ovl_flags_reset(None, 0, ws, ws.numel())
    return ws


def own_linear(s):
    from communication_overlap_amd import ovl
    if "desc" not in s:
        c = s["case"]
        s["desc"] = ovl.gemm_epilogue_desc(c["m"], c["n"], c["k"], act=c["act"], out_type=c["out"],
                                           res_type=c["residual"] or "bf16")
        s["ws"] = workspace(ovl.gemm_epilogue_workspace_bytes(s["desc"]))
    ovl.gemm_epilogue_run(s["desc"], s["a"], s["b"], s["bias"], s["residual"], s["out"], s["z"], s["ws"])
    return {"out": s["out"], "z": s["z"]} if s["z"] is not None else {"out": s["out"]}


def own_grad(s):
    from communication_overlap_amd import ovl
    if "desc" not in s:
        c = s["case"]
        s["desc"] = ovl.gemm_epilogue_grad_desc(c["m"], c["n"], c["k"], act_in=c["act"], da_type=c["da"],
                                                db_type=c["db"])
        s["ws"] = workspace(ovl.gemm_epilogue_grad_workspace_bytes(s["desc"]))
    ovl.gemm_epilogue_grad_run(s["desc"], s["dz"], s["a"], s["b"], s["z_in"], s["da"], s["db"], s["db_in"],
                               s["dbias"], s["dbias_in"], s["ws"])
    result = {"da": s["da"], "db": s["db"]}
    if s["dbias"] is not None:
        result["dbias"] = s["dbias"]
    return result


def own_moe(s):
    from communication_overlap_amd import ovl
    if "desc" not in s:
        c = s["case"]
        s["desc"] = ovl.moe_layer_desc(c["tokens"], c["hidden"], c["inter"], c["experts"], s["topk"].shape[1],
                                       act=c["act"], gated=c["gated"], w_type=c["weights"], out_type=c["out"],
                                       norm_topk=True)
        s["ws"] = workspace(ovl.moe_layer_workspace_bytes(s["desc"]))
    ovl.moe_layer_run(s["desc"], s["x"], s["router"], s["topk"], s["gates"], s["w1"], s["s1"], s["w2"], s["s2"],
                      s["out"], s["ws"])
    if s["router"] is not None:
        return {"out": s["out"], "topk": s["topk"], "gates": s["gates"]}
    return {"out": s["out"]}


def own_clip(s):
    from communication_overlap_amd import ovl
    if "plan" not in s:
        s["plan"] = ovl.grad_clip_plan(s["src"], s["dst"])
        s["ws"] = workspace(s["plan"].workspace_bytes)
        ovl.grad_clip_upload(s["plan"], s["ws"])
    ovl.grad_norm_clip_run(s["plan"], s["case"]["max_norm"], s["norm"], s["ws"])
    return {"norm": s["norm"], "dst": s["dst"]}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "linear":
        z = torch.matmul(s["a"].double(), s["b"].double())
        if case["bias"]:
            z += s["bias"].double()
        out = exact_act(z, case["act"])[0]
        if case["residual"]:
            out = out + s["residual"].double()
        return {"out": out, "z": z} if case["keep_z"] else {"out": out}
    if case["kind"] == "grad":
        dz = s["dz"].double()
        da = torch.matmul(dz, s["b"].double().t().contiguous())
        if s["z_in"] is not None:
            da *= exact_act(s["z_in"].double(), case["act"])[1]
        db = torch.matmul(s["a"].double().t().contiguous(), dz)
        if case["accumulate"]:
            db += s["db_in"].double()
        result = {"da": da, "db": db}
        if case["dbias"]:
            result["dbias"] = torch.ones(1, case["m"], device="cuda", dtype=torch.float64).matmul(dz).flatten()
            if case["accumulate"]:
                result["dbias"] += s["dbias_in"].double()
        return result
    if case["kind"] == "moe":
        return exact_moe(case, s)
    total = torch.zeros((), device="cuda", dtype=torch.float64)
    for v in s["src"]:
        total += torch.linalg.vector_norm(v, dtype=torch.float64) ** 2 if v.numel() else 0.0
    norm = math.sqrt(float(total))
    coef = min(1.0, case["max_norm"] / (norm + 1e-6))
    return {"norm": torch.tensor([norm], device="cuda", dtype=torch.float64),
            "dst": [v.double() * coef for v in s["src"]]}


def exact_act(z, kind):
    """The activation and its derivative at z, by the tail functions rather than by differences from one."""
    if kind == "none":
        return z, torch.ones_like(z)
    if kind == "relu":
        pos = (z > 0).double()
        return z * pos, pos
    if kind == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * torch.sigmoid(-z)
    if kind == "gelu":
        cdf = 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
        return z * cdf, cdf + z * torch.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi)
    # The tanh form is z sigma(2u), u = sqrt(2 / pi) (z + 0.044715 z^3).
    r = math.sqrt(2.0 / math.pi)
    s = torch.sigmoid(2.0 * r * (z + 0.044715 * z ** 3))
    t = torch.sigmoid(-2.0 * r * (z + 0.044715 * z ** 3))
    return z * s, s + 2.0 * z * s * t * r * (1.0 + 0.134145 * z ** 2)


def exact_moe(case, s):
    t, j, i = case["tokens"], s["topk"].shape[1], case["inter"]
    x = s["x"].double()
    result = {}
    if case["route"]:
        logits = torch.matmul(x, s["router"].double()).cpu()
        rows = [sorted(range(case["experts"]), key=lambda e: (-row[e], e))[:j] for row in logits.tolist()]
        topk = torch.tensor(rows, device="cuda")
        gates = torch.softmax(logits.cuda().gather(1, topk), dim=1)  # the softmax over all, renormalised
        result["topk"], result["gates"] = topk.to(torch.int32), gates
    else:
        topk, gates = s["topk"].long(), s["gates"].double()
    out = torch.zeros(t, case["hidden"], device="cuda", dtype=torch.float64)
    for e in sorted(set(topk.flatten().tolist())):
        if not 0 <= e < case["experts"]:
            continue
        tok, slot = (topk == e).nonzero(as_tuple=True)
        if case["weights"] == "bf16":
            w1, w2 = s["w1"][e].double(), s["w2"][e].double()
        else:
            w1 = (s["w1"][e].view(torch.float8_e4m3fn).double() * s["s1"][e].double().unsqueeze(1)).t().contiguous()
            w2 = (s["w2"][e].view(torch.float8_e4m3fn).double() * s["s2"][e].double().unsqueeze(1)).t().contiguous()
        u = torch.matmul(x[tok], w1)
        h = exact_act(u[:, :i], case["act"])[0]
        if case["gated"]:
            h = h * u[:, i:]
        out.index_add_(0, tok, torch.matmul(h, w2) * gates[tok, slot].unsqueeze(1))
    return {"out": out, **result}
