"""Feed-forward layers on one rank: the product with bias, activation and
residual, its gradient, the few-token mixture-of-experts layer, and the
global gradient norm with clipping, in float64 from exactly decoded inputs.

Every matrix is a numpy float64 array (the caller decodes bf16 and E4M3).
"""

import math

import numpy as np

GELU_R = math.sqrt(2.0 / math.pi)
GELU_C = 0.044715

_erf = np.vectorize(math.erf, otypes=[np.float64])


def _sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def act(z, kind: str):
    z = np.asarray(z, dtype=np.float64)
    if kind == "relu":
        return np.where(z < 0, 0.0, z)
    if kind == "gelu":
        return 0.5 * z * (1.0 + _erf(z / math.sqrt(2.0))) if z.size else z
    if kind == "gelu_tanh":
        return 0.5 * z * (1.0 + np.tanh(GELU_R * (z + GELU_C * z ** 3)))
    if kind == "silu":
        return z * _sigmoid(z)
    return z


def act_grad(z, kind: str):
    z = np.asarray(z, dtype=np.float64)
    if kind == "relu":
        return (z > 0).astype(np.float64)
    if kind == "gelu":
        if not z.size:
            return z
        return 0.5 * (1.0 + _erf(z / math.sqrt(2.0))) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if kind == "gelu_tanh":
        t = np.tanh(GELU_R * (z + GELU_C * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * GELU_R * (1.0 + 3.0 * GELU_C * z * z)
    if kind == "silu":
        s = _sigmoid(z)
        return s * (1.0 + z * (1.0 - s))
    return np.ones_like(z)


def gemm_epilogue(a, b, bias=None, residual=None, kind="none"):
    """(out, z) of out = act(z) + residual, z = a @ b + bias."""
    z = a @ b
    if bias is not None:
        z = z + bias
    out = act(z, kind)
    return (out if residual is None else out + residual), z


def gemm_epilogue_grad(dz, a, b, z_in=None, kind_in="none", db_in=None, dbias_in=None):
    """(da, db, dbias) from the gradient dz at a @ b + bias."""
    da = dz @ b.T
    if kind_in != "none":
        da = da * act_grad(z_in, kind_in)
    db = a.T @ dz
    dbias = dz.sum(axis=0)
    return da, db if db_in is None else db + db_in, dbias if dbias_in is None else dbias + dbias_in


def route(logits, topk: int, norm_topk: bool):
    """(ids int [T][topk], gates [T][topk]): the topk largest logits of each
    row, ties to the lower id, and their softmax weights over all experts, or
    over the chosen ones."""
    T, E = logits.shape
    ids = np.zeros((T, topk), dtype=np.int64)
    gates = np.zeros((T, topk))
    for t in range(T):
        order = sorted(range(E), key=lambda e: (-logits[t, e], e))[:topk]
        p = np.exp(logits[t] - logits[t].max())
        ids[t] = order
        gates[t] = p[order] / (p[order].sum() if norm_topk else p.sum())
    return ids, gates


def moe_layer(x, ids, gates, w1, w2, kind="silu", gated=True):
    """out [T][hidden] = sum over a token's choices of gate * (h @ w2[e]), h =
    act(x @ w1[e]) or act(gate half) * up half; ids that name no expert add
    nothing."""
    out = np.zeros((x.shape[0], w2.shape[2]))
    inter = w2.shape[1]
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if not 0 <= e < w1.shape[0]:
                continue
            u = x[t] @ w1[e]
            h = act(u[:inter], kind)
            if gated:
                h = h * u[inter:]
            out[t] += float(gates[t, j]) * (h @ w2[e])
    return out


def grad_norm_clip(tensors, max_norm: float):
    """(norm, clipped tensors)."""
    norm = math.sqrt(math.fsum(float(np.sum(np.square(np.asarray(g, dtype=np.float64)))) for g in tensors))
    coef = 1.0 if math.isinf(max_norm) else min(1.0, max_norm / (norm + 1e-6))
    return norm, [np.asarray(g, dtype=np.float64) * coef for g in tensors]
