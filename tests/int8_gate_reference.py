"""Plain float64 forms of the gate, its gradient and the int8 operators, for the tests (numpy, one
definition each, none of the library's code)."""
import numpy as np


def scores(l, score):
    l = l.astype(np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l))
        m = np.max(l, axis=1, keepdims=True)
        m = np.where(np.isneginf(m), 0.0, m)
        e = np.exp(l - m)
        z = e.sum(1, keepdims=True)
        return np.where(z == 0, 0.0, e / np.where(z == 0, 1.0, z))


def gate(l, k, score="softmax", bias=None, groups=1, topk_groups=1, group_top=2, renormalize=True, scale=1.0):
    """(ids [T, k], weights float64 [T, k], scores [T, E]); token by token."""
    T, E = l.shape
    s = scores(l, score)
    per = E // groups
    ids, w = np.zeros((T, k), np.int32), np.zeros((T, k))
    for t in range(T):
        c = s[t] + (0.0 if bias is None else bias.astype(np.float64))
        c = np.where(np.isneginf(l[t]), -np.inf, c)
        order_by = l[t].astype(np.float64) if bias is None else c
        allowed = np.ones(E, bool)
        if groups > 1:
            gs = []
            for g in range(groups):
                v = np.sort(c[g * per:(g + 1) * per])[::-1][:group_top]
                v = v[v > -np.inf]
                gs.append(v.sum() if v.size else -np.inf)
            kept = sorted(range(groups), key=lambda g: (-gs[g], g))[:topk_groups]
            allowed[:] = False
            for g in kept:
                allowed[g * per:(g + 1) * per] = True
        chosen = sorted(np.flatnonzero(allowed), key=lambda e: (-order_by[e], e))[:k]
        ids[t] = chosen
        v = s[t, chosen]
        total = v.sum() if renormalize else 1.0
        w[t] = scale * (v / total if total != 0 else 0.0 * v)
    return ids, w, s


def gate_backward(l, ids, dprobs, score, renormalize, scale):
    """dlogits float64 [T, E] by the chain rule with the full Jacobian of each token's scores; ids
    outside [0, E) are no slots."""
    T, E = l.shape
    s = scores(l, score)
    out = np.zeros((T, E))
    for t in range(T):
        sel = [(j, e) for j, e in enumerate(ids[t]) if 0 <= e < E]
        d = np.array([scale * np.float64(dprobs[t, j]) for j, _ in sel])
        v = np.array([s[t, e] for _, e in sel])
        if renormalize:
            S = v.sum()
            dv = (d - (d * v).sum() / S) / S if S != 0 else 0.0 * d
        else:
            dv = d
        ds = np.zeros(E)
        for (_, e), g in zip(sel, dv):
            ds[e] += g
        jac = np.diag(s[t] * (1 - s[t])) if score == "sigmoid" else np.diag(s[t]) - np.outer(s[t], s[t])
        out[t] = jac.T @ ds
    return out


def quantize(x):
    """(codes float64, scales float64) of rows: 127 x / max|x| to nearest even."""
    x = x.astype(np.float64)
    amax = np.abs(x).max(1, keepdims=True)
    safe = np.where(amax == 0, 1.0, amax)
    return np.rint(127.0 * x / safe), (amax / 127.0)[:, 0]


def matmul(rows, rows_scale, w, w_scale):
    return (rows.astype(np.float64) @ w.astype(np.float64)) * rows_scale.astype(np.float64)[:, None] * w_scale.astype(np.float64)


U = 2.0 ** -24           # half a step of float32


def ffn(rows, rows_scale, wg, sg, wu, su, wd, sd):
    """(y, slack): y of one expert's rows in float64, and what rounding in float32 on the way may move
    each output by, apart from its own final rounding.

    g and u carry three float32 roundings each; sigmoid(g) comes from exp2 of a rounded product (|g| U
    relative), a 1-ulp exp2 and a 1-ulp reciprocal (2 U each) and an addition: h is off by at most
    (16 + 2 |g|) U relative, its row maximum likewise.  A code can only differ (by one) where the real
    quotient lies closer to a half than that error allows; each such code moves an output by one step
    times its weight."""
    g = matmul(rows, rows_scale, wg, sg)
    u = matmul(rows, rows_scale, wu, su)
    h = g / (1 + np.exp(-g)) * u
    rel = (16 + 2 * np.abs(g).max(1, keepdims=True, initial=0)) * U
    codes, step = quantize(h)
    amax = np.abs(h).max(1, keepdims=True)
    q = 127.0 * h / np.where(amax == 0, 1, amax)
    near = np.abs(np.abs(q - np.floor(q)) - 0.5) <= 127 * 2 * rel
    wdv = np.abs(wd.astype(np.float64)) * sd.astype(np.float64)
    y = matmul(codes, step, wd, sd)
    slack = (near.astype(np.float64) @ wdv) * step[:, None] + (rel + 4 * U) * np.abs(y)
    return y, slack
