"""Plain float64 forms of the shared expert's operators, from their definitions, and the error bounds that the tests
hold the kernels to.  Tensors of any device; the results are float64 on that device.

Bounds.  A sum of K products of float32 or bfloat16 values, taken in float32 in any order, is off by at most
K 2^-23 sum|a b| (each addition rounds to, or truncates at, one part in 2^23 of a partial sum, which sum|a b| bounds;
bfloat16 products are exact, float32 ones lose at most 2^-23 more): ``sum_error``.  Functions of one value are taken to
FUNCTION relative error: float32 a few roundings and fits of 3e-7, bfloat16 an exponential whose argument, below 2^7, is off
by 2^-24 of itself.  One final rounding adds half a step of the output's type."""
import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
FUNCTION = {torch.bfloat16: 2.0 ** -16, torch.float32: 2.0 ** -20}


def sum_error(K, magnitude):
    return (K + 8) * 2.0 ** -23 * magnitude


def philox(counter, key):
    """Philox 4x32-10 of four counter words and two key words (ints)."""
    c, k = list(counter), list(key)
    low = 0xFFFFFFFF
    for _ in range(10):
        p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(p1 >> 32) ^ c[1] ^ k[0], p1 & low, (p0 >> 32) ^ c[3] ^ k[1], p0 & low]
        k = [(k[0] + 0x9E3779B9) & low, (k[1] + 0xBB67AE85) & low]
    return c


def threshold(p):
    return int(math.floor(p * 65536 + 0.5))


def keep_mask(seed, offset, rows, cols, p):
    """Truth values [rows, cols], and the factor of the kept ones."""
    t = threshold(p)
    seed, offset = seed % 2 ** 64, offset % 2 ** 64
    mask = torch.empty((rows, (cols + 7) // 8 * 8), dtype=torch.bool)
    for r in range(rows):
        for g in range((cols + 7) // 8):
            words = philox((g, r, offset & 0xFFFFFFFF, offset >> 32), (seed & 0xFFFFFFFF, seed >> 32))
            for i in range(8):
                mask[r, 8 * g + i] = ((words[i // 2] >> (16 * (i % 2))) & 0xFFFF) >= t
    return mask[:, :cols], (65536 / (65536 - t) if t < 65536 else 0.0)


def drop(v, mask):
    """D(v) for v float64; mask None: nothing is dropped."""
    if mask is None:
        return v
    keep, factor = mask
    return torch.where(keep.to(v.device), v * factor, torch.zeros_like(v))


def activation(g, act):
    """Value and slope."""
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    if act == "gelu":
        c = 0.5 * torch.erfc(-g / math.sqrt(2))
        return g * c, c + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    a, b = math.sqrt(2 / math.pi), 0.044715
    t = torch.tanh(a * (g + b * g ** 3))
    return g * (1 + t) / 2, (1 + t) / 2 + g * (1 - t * t) * a * (1 + 3 * b * g * g) / 2


def gated(x, wg, wu, act, mask=None):
    """(h, its bound without the final rounding, g, u, their bounds)."""
    function = FUNCTION[x.dtype]
    x, wg, wu = x.double(), wg.double(), wu.double()
    K = x.shape[1]
    g, u = x @ wg, x @ wu
    eg, eu = sum_error(K, x.abs() @ wg.abs()), sum_error(K, x.abs() @ wu.abs())
    a, slope = activation(g, act)
    # slopes vary by less than 1.2 per unit of g, and eg is far below one unit
    ea = (slope.abs() + 1.2 * eg) * eg + function * (a.abs() + eg)
    eh = ea * (u.abs() + eu) + a.abs() * eu
    return drop(a * u, mask), drop(eh, mask), g, u, eg, eu


def gated_backward(x, wg, wu, dh, act, mask=None, saved=None):
    """((dx, dwg, dwu), their bounds without the final rounding) for operands of x's type."""
    half, function = HALF_STEP[x.dtype], FUNCTION[x.dtype]
    x, wg, wu = x.double(), wg.double(), wu.double()
    K = x.shape[1]
    if saved is None:
        g, u = x @ wg, x @ wu
        eg, eu = sum_error(K, x.abs() @ wg.abs()), sum_error(K, x.abs() @ wu.abs())
    else:
        g, u = saved[0].double(), saved[1].double()
        eg = eu = torch.zeros_like(g)
    d = drop(dh.double(), mask)
    a, slope = activation(g, act)
    dg, du = d * u * slope, d * a
    # the second derivatives of the three activations stay below 1.2
    eslope, ea = 1.2 * eg + function * (1 + g.abs()), (slope.abs() + 1.2 * eg) * eg + function * (a.abs() + eg)
    edg = d.abs() * ((u.abs() + eu) * eslope + eu * slope.abs()) + 2 * half * dg.abs()
    edu = d.abs() * ea + 2 * half * du.abs()
    F, T = wg.shape[1], x.shape[0]
    dx = dg @ wg.t() + du @ wu.t()
    mag = (dg.abs() + edg) @ wg.abs().t() + (du.abs() + edu) @ wu.abs().t()
    edx = edg @ wg.abs().t() + edu @ wu.abs().t() + sum_error(2 * F, mag)
    out, err = [dx], [edx]
    for v, e in ((dg, edg), (du, edu)):
        out.append(x.t() @ v)
        err.append(x.abs().t() @ e + sum_error(T, x.abs().t() @ (v.abs() + e)))
    return out, err


def adapter(base, x, a, b, ids, scale, ranks):
    """(out, its bound without the final rounding)."""
    L, K, R = a.shape
    out, err = base.double().clone(), torch.zeros_like(base, dtype=torch.float64)
    for i in range(L):
        rows = torch.nonzero(ids == i)[:, 0]
        r = R if ranks is None else min(max(int(ranks[i]), 0), R)
        if rows.numel() == 0 or r == 0:
            continue
        xs, am, bm = x[rows].double(), a[i, :, :r].double(), b[i, :r].double()
        f = 1.0 if scale is None else float(scale[i])
        v = f * (xs @ am)
        # the scale, and keeping v to at least 16 bits in the second product
        ev = abs(f) * sum_error(K, xs.abs() @ am.abs()) + (2.0 ** -23 + 2.0 ** -16 * (base.dtype == torch.bfloat16)) * v.abs()
        out[rows] += v @ bm
        err[rows] = ev @ bm.abs() + sum_error(r + 1, (v.abs() + ev) @ bm.abs() + base[rows].double().abs())
    return out, err


def close(got, want, bound, name=""):
    """Every value of `got` within the bound and half a step of its type of `want`."""
    half = HALF_STEP[got.dtype]
    got = got.double()
    allowed = bound * (1 + half) + half * want.abs() * 1.0001 + 1e-38
    bad = ~((got - want).abs() <= allowed)
    bad &= ~(torch.isnan(got) & torch.isnan(want))
    if bool(bad.any()):
        at = tuple(int(v) for v in torch.nonzero(bad)[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} values off, first at {at}: got {float(got[at])}, "
                             f"want {float(want[at])}, allowed {float(allowed[at])}")
