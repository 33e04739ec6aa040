"""The gate (scores, bias, groups, renormalised weights) and its gradient against plain float64 forms.

Tolerances.  U = 2^-24 is half a step of float32, x the distance of a logit from the largest (softmax) or
from 0 (sigmoid).  An exponential goes through a rounded difference, a product with a rounded log2 e and a
1-ulp exp2: (2.5 x + 2) U relative.  The sum of at most 1024 positive terms (16 in a lane, 64 lanes) adds 22
roundings to the terms' own error, a reciprocal 2, two products and the quotient one each: a weight is
within (5 x + 32) U of its value.  (Tokens decided in float64 are within 2 U.)  The gradient's
q = w (d - sum d w) has the same relative errors on each product: (2 x + 96) U times w (|d| + sum |d| w),
its exponentials being within 2 ulp.  bfloat16 outputs add 2^-8 of the value."""
import numpy as np
import pytest
import torch

import int8_gate_reference as ref
import moe_expert_layer_amd as mel

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mel.library()


def _logits(T, E, dtype, seed, grid=False):
    rng = np.random.default_rng(seed)
    l = (1.5 * rng.standard_normal((T, E))).astype(np.float32)
    if grid:
        l[::2] = np.round(l[::2] * 2) / 2               # equal logits
    t = torch.from_numpy(l).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    return t, t.float().numpy()


def _spread(l):
    """x of the tolerances.  Scores below exp(-70) < 2^-100 are float64's when chosen, and add less than
    2^-90 to a sum otherwise: larger distances count as 70."""
    f = np.where(np.isfinite(l), l, 0).astype(np.float64)
    return min(np.abs(f - f.max(1, keepdims=True)).max(initial=0), 70) + min(np.abs(f).max(initial=0), 70)


def _check(t, l, k, **kw):
    bias = kw.get("bias")
    dev = dict(kw)
    if bias is not None:
        dev["bias"] = torch.from_numpy(bias).cuda()
    ids, probs = mel.router_gate(t.cuda(), k, **dev)
    torch.cuda.synchronize()
    rids, rw, _ = ref.gate(l, k, **kw)
    assert np.array_equal(ids.cpu().numpy(), rids)
    tol = (5 * _spread(l) + 32) * U
    got = probs.cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - rw) <= tol * np.abs(rw) + 2.0 ** -149), np.abs(got - rw).max()
    return ids, probs


CASES = [(1, 1, 1, 1, 1), (1, 256, 8, 8, 4), (7, 3, 3, 1, 1), (33, 65, 5, 5, 2), (100, 64, 64, 1, 1), (50, 96, 7, 8, 3),
         (20, 200, 16, 4, 4), (9, 1024, 64, 16, 8), (5, 1023, 33, 3, 1), (300, 8, 2, 4, 2), (17, 16, 4, 16, 5),
         (40, 30, 3, 2, 1), (11, 512, 10, 512, 77), (0, 8, 2, 1, 1), (70, 8, 3, 2, 1), (70, 16, 3, 4, 2),
         (50, 32, 5, 8, 3), (50, 64, 6, 16, 4), (40, 36, 4, 2, 1), (40, 148, 7, 4, 3),
         (40, 248, 9, 8, 5), (40, 511, 9, 7, 2), (20, 1000, 12, 8, 3), (30, 250, 5, 50, 9), (30, 9, 3, 3, 2), (6, 1024, 64, 512, 40),
         (6, 1024, 7, 1024, 20), (20, 16, 16, 16, 16), (12, 8, 3, 8, 5), (50, 128, 8, 2, 1), (30, 512, 12, 8, 3), (6, 700, 9, 1, 1)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups,topk_groups", CASES)
def test_gate(T, E, k, groups, topk_groups, score):
    rng = np.random.default_rng(T * 7 + E)
    for dtype in ("f32", "bf16"):
        for with_bias in (False, True):
            for renorm, top in ((True, 2), (False, 1)):
                print(f"[gate] {T}x{E} k={k} g={groups}/{topk_groups} {score} {dtype} bias={with_bias}", flush=True)
                t, l = _logits(T, E, dtype, seed=T + E)
                bias = (0.1 * rng.standard_normal(E)).astype(np.float32) if with_bias else None
                _check(t, l, k, score=score, bias=bias, groups=groups, topk_groups=topk_groups, group_top=top,
                       renormalize=renorm, scale=2.5)


@pytest.mark.parametrize("E,k,groups,topk_groups,T", [(64, 8, 8, 3, 33000), (128, 8, 4, 2, 16500), (256, 8, 8, 4, 8200),
                                                     (250, 6, 2, 1, 8300), (500, 10, 1, 1, 8200), (64, 64, 1, 1, 33000),
                                                     (120, 6, 8, 3, 17000), (8, 2, 1, 1, 70001), (6, 3, 1, 1, 66000), (16, 4, 4, 2, 40000),
                                                     (30, 5, 1, 1, 20000), (64, 8, 8, 3, 9000), (128, 8, 4, 2, 5000),
                                                     (256, 8, 8, 4, 3001), (256, 8, 4, 2, 3000), (256, 6, 1, 1, 2500),
                                                     (500, 10, 1, 1, 2100), (120, 6, 8, 3, 5000), (74, 5, 2, 1, 6000),
                                                     (15, 3, 5, 2, 40000), (16, 16, 16, 16, 40000), (16, 8, 8, 6, 40000), (336, 8, 4, 2, 2100), (250, 6, 2, 1, 2500), (1024, 8, 32, 4, 2100), (64, 64, 1, 1, 9000)])
def test_gate_of_many_tokens(E, k, groups, topk_groups, T):
    """Enough tokens for the layouts that share a wave among more of them; against the same gate on
    slices of few tokens, whose layout is another: ids equal, weights within both layouts' bound."""
    for dtype in ("f32", "bf16"):
        for score in ("softmax", "sigmoid"):
            for with_bias in (False, True):
                print(f"[gate] {T}x{E} k={k} g={groups}/{topk_groups} {score} {dtype} bias={with_bias}", flush=True)
                t, l = _logits(T, E, dtype, seed=T, grid=dtype == "f32" and score == "sigmoid")
                x = t.cuda()
                kw = dict(score=score, groups=groups, topk_groups=topk_groups, scale=1.5, renormalize=with_bias)
                if with_bias:
                    kw["bias"] = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(E)).cuda()
                ids, probs = mel.router_gate(x, k, **kw)
                few = [mel.router_gate(x[i:i + 300], k, **kw) for i in range(0, T, 300)]
                assert torch.equal(ids, torch.cat([f[0] for f in few]))
                torch.testing.assert_close(probs, torch.cat([f[1] for f in few]), rtol=2 * (5 * _spread(l) + 32) * U, atol=0)
                at = np.random.default_rng(0).choice(T, 40, replace=False)
                kw["bias"] = kw["bias"].cpu().numpy() if with_bias else None
                rids, rw, _ = ref.gate(l[at], k, **kw)
                assert np.array_equal(ids.cpu().numpy()[at], rids)
                assert np.all(np.abs(probs.cpu().numpy()[at] - rw) <= (5 * _spread(l) + 32) * U * rw)


@pytest.mark.parametrize("E,k,groups,topk_groups", [(8, 3, 1, 1), (48, 6, 6, 2), (256, 8, 8, 4)])
def test_equal_logits_and_equal_biases(E, k, groups, topk_groups):
    """Ties go to the lower id, between groups to the lower group."""
    t, l = _logits(64, E, "f32", 3, grid=True)
    _check(t, l, k, groups=groups, topk_groups=topk_groups)
    z = np.zeros((4, E), np.float32)
    z[1, 1::2] = -0.0
    for bias in (None, np.full(E, 0.25, np.float32)):
        ids, _ = _check(torch.from_numpy(z), z, k, score="sigmoid", bias=bias, groups=groups, topk_groups=topk_groups)
        assert np.array_equal(ids.cpu().numpy(), np.tile(np.arange(k, dtype=np.int32), (4, 1)))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("groups", [1, 4])
def test_masked_experts_and_rows(score, with_bias, groups):
    """-inf logits are taken last with weight 0, whatever their bias; a row of them has ids 0 .. k-1 of
    the first groups and weights 0.  The type's lowest value is an ordinary, very small logit."""
    E, k = 16, 6
    t, l = _logits(32, E, "f32", 9)
    l = l.copy()
    l[:, 2:14] = -np.inf
    l[5] = -np.inf
    l[6, 1:] = -np.inf
    l[7] = np.finfo(np.float32).min
    bias = np.linspace(0.5, -0.5, E).astype(np.float32) if with_bias else None
    if with_bias:
        bias[3] = 9.0
        bias[15] = -np.inf
    ids, probs = _check(torch.from_numpy(l), l, k, score=score, bias=bias, groups=groups, topk_groups=groups // 2 or 1)
    assert np.all(probs[5].cpu().numpy() == 0)
    assert np.array_equal(ids[5].cpu().numpy(), np.arange(k))


@pytest.mark.parametrize("E,groups", [(8, 1), (64, 1), (64, 8), (250, 1), (256, 4), (1000, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_values_that_float32_cannot_tell_apart(E, groups, score):
    """Biases that make every expert's score plus bias one value up to float32's rounding: the order is
    float64's.  Every other token is an ordinary one."""
    rng = np.random.default_rng(E)
    t, l = _logits(9, E, "f32", 13)
    l = l.copy()
    l[1::2] = l[0]
    bias = (0.5 - ref.scores(l, score)[0]).astype(np.float32)
    l[2::2] = rng.standard_normal(l[2::2].shape).astype(np.float32)
    _check(torch.from_numpy(l), l, min(8, E // 2), score=score, bias=bias, groups=groups, topk_groups=max(1, groups // 2))


def test_float32_logits_one_step_apart():
    l = np.full((5, 64), 1.25, np.float32)
    for j in range(64):
        l[:, j] += np.float32((j * 37 % 64) * 2.0 ** -23)
    l[1] = -l[1]
    l[2] *= np.float32(2.0 ** -120)
    for groups in (1, 8):
        _check(torch.from_numpy(l), l, 8, groups=groups, topk_groups=min(groups, 4))


def test_nan_and_infinite_logits_stay_in_range():
    E, k = 40, 5
    for score in ("softmax", "sigmoid"):
        for bias in (None, torch.zeros(E, device="cuda")):
            for groups in (1, 8):
                t, l = _logits(16, E, "f32", 4)
                l = l.copy()
                l[0, 7] = np.nan
                l[1] = np.nan
                l[2, 3] = np.inf
                l[3, 3] = -np.nan
                ids, probs = mel.router_gate(torch.from_numpy(l).cuda(), k, score=score, bias=bias, groups=groups,
                                             topk_groups=min(groups, 4))
                ids = ids.cpu().numpy()
                assert ids.min() >= 0 and ids.max() < E
                assert all(len(set(r)) == k for r in ids)
                assert np.all(np.isnan(probs[1].cpu().numpy()))
                assert np.all(np.isfinite(probs[4:].cpu().numpy()))
                if groups == 1:
                    assert ids[0, 0] == 7 and ids[3, 0] == 3


def test_plain_softmax_agrees_with_the_plain_router():
    t, l = _logits(777, 128, "f32", 21, grid=True)
    a, b = mel.router_gate(t.cuda(), 8), mel.router_topk(t.cuda(), 8)
    assert torch.equal(a[0], b[0])
    torch.testing.assert_close(a[1], b[1], rtol=(5 * _spread(l) + 64) * U, atol=0)


# ------------------------------------------------------------------------------------------- gradient

def _check_backward(t, l, ids, dp, score, renorm, scale):
    got = mel.router_gate_backward(t.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(dp).cuda(), score=score,
                                   renormalize=renorm, scale=scale)
    torch.cuda.synchronize()
    assert got.dtype == t.dtype
    got = got.float().cpu().numpy().astype(np.float64)
    r = ref.gate_backward(l, ids, dp, score, renorm, scale)
    s = ref.scores(l, score)
    valid = (ids >= 0) & (ids < l.shape[1])
    sel = np.where(valid, np.take_along_axis(s, np.where(valid, ids, 0), 1), 0)
    d = np.where(valid, np.abs(dp.astype(np.float64) * scale), 0)
    total = sel.sum(1, keepdims=True)
    w = sel / np.where(total == 0, 1, total) if renorm else sel
    mag = np.zeros_like(r)
    dot = (d * w).sum(1)
    for t_ in range(l.shape[0]):
        for j in range(ids.shape[1]):
            if valid[t_, j]:
                mag[t_, ids[t_, j]] += w[t_, j] * (d[t_, j] + dot[t_])
        if score == "softmax" and not renorm:
            mag[t_] += s[t_] * dot[t_]
    # The reference's own rounding: a renormalised softmax's gradient is zero outside the selection, which
    # its Jacobian reaches as s_e sum_i ds_i s_i with |ds_i| s_i <= w_i (d_i + dot): a sum of k <= 64
    # products that cancel, each and every addition right to 2^-53, so off by at most (2 k + 6) 2^-53
    # < 2^-45 of s_e sum_i w_i (d_i + dot).
    own = 2.0 ** -45 * s * (w * (d + dot[:, None])).sum(1, keepdims=True)
    tol = (2 * _spread(l) + 96) * U * mag + 2.0 ** -120 + own
    if t.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(r)
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - r) <= tol), (np.abs(got - r) / tol).max()
    return got


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k,_g,_t", CASES)
def test_gate_backward(T, E, k, _g, _t, score, renorm):
    rng = np.random.default_rng(T + 3 * E)
    for dtype in ("f32", "bf16"):
        print(f"[gate backward] {T}x{E} k={k} {score} {dtype}", flush=True)
        t, l = _logits(T, E, dtype, seed=T + E + 1)
        ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32) if T else np.zeros((0, k), np.int32)
        dp = rng.standard_normal((T, k)).astype(np.float32)
        _check_backward(t, l, ids, dp, score, renorm, 2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gate_backward_masked_repeated_and_invalid_ids(score, renorm):
    t, l = _logits(24, 20, "f32", 31)
    l = l.copy()
    l[:, 12:] = -np.inf
    l[3] = -np.inf
    rng = np.random.default_rng(2)
    ids = np.stack([rng.permutation(20)[:6] for _ in range(24)]).astype(np.int32)
    ids[4] = 7                                            # one expert in every slot
    ids[5, 2] = ids[5, 0]
    ids[6, 1], ids[6, 3] = -1, 20
    ids[7] = -5                                           # no slot at all
    ids[8] = [12, 13, 14, 15, 16, 17]                     # masked experts alone
    dp = rng.standard_normal((24, 6)).astype(np.float32)
    got = _check_backward(torch.from_numpy(l), l, ids, dp, score, renorm, 1.0)
    assert np.all(got[3] == 0) and np.all(got[7] == 0) and np.all(got[8] == 0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gate_backward_against_differences(score, renorm):
    """Central differences of the gate's own weights, selection unchanged: with a step of 2^-5 the third
    derivative (at most 2 for these scores) leaves 2^-10 / 6 * 2 and the weights' rounding 2 * 8 U / 2^-4
    per slot."""
    T, E, k, h = 6, 12, 4, 2.0 ** -5
    t, l = _logits(T, E, "f32", 77)
    l = (np.round(l * 8) / 8 + np.arange(E, dtype=np.float32) * 2.0 ** -8).astype(np.float32)
    rng = np.random.default_rng(1)
    dp = rng.standard_normal((T, k)).astype(np.float32)
    kw = dict(score=score, renormalize=renorm, scale=1.0)
    ids, _ = mel.router_gate(torch.from_numpy(l).cuda(), k, **kw)
    got = mel.router_gate_backward(torch.from_numpy(l).cuda(), ids, torch.from_numpy(dp).cuda(), **kw).cpu().numpy()
    bound = (2.0 ** -10 / 3 + 2 * 40 * U / (2 * h)) * np.abs(dp).sum(1)
    checked = 0
    for e in range(E):
        moved = []
        for sgn in (1, -1):
            m = l.copy()
            m[:, e] += np.float32(sgn * h)
            i2, p2 = mel.router_gate(torch.from_numpy(m).cuda(), k, **kw)
            i2, p2 = i2.cpu().numpy(), p2.cpu().numpy().astype(np.float64)
            # the weights of the same experts, in the order of `ids` (nan: no longer chosen)
            at = np.full((T, k), np.nan)
            for r in range(T):
                for j, x in enumerate(ids[r].tolist()):
                    q = np.flatnonzero(i2[r] == x)
                    if q.size:
                        at[r, j] = p2[r, q[0]]
            moved.append(at)
        diff = ((moved[0] - moved[1]) / (2 * h) * dp).sum(1)
        ok = np.isfinite(diff)
        checked += ok.sum()
        assert np.all(np.abs(diff - got[:, e])[ok] <= bound[ok])
    assert checked > T * E // 2


# ------------------------------------------------------------------------------------------- how it is called

def test_gate_on_a_stream_and_in_a_graph():
    """Capture of gate and gradient, replayed on new logits with eager work between; also on a stream
    that is not the current one of the default."""
    t, _ = _logits(500, 64, "f32", 5)
    x = t.cuda()
    bias = torch.linspace(-0.1, 0.1, 64, device="cuda")
    dp = torch.randn(500, 6, device="cuda")
    kw = dict(score="sigmoid", renormalize=True, scale=2.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ids, p = mel.router_gate(x, 6, bias=bias, groups=8, topk_groups=4, **kw)
        mel.router_gate_backward(x, ids, dp, **kw)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gi, gp = mel.router_gate(x, 6, bias=bias, groups=8, topk_groups=4, **kw)
        gd = mel.router_gate_backward(x, gi, dp, **kw)
    for seed in range(3):
        x.copy_(_logits(500, 64, "f32", 50 + seed)[0])
        ei, ep = mel.router_gate(x, 6, bias=bias, groups=8, topk_groups=4, **kw)
        ed = mel.router_gate_backward(x, ei, dp, **kw)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(gi, ei) and torch.equal(gp, ep) and torch.equal(gd, ed)


def test_refusals():
    x = torch.zeros((4, 8), device="cuda")
    for kw in (dict(k=0), dict(k=9), dict(k=2, groups=3), dict(k=3, groups=4, topk_groups=1), dict(k=1, topk_groups=2),
               dict(k=1, group_top=3), dict(k=1, scale=float("inf")), dict(k=1, scale=float("nan"))):
        with pytest.raises(mel.MoeError):
            mel.router_gate(x, **kw)
    with pytest.raises(ValueError):
        mel.router_gate(x, 2, score="tanh")
    with pytest.raises(ValueError):
        mel.router_gate(x.half(), 2)
    with pytest.raises(ValueError):
        mel.router_gate(x[:, ::2], 2)
    with pytest.raises(ValueError):
        mel.router_gate(x, 2, bias=torch.zeros(7, device="cuda"))
    with pytest.raises(ValueError):
        mel.router_gate(x.cpu(), 2)
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        mel.router_gate_backward(x, ids, torch.zeros((4, 3), device="cuda"))


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gate_backward_of_very_small_sigmoids(dtype, renorm):
    """Selected logits about and far below the one whose sigmoid float32 can hold (-87), alone and beside ordinary
    ones.  Renormalised, what counts is their ratio.  Scores that float64 does not hold (below -709.78) are zero."""
    T, E, k = 96, 20, 6
    t, l = _logits(T, E, dtype, 41)
    rng = np.random.default_rng(6)
    l = l.copy()
    for i, level in enumerate((0, 60, 80, 87, 88, 89, 90, 100, 103, 120, 300, 700)):
        l[i::24] -= level                                # the whole token
        l[12 + i::24, ::2] -= level                      # every other expert
    l[5, 3:] = -800
    l[6] = -800
    l[7, ::3] = -np.inf
    t = torch.from_numpy(l).to(t.dtype)
    l = t.float().numpy()
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    dp = rng.standard_normal((T, k)).astype(np.float32)
    got = _check_backward(t, l, ids, dp, "sigmoid", renorm, 2.0)
    assert np.all(got[6] == 0)
    if renorm:
        low = [i for i in range(T) if i % 24 < 12 and i not in (5, 6)]
        assert np.all(np.abs(got[low]).max(1) > 0)


def test_gate_backward_of_two_small_sigmoids():
    """By hand: weights 1 / (1 + 1/e) and 1 / (1 + e) for logits one apart, far below 0; dlogits = w (1 - s) (d - sum d w)."""
    for top in (-80.0, -88.0, -90.0, -200.0):
        l = torch.tensor([[top, top - 1.0, 3.0]], device="cuda")
        ids = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
        got = mel.router_gate_backward(l, ids, torch.tensor([[1.0, -1.0]], device="cuda"), score="sigmoid").cpu().numpy()[0]
        a = 1 / (1 + np.exp(-1.0))
        want = 2 * a * (1 - a)
        assert np.all(np.abs(got - [want, -want, 0.0]) <= 64 * U * want)


def _chosen_with_a_nan(l, k, score, bias, groups, topk_groups, group_top):
    """The choice for one token with a NaN (or, with softmax, +inf) logit: the NaN counts as the largest, for its expert
    and for its group.  A softmax has no scores then: the logits are compared, without the bias."""
    if score == "softmax":
        c = l.astype(np.float64)
    else:
        with np.errstate(over="ignore"):
            c = 1 / (1 + np.exp(-l.astype(np.float64))) + (0 if bias is None else bias)
    by = c if bias is not None or score == "softmax" else l.astype(np.float64)
    c, by = np.where(np.isnan(c), 1e300, c), np.where(np.isnan(by), 1e300, by)
    c, by = np.where(np.isneginf(l), -np.inf, c), np.where(np.isneginf(l), -np.inf, by)
    per = l.size // groups
    top = [np.sort(c[g * per:(g + 1) * per])[::-1][:group_top] for g in range(groups)]
    sums = [v[v > -np.inf].sum() if (v > -np.inf).any() else -np.inf for v in top]
    kept = sorted(range(groups), key=lambda g: (-sums[g], g))[:topk_groups]
    return sorted((e for g in kept for e in range(g * per, (g + 1) * per)), key=lambda e: (-by[e], e))[:k]


@pytest.mark.parametrize("E,groups,topk_groups", [(40, 8, 3), (64, 8, 2), (64, 4, 1), (250, 5, 2), (24, 24, 5)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_a_nan_logit_is_chosen_in_any_group(E, groups, topk_groups, score, with_bias):
    """A NaN in a token's last, first or middle group (with softmax also +inf): its expert comes first, the weights
    are NaN (sigmoid without renormalising: its own alone), and the other tokens are as ever."""
    rng = np.random.default_rng(E + groups)
    T, k = 24, 4
    t, l = _logits(T, E, "f32", 17)
    l = l.copy()
    where = {}
    for i, e in enumerate((E - 1, 0, E // 2, E - 2, E // 3, 1)):
        value = [np.nan, -np.nan, np.inf][i % 3 if score == "softmax" else i % 2]
        l[3 * i, e] = value
        where[3 * i] = e
        if i >= 3:
            l[3 * i, rng.permutation(np.delete(np.arange(E), e))[:E // 4]] = -np.inf
    bias = (0.3 * rng.standard_normal(E)).astype(np.float32) if with_bias else None
    for top in (1, 2):
        for renorm in (True, False):
            ids, probs = mel.router_gate(torch.from_numpy(l).cuda(), k, score=score, groups=groups, topk_groups=topk_groups,
                                         bias=None if bias is None else torch.from_numpy(bias).cuda(), group_top=top,
                                         renormalize=renorm)
            ids, probs = ids.cpu().numpy(), probs.cpu().numpy()
            for row, e in where.items():
                assert ids[row].tolist() == _chosen_with_a_nan(l[row], k, score, bias, groups, topk_groups, top)
                assert ids[row, 0] == e
                nan = np.isnan(probs[row])
                assert nan.all() if renorm or score == "softmax" else nan.tolist() == [True] + [False] * (k - 1)
            rest = [r for r in range(T) if r not in where]
            rids, rw, _ = ref.gate(l[rest], k, score=score, bias=bias, groups=groups, topk_groups=topk_groups, group_top=top,
                                   renormalize=renorm)
            assert np.array_equal(ids[rest], rids)
            assert np.all(np.abs(probs[rest] - rw) <= (5 * _spread(l[rest]) + 32) * U * rw)


@pytest.mark.parametrize("E,T,groups", [(8, 300, 1), (64, 300, 1), (64, 33000, 1), (256, 300, 8), (256, 9000, 8), (1000, 100, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_weights_far_from_the_largest(E, T, groups, score, renorm):
    """Weights to float32's accuracy whatever the logits' distance.  A chosen expert's exponential is within 4 U: the
    argument's rounding is made good, a 1-ulp exp (2 U), with sigmoid an addition and a quotient.  Of k <= 8 chosen ones
    the sum adds 3 U, quotient and scale 2 U: 13 U, and 16 U here.  A softmax over all experts sums up to 1024 terms that
    are off by (2.5 x + 2) U each at the distance x, on average at most ln 1024, by up to 22 additions: 20 + 22 + 4 + 2 = 48 U."""
    rng = np.random.default_rng(E + T)
    l = (1.5 * rng.standard_normal((T, E))).astype(np.float32)
    far = rng.choice([0.0, 7.0, 20.0, 40.0, 60.0], T).astype(np.float32)[:, None]
    if score == "sigmoid":
        l -= far
    else:
        l[np.arange(T), rng.integers(0, E, T)] += far[:, 0]
    k = min(8, E // 2)
    kw = dict(score=score, renormalize=renorm, groups=groups, topk_groups=max(1, groups // 2), scale=1.5)
    ids, probs = mel.router_gate(torch.from_numpy(l).cuda(), k, **kw)
    at = np.arange(T) if T <= 300 else np.random.default_rng(1).choice(T, 300, replace=False)
    rids, rw, _ = ref.gate(l[at], k, **kw)
    assert np.array_equal(ids.cpu().numpy()[at], rids)
    err = np.abs(probs.cpu().numpy()[at].astype(np.float64) - rw) / rw
    print(f"[gate weights] E={E} T={T} {score} renorm={renorm}: {err.max() / U:.1f} U", flush=True)
    assert err.max() <= (48 if score == "softmax" and not renorm else 16) * U


@pytest.mark.parametrize("E,T", [(8, 50), (64, 50), (64, 33000)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("scale", [2.0 ** 126, 2.0 ** 100, 2.0 ** -100])
def test_any_finite_scale(E, T, score, renorm, scale):
    """Weights and gradient are those of scale 1 (at most 1 in size) times a power of two: exact, but for values that
    float32's subnormal steps of 2^-149 hold.  The scores, and the sums of the chosen ones, are small."""
    l = _logits(T, E, "f32", E)[0]
    if score == "sigmoid":
        l = l - 40.0
    l, k = l.cuda(), 4
    ids, one = mel.router_gate(l, k, score=score, renormalize=renorm)
    again, probs = mel.router_gate(l, k, score=score, renormalize=renorm, scale=scale)
    assert torch.equal(ids, again)
    torch.testing.assert_close(probs.double(), one.double() * scale, rtol=0, atol=2.0 ** -148)
    dp = torch.randn((T, k), generator=torch.Generator().manual_seed(1)).cuda()
    dp[:, 1] *= 8
    small = mel.router_gate_backward(l, ids, dp / 64, score=score, renormalize=renorm)
    large = mel.router_gate_backward(l, ids, dp / 64, score=score, renormalize=renorm, scale=scale)
    torch.testing.assert_close(large.double(), small.double() * scale, rtol=0, atol=2.0 ** -140)
