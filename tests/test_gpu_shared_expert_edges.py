"""The shared expert's operators on the GPU where their kernels change hands or their values stop being ordinary: few values,
infinities, the tails of the activations, operands that need all their bits, the limits between the ways a call runs."""
import math

import pytest

import shared_expert_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
mel = pytest.importorskip("moe_expert_layer_amd")

BF, F32 = torch.bfloat16, torch.float32
TYPES = pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
ACTS = pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def randn(seed, *shape, dtype=F32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(shape, generator=g)).to(dtype).cuda()


def poisoned(nbytes):
    """A workspace that holds NaN in every type."""
    return torch.full((max(nbytes, 1),), 0xFF, dtype=torch.uint8, device="cuda")


def adapter_ops(T, K, N, L, R, dtype):
    """base, x, A, B and ids, every adapter used and some rows without one."""
    ids = (torch.arange(T) % (L + 1) - 1).to(torch.int32).cuda()
    return (randn(1, T, N, dtype=dtype), randn(2, T, K, dtype=dtype), randn(3, L, K, R, dtype=dtype, scale=K ** -0.5),
            randn(4, L, R, N, dtype=dtype, scale=R ** -0.5), ids)


def add_adapters(base, x, a, b, ids, **kw):
    (T, K), (L, _, R), N = x.shape, a.shape, base.shape[1]
    ws = poisoned(mel.adapter_workspace_size(T, K, N, L, R, mel.BF16 if x.dtype == BF else mel.F32))
    return mel.adapter_add(base, x, a, b, ids, workspace=ws, **kw)


def coded(t):
    """Numbers that compare in place of infinities and NaN."""
    return torch.nan_to_num(t.double(), nan=7e40, posinf=1e40, neginf=-1e40)


# ------------------------------------------------------------------------------------------- adapters

@TYPES
@pytest.mark.parametrize("T", [25, 1000])
@pytest.mark.parametrize("K,R,L", [(1, 1, 16), (1, 3, 5), (2, 2, 2), (4, 1, 2), (6, 1, 3), (3, 2, 9), (1, 7, 3), (7, 1, 2)])
def test_adapters_of_fewer_than_eight_values(dtype, T, K, R, L):
    """Eight values from inside such an adapter on may pass the tensor's end, whichever adapter it is; single rows and tiles."""
    ops = adapter_ops(T, K, 19, L, R, dtype)
    ref.close(add_adapters(*ops), *ref.adapter(*ops, None, None), "adapter")


def _product(x, a):
    """x @ a in float64, term by term (no library product: zero times infinity is NaN where it stands)."""
    return (x.double()[:, :, None] * a.double()[None]).sum(1)


@TYPES
@pytest.mark.parametrize("T", [40, 1200])
@pytest.mark.parametrize("where", ["x", "a", "b", "all"])
def test_adapters_of_infinite_values(dtype, T, where):
    """Infinities give what the formula gives, by single rows and by tiles alike; finite results stay what they are."""
    K, N, L, R = 300, 40, 3, 12
    base, x, a, b, ids = adapter_ops(T, K, N, L, R, dtype)
    ranks = torch.tensor([R, 9, 1], dtype=torch.int32, device="cuda")
    scale = torch.tensor([0.5, 2.0, -1.0], device="cuda")
    if where in ("x", "all"):
        x[5, 7], x[6, 299], x[7, 100], x[11, 0] = INF, -INF, INF, -INF
        x[10, 1], x[10, 2] = INF, -INF
    if where in ("a", "all"):
        a[1, 250, 3], a[2, 20, 0] = INF, INF
    if where in ("b", "all"):
        b[0, 2, 5], b[0, 3, 6], b[0, 4, 6] = INF, INF, -INF
        b[1, 10, 7] = INF                                  # past the rank: counts for nothing
        b[2, :, 39] = -INF
    # one value of v that is zero, one that its first plane holds whole: zero times infinity is NaN, others are infinite
    x[13], x[17] = 0.0, 0.0
    x[17, 0] = 1.0
    a[0, 0] = 2.0                                          # row 17 has adapter 0
    want = base.double().clone()
    for i in range(L):
        rows, r = torch.nonzero(ids == i)[:, 0], int(ranks[i])
        v = scale[i].double() * _product(x[rows], a[i, :, :r])
        want[rows] += _product(v, b[i, :r])
    got = add_adapters(base, x, a, b, ids, scale=scale, ranks=ranks).double()
    odd = ~torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), ~odd), (torch.isfinite(got) == odd).nonzero()[:8]
    assert torch.equal(coded(got[odd]), coded(want[odd]))
    # where no infinity takes part the bound is that of finite operands
    zeroed = [torch.nan_to_num(t, posinf=0.0, neginf=0.0) for t in (x, a, b)]
    bound = ref.adapter(base, *zeroed, ids, scale, ranks)[1]
    ref.close(got[~odd].to(dtype), want[~odd], bound[~odd], "finite")
    inplace = base.clone()
    mel.adapter_add(inplace, x, a, b, ids, scale=scale, ranks=ranks, out=inplace)
    assert torch.equal(coded(inplace), coded(got))


@TYPES
@pytest.mark.parametrize("T,K,N,L,R", [(896, 40, 24, 3, 4), (897, 40, 24, 3, 4), (300, 64, 9001, 3, 4), (260, 24, 20000, 2, 3)])
def test_adapter_limits_of_single_rows(dtype, T, K, N, L, R):
    """The most single rows and one more; rows of more columns than one pass of a workgroup takes."""
    ops = adapter_ops(T, K, N, L, R, dtype)
    out = add_adapters(*ops)
    ref.close(out, *ref.adapter(*ops, None, None), "adapter")
    assert torch.equal(out[ops[4] < 0], ops[0][ops[4] < 0])
    inplace = ops[0].clone()
    add_adapters(inplace, *ops[1:], out=inplace)
    assert torch.equal(inplace, out)


# ------------------------------------------------------------------------------------------- gated block: values

@TYPES
@ACTS
@pytest.mark.parametrize("T", [1, 70])
def test_gated_gates_that_are_not_finite(dtype, act, T):
    """Finite factors whose product is past the type's range, and a NaN.  By the formulas act(+inf) is +inf; act(-inf) is
    -inf times zero, NaN."""
    x = torch.full((T, 1), 3e38, dtype=dtype, device="cuda")
    wg = torch.tensor([[2.0, -2.0, NAN, 0.0, 2.0]], dtype=dtype, device="cuda")
    wu = torch.tensor([[2.0 ** -120, 2.0 ** -120, 2.0 ** -120, 2.0 ** -120, -(2.0 ** -120)]], dtype=dtype, device="cuda")
    kept = torch.empty((2, T, 5), dtype=dtype, device="cuda")
    h = mel.gated_projection(x, wg, wu, activation=act, saved_gu=kept)
    want = torch.tensor([INF, NAN, NAN, 0.0, -INF], device="cuda").expand(T, 5)
    assert torch.equal(coded(h), coded(want)), h[0]
    gates = torch.tensor([INF, -INF, NAN, 0.0, INF], device="cuda").expand(T, 5)
    assert torch.equal(coded(kept[0]), coded(gates)), kept[0, 0]


@TYPES
@ACTS
def test_gated_backward_from_infinite_gates(dtype, act):
    """At g = +inf the slope is 1: dg = d u, and du = +inf.  A NaN gate gives NaN in its own column alone."""
    T = 5
    kept = torch.ones((2, T, 3), dtype=dtype, device="cuda")
    kept[0, :, 0], kept[0, :, 1], kept[0, :, 2], kept[1] = INF, 0.0, NAN, 2.0
    one = torch.ones((T, 3), dtype=dtype, device="cuda")
    x, w = torch.ones((T, 1), dtype=dtype, device="cuda"), torch.ones((1, 3), dtype=dtype, device="cuda")
    _, dwg, dwu = mel.gated_projection_backward(x, w, w, one, activation=act, saved_gu=kept)
    assert float(dwg[0, 0]) == 2.0 * T and float(dwg[0, 1]) == T and bool(torch.isnan(dwg[0, 2]))
    assert float(dwu[0, 1]) == 0.0 and bool(torch.isnan(dwu[0, 2]))
    if dtype == BF:                                        # float32 products of an infinite factor may be NaN
        assert float(dwu[0, 0]) == INF


def activation(g, act):
    """Value and slope in float64; the tanh form by the logistic function, (1 + tanh y) / 2 = s(2 y), since 1 + tanh y cancels
    to nothing far out."""
    if act != "gelu_tanh":
        return ref.activation(g, act)
    a, b = (8 / math.pi) ** 0.5, 0.044715
    z = a * (g + b * g ** 3)
    s = torch.sigmoid(z)
    return g * s, s + g * s * torch.sigmoid(-z) * a * (1 + 3 * b * g * g)


@ACTS
@pytest.mark.parametrize("T", [1, 70])
def test_activations_to_float32(act, T):
    """One product by 1, so that the gate is exact: what is left is the function.  Its roundings: the hardware's 2^y 2^-23
    and what puts the argument's rest back 2^-24; the reciprocal and 1 + e 2^-23 and 2^-24; three products 3 2^-24; gelu's
    fit 3e-7 < 5 2^-24 and its argument 2^-23: at most 15 2^-24, below 2^-20.  Down to where e^-z leaves float32's range."""
    low = {"silu": -80.0, "gelu": -12.5, "gelu_tanh": -9.5}[act]
    g = torch.cat([torch.linspace(low, 12.0, 4001), torch.logspace(-20, -1, 200), -torch.logspace(-20, -1, 200)]).cuda()[None]
    one = torch.ones((T, 1), device="cuda")
    h = mel.gated_projection(one, g, torch.ones_like(g), activation=act)
    want = activation(g.double(), act)[0].expand(T, -1)
    assert bool(((h.double() - want).abs() <= 2.0 ** -20 * want.abs()).all()), \
        float(((h.double() - want).abs() / want.abs()).max())
    # the slope, from the gradient's first factor: dwg = x dh u act'(g)
    dh = torch.zeros((T, g.shape[1]), device="cuda")
    dh[0] = 1.0
    dwg = mel.gated_projection_backward(one, g, torch.ones_like(g), dh, activation=act)[1]
    value, slope = activation(g.double(), act)
    # s + g s (1 - s) z' and its like, which cancel near the slope's zero; the second term has a few roundings more
    terms = slope.abs() + 2 * (slope - value / g.double()).abs()
    assert bool(((dwg.double() - slope).abs() <= 2.0 ** -19 * terms + 1e-37).all())


@ACTS
@pytest.mark.parametrize("T,H,F", [(2100, 520, 2056), (4100, 200, 1000)])
def test_dropout_in_the_largest_tiles(act, T, H, F):
    """bfloat16 products of 256 x 256 tiles with dropout, forward and both gradients.  The mask is that of dropout() with the
    same rng, whose own test compares it with the generator."""
    p = 0.3
    x = randn(1, T, H, dtype=BF)
    wg, wu = (randn(2 + i, H, F, dtype=BF, scale=H ** -0.5) for i in range(2))
    dh = randn(4, T, F, dtype=BF)
    rng = torch.tensor([2 ** 40 + 3, -9], dtype=torch.int64, device="cuda")
    keep = mel.dropout(torch.ones((T, F), dtype=BF, device="cuda"), p, rng) != 0
    mask = (keep, 65536 / (65536 - ref.threshold(p)))
    h, eh, *_ = ref.gated(x, wg, wu, act, mask)
    got = mel.gated_projection(x, wg, wu, activation=act, dropout=p, rng=rng)
    ref.close(got, h, eh, "h")
    assert bool((got[~keep] == 0).all())
    ws = poisoned(mel.gated_workspace_size(T, H, F, mel.BF16, backward=True))
    grads = mel.gated_projection_backward(x, wg, wu, dh, activation=act, dropout=p, rng=rng, workspace=ws)
    want, bounds = ref.gated_backward(x, wg, wu, dh, act, mask)
    for name, a, b, e in zip(("dx", "dw_gate", "dw_up"), grads, want, bounds):
        ref.close(a, b, e, name)


# ------------------------------------------------------------------------------------------- float32 products in planes


def hard(seed, *shape):
    """Values in [1, 1.25) whose second and third bfloat16 planes are as large as they come (2^-8.4 and 2^-17.4 at least): the
    loss of one product of planes changes a product of two of them by 2^-17.7 = 4.6e-6 or more."""
    g = torch.Generator().manual_seed(seed)
    j, m, n = (torch.randint(lo, hi, shape, generator=g).double() for lo, hi in ((0, 32), (64, 128), (16, 32)))
    return (1 + j / 128 + 2.0 ** -9 * (1 + m / 128) + 2.0 ** -18 * (1 + n / 32)).float().cuda()


def sparse(seed, rows, cols):
    """Rows of eight hard values at random places, zeros between them."""
    g = torch.Generator().manual_seed(seed)
    at = torch.stack([torch.randperm(cols, generator=g)[:8] for _ in range(rows)]).cuda()
    return torch.zeros((rows, cols), device="cuda").scatter_(1, at, hard(seed, rows, 8))


# sums of eight positive products: each addition 2^-23 of the sum, the products left out 2^-23, the roundings 2^-24
EIGHT = 10 * 2.0 ** -23


def relative(got, want):
    return float(((got.double() - want).abs() / want.abs()).max())


@pytest.mark.parametrize("T,H,F", [(65, 513, 130), (200, 1024, 328), (1000, 250, 1500)])
def test_float32_tiles_keep_every_plane(T, H, F):
    """Each product of planes at each place of K, in the tiles of the forward and of both gradients (in one launch and in
    parts): eight terms a sum, so that a lost product is larger than what the sum may be off by."""
    x, w = sparse(1, T, H), hard(2, H, F)
    kept = torch.empty((2, T, F), device="cuda")
    mel.gated_projection(x, w, w.flip(1).contiguous(), saved_gu=kept)
    assert relative(kept[0], x.double() @ w.double()) <= EIGHT
    assert relative(kept[1], x.double() @ w.flip(1).double()) <= EIGHT
    # silu at g = 0: value 0, slope 1/2, so with u = 2: dg = dh, du = 0
    kept[0], kept[1] = 0.0, 2.0
    dh = sparse(3, T, F)
    dx = mel.gated_projection_backward(x, w, w, dh, saved_gu=kept)[0]
    assert relative(dx, dh.double() @ w.double().t()) <= EIGHT
    dh, x = sparse(4, F, T).t().contiguous(), hard(5, T, H)
    dwg, dwu = mel.gated_projection_backward(x, w, w, dh, saved_gu=kept)[1:]
    assert relative(dwg, x.double().t() @ dh.double()) <= EIGHT
    assert bool((dwu == 0).all())


def test_float32_tiles_keep_24_bits():
    """Single products of operands that need all their bits, in every row and column of several tiles: what is left out is
    below 2^-23, one rounding."""
    T, F = 200, 300
    g = torch.Generator().manual_seed(9)
    x, w = ((1 + torch.randint(0, 2 ** 23, s, generator=g) / 2.0 ** 23).float().cuda() for s in ((T, 1), (1, F)))
    x[:6, 0] = torch.tensor([1 + 2.0 ** -23, 1 - 2.0 ** -24, 3.0000002, 1 / 3, 3.3e38, -3.4e38])
    w[0, :5] = torch.tensor([1 - 2.0 ** -24, 1 + 2.0 ** -23, 0.1, 1.0, 1e-3])
    w[0, 5:] *= 0.25                                       # no product of the largest value is past the range
    w[0, 1] = 1 - 2.0 ** -23
    kept = torch.empty((2, T, F), device="cuda")
    mel.gated_projection(x, w, w, saved_gu=kept)
    assert relative(kept[0], x.double() @ w.double()) <= 2.0 ** -22
    # dx and dWg as products of one term: at g = 0 with u = 1, dg = dh / 2 and du = 0
    kept[0], kept[1] = 0.0, 1.0
    want = 0.5 * (x.double() @ w.double())
    dx = mel.gated_projection_backward(x.new_zeros((T, F)), w.t().contiguous(), w.t().contiguous(), x,
                                       saved_gu=kept[:, :, :1].contiguous())[0]
    assert relative(dx, want) <= 2.0 ** -22
    dwg = mel.gated_projection_backward(x.t().contiguous(), w.new_ones((T, F)), w.new_ones((T, F)), w,
                                        saved_gu=kept[:, :1].contiguous())[1]
    assert relative(dwg, want) <= 2.0 ** -22


def test_float32_adapter_tiles_keep_every_plane():
    """v from eight terms, out from one: two sums' roundings."""
    T, K, N, L, R = 1000, 700, 264, 3, 40
    ids = (torch.arange(T) % L).to(torch.int32).cuda()
    x, a = sparse(6, T, K), hard(7, L, K, R)
    b = hard(8, L, R, N) * (torch.arange(N, device="cuda") % R == torch.arange(R, device="cuda")[:, None])
    out = mel.adapter_add(torch.zeros((T, N), device="cuda"), x, a, b, ids)
    for i in range(L):
        rows = ids == i
        assert relative(out[rows], (x[rows].double() @ a[i].double()) @ b[i].double()) <= EIGHT + 3 * 2.0 ** -23


@pytest.mark.parametrize("T", [6, 200])
@pytest.mark.parametrize("e", [-110, -118, -125, -130])
def test_float32_small_factors(T, e):
    """24 bits down to 2^-110, below that the nearest multiple of 2^-133 (and one rounding of the product)."""
    x, w = hard(11, T, 1) * 2.0 ** -100 * 2.0 ** (e + 100), hard(12, 1, 70) * 2.0 ** 60
    kept = torch.empty((2, T, 70), device="cuda")
    mel.gated_projection(x, w, w, saved_gu=kept)
    want = x.double() @ w.double()
    lost = 2.0 ** -134 * w.double() if e < -110 else 0.0
    assert bool(((kept[0].double() - want).abs() <= 2.0 ** -22 * want + lost).all())


# ------------------------------------------------------------------------------------------- replays, far offsets

@TYPES
def test_captured_adapters_by_tiles_follow_their_ids(dtype):
    """A captured call by tiles, replayed with other ids, ranks and factors: the plan is made anew each time."""
    T, L = 1100, 5
    base, x, a, b, ids = adapter_ops(T, 520, 264, L, 24, dtype)
    ranks, scale = torch.full((L,), 24, dtype=torch.int32, device="cuda"), torch.ones(L, device="cuda")
    mel.adapter_add(base, x, a, b, ids, scale=scale, ranks=ranks)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = mel.adapter_add(base, x, a, b, ids, scale=scale, ranks=ranks)
    for i in range(4):
        ids.copy_((torch.arange(T) * (2 * i + 1) // 7 % (L + 1) - 1).to(torch.int32) if i < 3 else torch.full((T,), L))
        ranks.copy_((torch.arange(L) * 7 + i) % 25)
        scale.copy_(torch.arange(L) - 1.5 * i)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, mel.adapter_add(base, x, a, b, ids, scale=scale, ranks=ranks))
        ref.close(got, *ref.adapter(base, x, a, b, ids, scale, ranks), i)


def test_offsets_past_32_bits():
    """Tensors of more than 2^31 values: the last rows are what they are alone."""
    T, N = 70000, 32768
    base = torch.zeros((T, N), dtype=BF, device="cuda")
    tail = randn(1, 100, N, dtype=BF)
    base[-100:] = tail
    rng = torch.tensor([77, 5], dtype=torch.int64, device="cuda")
    out = mel.dropout(base, 0.5, rng)
    bits = [ref.philox((g, T - 1, 5, 0), (77, 0)) for g in range(N // 8)]
    keep = torch.tensor([(w[i // 2] >> (16 * (i % 2)) & 0xFFFF) >= ref.threshold(0.5) for w in bits for i in range(8)]).cuda()
    assert torch.equal(out[-1], torch.where(keep, tail[-1] * 2, torch.zeros_like(tail[-1])))
    assert bool((out[:-100] == 0).all())
    del out
    K, L, R = 40, 2, 8
    x, a, b = randn(2, T, K, dtype=BF), randn(3, L, K, R, dtype=BF), randn(4, L, R, N, dtype=BF)
    ids = (torch.arange(T) % (L + 1) - 1).to(torch.int32).cuda()
    mel.adapter_add(base, x, a, b, ids, out=base)
    ref.close(base[-100:], *ref.adapter(tail, x[-100:], a, b, ids[-100:], None, None), "adapter")
    wg, wu = randn(5, K, N, dtype=BF, scale=0.1), randn(6, K, N, dtype=BF, scale=0.1)
    mel.gated_projection(x, wg, wu, out=base)
    want, bound, *_ = ref.gated(x[-100:], wg, wu, "silu")
    ref.close(base[-100:], want, bound, "h")
    dh = base
    dh[:-100] = 0                                          # gradients of the last rows alone
    dx, dwg, dwu = mel.gated_projection_backward(x, wg, wu, dh)
    grads, bounds = ref.gated_backward(x[-100:], wg, wu, dh[-100:], "silu")
    ref.close(dx[-100:], grads[0], bounds[0], "dx")
    assert bool((dx[:-100] == 0).all())
    ref.close(dwg, grads[1], bounds[1], "dw_gate")
    ref.close(dwu, grads[2], bounds[2], "dw_up")
