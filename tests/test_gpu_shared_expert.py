"""The shared expert's operators on the GPU against their float64 forms: dropout, the gated block with its gradient, the
low-rank adapters."""
import itertools

import pytest

import shared_expert_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
mel = pytest.importorskip("moe_expert_layer_amd")

BF, F32 = torch.bfloat16, torch.float32
TYPES = pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def randn(seed, *shape, dtype=F32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(shape, generator=g)).to(dtype).cuda()


def rng_of(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


def guarded(shape, dtype, value=7.0):
    """A tensor inside a larger one, and a check that nothing around it was written."""
    n = 1
    for s in shape:
        n *= s
    pad = 4096
    whole = torch.full((n + 2 * pad,), value, dtype=dtype, device="cuda")

    def check():
        assert bool((whole[:pad] == value).all()) and bool((whole[pad + n:] == value).all()), "written outside the output"

    return whole[pad:pad + n].view(shape), check


def poisoned(nbytes):
    """A workspace that holds NaN in every type."""
    return torch.full((max(nbytes, 1),), 0xFF, dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------------------------------- dropout

@TYPES
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols,p", [(1, 1, 0.5), (1, 8, 0.3), (3, 7, 0.1), (5, 9, 0.9), (17, 64, 0.05), (2, 1001, 0.5),
                                         (129, 40, 0.25), (4, 2048, 1e-4)])
def test_dropout(dtype, residual, rows, cols, p):
    x = randn(1, rows, cols, dtype=dtype)
    r = randn(2, rows, cols, dtype=dtype) if residual else None
    seed, offset = -5 + rows, 3 * 2 ** 32 + cols
    out, check = guarded((rows, cols), dtype)
    mel.dropout(x, p, rng_of(seed, offset), residual=r, out=out)
    mask = ref.keep_mask(seed, offset, rows, cols, p)
    want = ref.drop(x.double(), mask)
    bound = want.abs() * 2.0 ** -23                       # the factor and its product, in float32
    if residual:
        want = want + r.double()
        bound = bound + want.abs() * 2.0 ** -24
    ref.close(out, want, bound, "dropout")
    check()


@TYPES
def test_dropout_special_values(dtype):
    """Dropped infinities and NaN are zero, kept ones stay; p = 0 and p = 1; in place."""
    x = torch.full((16, 100), float("nan"), dtype=dtype, device="cuda")
    x[:, ::2] = float("inf")
    mask, _ = ref.keep_mask(9, 1, 16, 100, 0.5)
    out = mel.dropout(x, 0.5, rng_of(9, 1))
    mask = mask.cuda()
    assert bool((out[~mask] == 0).all())
    assert bool(torch.isinf(out[:, ::2][mask[:, ::2]]).all()) and bool(torch.isnan(out[:, 1::2][mask[:, 1::2]]).all())
    y = randn(3, 16, 100, dtype=dtype)
    assert torch.equal(mel.dropout(y, 0.0), y)
    assert torch.equal(mel.dropout(y, 1.0, rng_of(1, 1), residual=y), y)
    assert bool((mel.dropout(x, 1.0, rng_of(1, 1)) == 0).all())
    want = mel.dropout(y, 0.3, rng_of(4, 5), residual=y)
    z = y.clone()
    assert mel.dropout(z, 0.3, rng_of(4, 5), residual=z, out=z) is z and torch.equal(z, want)
    assert mel.dropout(y[:0], 0.3, rng_of(4, 5)).shape == (0, 100)


def test_dropout_unaligned_rows_and_many_groups():
    """A view that starts at an odd element; more groups than one workgroup takes."""
    flat = randn(5, 40 * 1000 + 1, dtype=BF)
    x = flat[1:].view(40, 1000)
    assert torch.equal(mel.dropout(x, 0.2, rng_of(1, 2)), mel.dropout(x.clone(), 0.2, rng_of(1, 2)))
    big = torch.ones((3000, 1024), dtype=BF, device="cuda")
    out = mel.dropout(big, 0.25, rng_of(7, 7))
    kept = out != 0
    assert torch.equal(out[kept], torch.full_like(out[kept], 4 / 3))
    # the share of kept values: 6 standard deviations of a binomial
    n = big.numel()
    assert abs(int(kept.sum()) - 0.75 * n) <= 6 * (n * 0.25 * 0.75) ** 0.5
    for i in (0, 1, 1499, 2999):
        row = out[i:i + 1].cpu()
        mask = _row_mask(7, 7, i, 1024, 0.25)
        assert torch.equal(row[0] != 0, mask)


def _row_mask(seed, offset, row, cols, p):
    bits = []
    for g in range(cols // 8):
        w = ref.philox((g, row, offset, 0), (seed, 0))
        bits += [(w[i // 2] >> (16 * (i % 2))) & 0xFFFF for i in range(8)]
    return torch.tensor(bits) >= ref.threshold(p)


# ------------------------------------------------------------------------------------------- gated block

def block_inputs(T, H, F, dtype, seed=0):
    x = randn(seed + 1, T, H, dtype=dtype)
    wg, wu = (randn(seed + 2 + i, H, F, dtype=dtype, scale=H ** -0.5) for i in range(2))
    return x, wg, wu


SIZES = [(1, 1, 1), (1, 8, 8), (2, 7, 9), (1, 64, 64), (3, 65, 63), (16, 72, 136), (17, 128, 100), (33, 200, 264),
         (64, 64, 128), (65, 127, 129), (127, 320, 72), (128, 256, 256), (129, 130, 257), (200, 520, 328), (257, 1001, 130),
         (300, 96, 1032), (1, 1000, 520), (5, 2056, 24), (31, 24, 2000),
         # few rows: every row block, K cut over workgroups and not, many columns
         (1, 4096, 264), (16, 2047, 65), (17, 1030, 8), (32, 777, 1003), (48, 600, 70), (64, 4100, 33), (3, 40, 8200),
         (16, 4100, 130), (63, 3001, 70), (2, 8190, 9), (8, 33, 4), (50, 2000, 3), (64, 31, 6),
         # the largest tiles, and more tiles than are resident at once
         (2100, 1000, 2056), (1500, 129, 4001)]


@TYPES
@pytest.mark.parametrize("T,H,F", SIZES)
def test_gated(dtype, T, H, F):
    x, wg, wu = block_inputs(T, H, F, dtype)
    act = ["silu", "gelu", "gelu_tanh"][(T + H + F) % 3]
    out, check = guarded((T, F), dtype)
    kept, check_kept = guarded((2, T, F), dtype)
    ws = poisoned(mel.gated_workspace_size(T, H, F, mel.BF16 if dtype == BF else mel.F32))
    mel.gated_projection(x, wg, wu, activation=act, saved_gu=kept, out=out, workspace=ws)
    h, eh, g, u, eg, eu = ref.gated(x, wg, wu, act)
    ref.close(kept[0], g, eg, "g")
    ref.close(kept[1], u, eu, "u")
    ref.close(out, h, eh, "h")
    check()
    check_kept()
    assert torch.equal(mel.gated_projection(x, wg, wu, activation=act), out)


@TYPES
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("T,H,F", [(5, 40, 72), (70, 64, 33)])
def test_gated_activations_and_dropout(dtype, act, T, H, F):
    x, wg, wu = block_inputs(T, H, F, dtype, seed=10)
    wg = wg * 6                                           # far into both tails of the activation
    mask = ref.keep_mask(11, 12, T, F, 0.3)
    out = mel.gated_projection(x, wg, wu, activation=act, dropout=0.3, rng=rng_of(11, 12))
    h, eh, *_ = ref.gated(x, wg, wu, act, mask)
    ref.close(out, h, eh, "h")


@TYPES
def test_gated_extreme_values(dtype):
    """Activations far out: no NaN for finite inputs, the limits of the functions."""
    big = torch.tensor([[-1e30, -200.0, -88.0, -20.0, -1e-30, 0.0, 1e-30, 20.0, 88.0, 200.0, 1e18]], dtype=dtype, device="cuda")
    F = big.shape[1]
    x = torch.ones((1, 1), dtype=dtype, device="cuda")
    one = torch.ones((1, F), dtype=dtype, device="cuda")
    for act in ("silu", "gelu", "gelu_tanh"):
        h = mel.gated_projection(x, big, one, activation=act)
        assert bool(torch.isfinite(h).all())
        assert torch.equal(h[0, -2:], big[0, -2:]) and bool((h[0, :2] == 0).all())
        dx, dwg, dwu = mel.gated_projection_backward(x, big, one, one, activation=act)
        assert bool(torch.isfinite(dwg).all()) and bool(torch.isfinite(dwu).all())
        assert torch.equal(dwg[0, -2:], one[0, -2:]) and bool((dwg[0, :2] == 0).all())


BWD_SIZES = [(1, 1, 1), (1, 8, 16), (2, 7, 9), (16, 72, 136), (33, 65, 63), (64, 128, 64), (65, 200, 100), (129, 257, 130),
             (130, 128, 264), (200, 136, 520), (300, 1000, 24), (7, 24, 1001),
             (2, 2050, 70), (30, 1000, 40), (61, 3000, 200),
             # both gradients in one launch in parts, and one after the other in tiles of every size
             (700, 136, 520), (22, 2880, 602), (1300, 1000, 72), (4001, 4001, 264), (2001, 4001, 4001)]


@TYPES
@pytest.mark.parametrize("saved", [False, True], ids=["recompute", "saved"])
@pytest.mark.parametrize("T,H,F", BWD_SIZES)
def test_gated_backward(dtype, saved, T, H, F):
    x, wg, wu = block_inputs(T, H, F, dtype, seed=20)
    dh = randn(29, T, F, dtype=dtype)
    act = ["silu", "gelu", "gelu_tanh"][(T + H + F) % 3]
    p = 0.25 if F % 2 == 0 else 0.0
    mask = ref.keep_mask(3, 4, T, F, p) if p else None
    kept = torch.stack([x @ wg, x @ wu]) if saved else None
    ws = poisoned(mel.gated_workspace_size(T, H, F, mel.BF16 if dtype == BF else mel.F32, backward=True))
    got = mel.gated_projection_backward(x, wg, wu, dh, activation=act, dropout=p, rng=rng_of(3, 4), saved_gu=kept,
                                        workspace=ws)
    want, bounds = ref.gated_backward(x, wg, wu, dh, act, mask, kept)
    for name, a, b, e in zip(("dx", "dw_gate", "dw_up"), got, want, bounds):
        ref.close(a, b, e, name)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gated_backward_against_differences(act):
    """float32 gradients against central differences of the library's own forward: with step 2^-6 the difference of a
    sum of h over 12 x 20 values, each off by about 2^-22, is off by 240 2^-22 2^5 = 2e-3 at most, and the third
    derivatives add step^2 / 6 times a few units, 1e-3."""
    T, H, F = 12, 9, 20
    x, wg, wu = block_inputs(T, H, F, F32, seed=40)
    dh = randn(44, T, F)
    rng = rng_of(8, 9)
    grads = mel.gated_projection_backward(x, wg, wu, dh, activation=act, dropout=0.2, rng=rng)

    def value(*ops):
        return float((mel.gated_projection(*ops, activation=act, dropout=0.2, rng=rng).double() * dh.double()).sum())

    step = 2.0 ** -6
    for which, (t, grad) in enumerate(zip((x, wg, wu), grads)):
        for at in [(0, 0), (t.shape[0] - 1, t.shape[1] - 1), (t.shape[0] // 2, t.shape[1] // 3)]:
            ops = [x, wg, wu]
            side = []
            for sign in (1, -1):
                moved = t.clone()
                moved[at] += sign * step
                ops[which] = moved
                side.append(value(*ops))
            got = float(grad[at])
            assert abs((side[0] - side[1]) / (2 * step) - got) <= 5e-3 * max(1.0, abs(got)), (which, at)


@TYPES
def test_gated_backward_without_tokens_and_dropped_infinities(dtype):
    x, wg, wu = block_inputs(0, 24, 40, dtype)
    dx, dwg, dwu = mel.gated_projection_backward(x, wg, wu, x.new_empty((0, 40)))
    assert dx.shape == (0, 24) and bool((dwg == 0).all()) and bool((dwu == 0).all())
    assert mel.gated_projection(x, wg, wu).shape == (0, 40)
    # an infinite dh at a dropped place changes nothing
    x, wg, wu = block_inputs(20, 24, 40, dtype, seed=50)
    dh = randn(55, 20, 40, dtype=dtype)
    mask, _ = ref.keep_mask(1, 2, 20, 40, 0.5)
    bad = torch.where(mask.cuda(), dh, torch.full_like(dh, float("inf")))
    for a, b in zip(*(mel.gated_projection_backward(x, wg, wu, d, dropout=0.5, rng=rng_of(1, 2)) for d in (dh, bad))):
        assert torch.equal(a, b)


def test_gated_float32_keeps_24_bits():
    """Products of float32 operands that need all their bits: (1 + 2^-23) (1 - 2^-23) and its neighbours."""
    a = torch.tensor([[1 + 2.0 ** -23, 1 - 2.0 ** -24, 3.0000002, 1 / 3, 3.3e38, -3.4e38]], device="cuda").t().contiguous()
    w = torch.tensor([[1 - 2.0 ** -24, 1 + 2.0 ** -23, 0.1, 1.0, 1e-3]], device="cuda")
    kept = torch.empty((2, 6, 5), device="cuda")
    mel.gated_projection(a, w, w, saved_gu=kept)
    want = a.double() @ w.double()
    # 2^-23 left out, a few roundings of partial sums
    assert bool(((kept[0].double() - want).abs() <= 2.0 ** -22 * want.abs()).all())


# ------------------------------------------------------------------------------------------- adapters

@TYPES
@pytest.mark.parametrize("T,K,N,L,R", [(1, 1, 1, 1, 1), (1, 64, 64, 2, 8), (3, 33, 9, 4, 3), (16, 128, 256, 5, 16),
                                       (17, 100, 130, 3, 13), (64, 520, 72, 40, 32), (200, 64, 1000, 7, 64), (90, 257, 65, 2, 100),
                                       (33, 1024, 40, 9, 128), (40, 48, 48, 3, 128), (300, 72, 520, 1, 4),
                                       # rows and adapters of a few values, whatever is last in its tensor
                                       (4, 3, 8, 1, 2), (4, 4, 9, 1, 2), (70, 5, 7, 2, 9), (6, 50, 11, 3, 9), (1, 7, 8, 1, 1),
                                       # beyond what single rows are used for: every width of rank and of tile
                                       (1, 14336, 264, 2, 128), (700, 4096, 1024, 9, 96), (130, 9000, 300, 3, 61),
                                       (2500, 1000, 4104, 1023, 32), (600, 5001, 2003, 5, 24), (900, 2053, 1021, 4, 13),
                                       (2000, 1030, 15, 2, 100), (3000, 513, 130, 1, 5),
                                       (1024, 40, 24, 3, 4), (1025, 40, 24, 3, 4), (70000, 5, 7, 3, 2)])
def test_adapter(dtype, T, K, N, L, R):
    base, x = randn(1, T, N, dtype=dtype), randn(2, T, K, dtype=dtype)
    a, b = randn(3, L, K, R, dtype=dtype, scale=K ** -0.5), randn(4, L, R, N, dtype=dtype, scale=R ** -0.5)
    g = torch.Generator().manual_seed(T)
    ids = torch.randint(-1, L, (T,), generator=g, dtype=torch.int32).cuda()
    if T > 2:
        ids[1], ids[2] = L, -7                            # out of range: no adapter
    scale = (0.5 + torch.rand(L, generator=g)).cuda()
    ranks = torch.randint(0, R + 1, (L,), generator=g, dtype=torch.int32).cuda()
    out, check = guarded((T, N), dtype)
    ws = poisoned(mel.adapter_workspace_size(T, K, N, L, R, mel.BF16 if dtype == BF else mel.F32))
    for s, r in ((scale, ranks), (None, None)):
        mel.adapter_add(base, x, a, b, ids, scale=s, ranks=r, out=out, workspace=ws)
        want, bound = ref.adapter(base, x, a, b, ids, s, r)
        ref.close(out, want, bound, "adapter")
        none = (ids < 0) | (ids >= L)
        assert torch.equal(out[none], base[none])
        check()
    inplace = base.clone()
    mel.adapter_add(inplace, x, a, b, ids, out=inplace)
    assert torch.equal(inplace, out)


@TYPES
@pytest.mark.parametrize("order", ["one", "segments", "mixed", "none"])
def test_adapter_many_rows(dtype, order):
    T, K, N, L, R = 1500, 200, 264, 12, 24
    base, x = randn(1, T, N, dtype=dtype), randn(2, T, K, dtype=dtype)
    a, b = randn(3, L, K, R, dtype=dtype, scale=K ** -0.5), randn(4, L, R, N, dtype=dtype, scale=R ** -0.5)
    t = torch.arange(T)
    ids = {"one": torch.full((T,), 3), "segments": t * L // T, "mixed": (t * 7919) % (L + 1) - 1,
           "none": torch.full((T,), -1)}[order].to(torch.int32).cuda()
    out = mel.adapter_add(base, x, a, b, ids)
    want, bound = ref.adapter(base, x, a, b, ids, None, None)
    ref.close(out, want, bound, order)


@TYPES
@pytest.mark.parametrize("T", [20, 1200])
def test_adapter_leaves_unread_what_lies_past_a_rank(dtype, T):
    """NaN in the columns and rows past an adapter's rank, in unused adapters, and in rows without one."""
    K, N, L, R = 96, 80, 4, 16
    base, x = randn(1, T, N, dtype=dtype), randn(2, T, K, dtype=dtype)
    a, b = randn(3, L, K, R, dtype=dtype), randn(4, L, R, N, dtype=dtype)
    ranks = torch.tensor([5, 0, 16, -3], dtype=torch.int32, device="cuda")
    ids = torch.tensor([0, 1, 3, -1] * (T // 4), dtype=torch.int32, device="cuda")
    want, bound = ref.adapter(base, x, a, b, ids, None, ranks)
    nan = float("nan")
    a[0, :, 5:], b[0, 5:] = nan, nan
    a[1:], b[1:] = nan, nan
    x[ids != 0] = nan
    ref.close(mel.adapter_add(base, x, a, b, ids, ranks=ranks), want, bound, "ranks")


def test_adapter_unaligned():
    T, K, N, L, R = 9, 64, 48, 3, 8

    def shifted(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        flat[1:] = t.reshape(-1)
        return flat[1:].view(t.shape)

    ops = [randn(1, T, N, dtype=BF), randn(2, T, K, dtype=BF), randn(3, L, K, R, dtype=BF), randn(4, L, R, N, dtype=BF)]
    ids = (torch.arange(T) % 4 - 1).to(torch.int32).cuda()
    want, bound = ref.adapter(*ops, ids, None, None)
    ref.close(mel.adapter_add(*[shifted(t) for t in ops], ids), want, bound, "unaligned")


# ------------------------------------------------------------------------------------------- together

def _shared_expert_step(x, wg, wu, wd, rng, rng2):
    """Forward and backward of a shared expert with dropout on h and on its output, beside the residual stream."""
    kept = torch.empty((2, x.shape[0], wg.shape[1]), dtype=x.dtype, device="cuda")
    h = mel.gated_projection(x, wg, wu, dropout=0.1, rng=rng, saved_gu=kept)
    out = mel.dropout(h @ wd, 0.2, rng2, residual=x)
    dy = mel.dropout(out, 0.2, rng2)                       # of the loss |out|^2 / 2: dout = out
    dh = dy @ wd.t().contiguous()
    dx, dwg, dwu = mel.gated_projection_backward(x, wg, wu, dh, dropout=0.1, rng=rng, saved_gu=kept)
    return out, dx + out, dwg, dwu


def test_training_step_together():
    """The step's results against the same steps in float64; tolerances: what each call is off by is tested above, here
    the bfloat16 roundings of five tensors in a row, 5 2^-8 of the norm at most."""
    T, H, F = 100, 128, 192
    x, wg, wu = block_inputs(T, H, F, BF, seed=60)
    wd = randn(66, F, H, dtype=BF, scale=F ** -0.5)
    got = _shared_expert_step(x, wg, wu, wd, rng_of(1, 1), rng_of(1, 2))
    m1, m2 = ref.keep_mask(1, 1, T, F, 0.1), ref.keep_mask(1, 2, T, H, 0.2)
    h = ref.gated(x, wg, wu, "silu", m1)[0]
    out = x.double() + ref.drop(h @ wd.double(), m2)
    dh = ref.drop(out, m2) @ wd.double().t()
    (dx, dwg, dwu), _ = ref.gated_backward(x, wg, wu, dh, "silu", m1)
    for name, a, b in zip(("out", "dx", "dwg", "dwu"), got, (out, dx + out, dwg, dwu)):
        assert float((a.double() - b).norm() / b.norm()) <= 5 * 2.0 ** -8, name


def test_serving_step_beside_the_expert_layer():
    """One decoded token and a small batch: the routed layer, the shared expert with its down projection's adapters."""
    H, F, E, L, R = 256, 256, 4, 3, 8
    wg, wu = (randn(70 + i, H, F, dtype=BF, scale=H ** -0.5) for i in range(2))
    wd = randn(72, F, H, dtype=BF, scale=F ** -0.5)
    eg, eu = (randn(73 + i, E, H, F, dtype=BF, scale=H ** -0.5) for i in range(2))
    ed = randn(75, E, F, H, dtype=BF, scale=F ** -0.5)
    a, b = randn(76, L, F, R, dtype=BF, scale=F ** -0.5), randn(77, L, R, H, dtype=BF, scale=R ** -0.5)
    for T in (1, 24):
        x = randn(78, T, H, dtype=BF)
        ids, probs = mel.router_gate(randn(79, T, E), 2)
        routed = mel.expert_forward(x, eg, eu, ed, ids, probs)
        h = mel.gated_projection(x, wg, wu)
        y = h @ wd
        who = (torch.arange(T) % (L + 1) - 1).to(torch.int32).cuda()
        shared = mel.adapter_add(y, h, a, b, who)
        ref.close(shared, *ref.adapter(y, h, a, b, who, None, None), "adapter")
        want, bound, *_ = ref.gated(x, wg, wu, "silu")
        ref.close(h, want, bound, "h")
        assert bool(torch.isfinite(shared + routed).all())


@pytest.mark.parametrize("T,H,F", [(1, 64, 128), (70, 72, 100), (300, 256, 384)])
def test_captured_step_draws_what_rng_says(T, H, F):
    """A captured forward and backward, replayed with eager work between; rng changes between the replays."""
    x, wg, wu = block_inputs(T, H, F, BF, seed=80)
    dh = randn(85, T, F, dtype=BF)
    rng = rng_of(5, 6)
    kept = torch.empty((2, T, F), dtype=BF, device="cuda")
    L, R = 3, 8
    a, b = randn(86, L, F, R, dtype=BF), randn(87, L, R, H, dtype=BF)
    ids = (torch.arange(T) % (L + 1) - 1).to(torch.int32).cuda()

    def step():
        h = mel.gated_projection(x, wg, wu, dropout=0.3, rng=rng, saved_gu=kept)
        y = mel.dropout(x, 0.2, rng, residual=x)
        return (h, y, mel.adapter_add(y, h, a, b, ids),
                *mel.gated_projection_backward(x, wg, wu, dh, dropout=0.3, rng=rng, saved_gu=kept),
                *mel.gated_projection_backward(x, wg, wu, dh, dropout=0.3, rng=rng))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for i in range(4):
        rng.copy_(rng_of(100 + i, 2 ** 40 * i))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in captured]
        for p, q in zip(got, step()):
            assert torch.equal(p, q)
        torch.cuda.synchronize()


def test_two_streams():
    """Two calls in flight, each with its own workspace, give what they give alone."""
    cases = [block_inputs(200, 264, 520, BF, seed=90), block_inputs(37, 264, 520, F32, seed=95)]
    alone = [mel.gated_projection(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = []
    for s, c in itertools.islice(zip(itertools.cycle(streams), itertools.cycle(cases)), 8):
        with torch.cuda.stream(s):
            outs.append(mel.gated_projection(*c))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, alone[i % 2])
