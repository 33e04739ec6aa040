"""The int8 operators against plain float64 forms.

Tolerances.  U = 2^-24 is half a step of float32.  A product's sum is exact in int32; its conversion and
two scalings are three roundings: 4 U relative, plus 2^-8 of the value for bfloat16 outputs.  For the
FFN see int8_gate_reference.ffn; the layer may round each slot's row to bfloat16 (2^-8 of probs * y; it
keeps 2^-11, to which test_layer_slots_are_summed_beyond_bfloat16 holds it) and sums k slots in float32 (k U
each) before its own final rounding."""
import numpy as np
import pytest
import torch

import int8_gate_reference as ref
import moe_expert_layer_amd as mel

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mel.library()


def _codes(rng, *shape):
    return rng.integers(-127, 128, shape, dtype=np.int8)


def _scale(rng, *shape, level=0.01):
    return (level * np.exp(0.5 * rng.standard_normal(shape))).astype(np.float32)


def _dev(*arrays):
    return [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in arrays]


def _host(t):
    return t.float().cpu().numpy().astype(np.float64)


# ------------------------------------------------------------------------------------------- quantiser

def _check_codes(t):
    codes, scales = mel.int8_quantize(t.cuda())
    torch.cuda.synchronize()
    q, s = ref.quantize(t.float().numpy())
    assert np.array_equal(codes.cpu().numpy().astype(np.float64), q)
    assert np.all(np.abs(scales.cpu().numpy() - s) <= U * s + 2.0 ** -149)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 4096), (17, 65), (64, 128), (9, 8192), (2, 20000),
                                       (33, 8191), (4, 8200), (700, 1000), (0, 8)])
def test_quantize(rows, cols, dtype):
    rng = np.random.default_rng(rows * 31 + cols)
    x = rng.standard_normal((rows, cols)) * np.exp(3 * rng.standard_normal((rows, 1)))
    print(f"[int8 quantize] {rows}x{cols} {dtype}", flush=True)
    _check_codes(torch.from_numpy(x).to(dtype))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(37, 256), (37, 257), (100, 40), (21, 1032), (21, 2047), (5, 2048), (6, 2056)])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_quantize_rows_at_any_address(rows, cols, shift, dtype):
    """Rows of each kernel's widths from a base that only its own type aligns."""
    rng = np.random.default_rng(rows + cols + shift)
    flat = torch.from_numpy(rng.standard_normal(rows * cols + shift)).to(dtype).cuda()
    x = flat[shift:].view(rows, cols)
    codes, scales = mel.int8_quantize(x)
    torch.cuda.synchronize()
    q, s = ref.quantize(_host(x))
    assert np.array_equal(codes.cpu().numpy().astype(np.float64), q)
    assert np.all(np.abs(scales.cpu().numpy() - s) <= U * s + 2.0 ** -149)


def test_quantize_more_rows_than_a_grid_has():
    """Rows of one column: the code is the value's sign times 127, the scale its 127th part."""
    x = torch.randn((1 << 25) + 5, 1, device="cuda").to(torch.bfloat16)
    codes, scales = mel.int8_quantize(x)
    assert torch.equal(codes.float(), 127 * torch.sign(x.float()))
    want = x.double().abs().view(-1) / 127
    assert bool(((scales.double() - want).abs() <= U * want + 2.0 ** -149).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantize_halves_extremes_and_zero_rows(dtype):
    """Quotients that are exactly a half (ties to even), float32 neighbours of a half, the largest and
    the smallest values of the type, and rows of zeros."""
    k = np.arange(-127, 127)
    half = np.concatenate([[127.0], k + 0.5])
    rows = [half * 2.0 ** e for e in (0, 100, 120, -100, -133)]
    near = np.concatenate([[127.0], np.nextafter(np.float32(k + 0.5), np.float32(200)).astype(np.float64)])
    rows += [near, near * 2.0 ** 120]
    third = np.concatenate([[3.0], 3.0 * (k + 0.5) / 127.0])
    rows += [third, np.zeros(255), np.linspace(-3.3e38, 3.3e38, 255), np.full(255, 1e-45)]
    _check_codes(torch.from_numpy(np.array(rows)).to(torch.float32).to(dtype))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantize_rows_that_are_not_finite(dtype):
    x = torch.randn((6, 300)).to(dtype)
    x[1, 5], x[2, 299], x[4, 0] = float("nan"), float("inf"), -float("inf")
    codes, scales = mel.int8_quantize(x.cuda())
    codes, scales = codes.cpu(), scales.cpu()
    for r in (1, 2, 4):
        assert torch.isnan(scales[r]) and not codes[r].any()
    q, _ = ref.quantize(x[[0, 3, 5]].float().numpy())
    assert np.array_equal(codes[[0, 3, 5]].numpy().astype(np.float64), q)


# ------------------------------------------------------------------------------------------- product

def _offsets(counts, gap=0):
    return np.concatenate([[gap], gap + np.cumsum(counts)]).astype(np.int32)


# The library picks the row tile (64, 128 or 256) and the cuts of K from M, the number of groups, K and N;
# the comments name what these sizes take.
PRODUCTS = [
    # counts of rows per group, K, N
    ([1], 128, 128),
    ([1, 0, 2], 256, 384),
    ([0, 0], 128, 256),
    ([40, 64, 65, 3], 384, 256),
    ([130, 0, 100, 161], 640, 512),
    ([300, 257, 1, 512], 256, 640),
    ([1000], 1152, 128),
    ([5] * 100, 128, 128),
    ([700, 0, 900], 128, 256),
    ([3] * 300, 256, 640),                                   # several tasks per workgroup, two steps each
    ([2, 0, 1] * 400, 128, 128),                             # more groups than one pass of the tile builder takes
    ([1] * 1024, 128, 128),
    ([2], 16384, 256),                                       # 64 rows, 16 cuts
    ([30, 0, 64, 7], 2048, 384),                             # cuts
    ([150, 100, 90], 1664, 256),                             # cuts of unequal length
    ([130, 0, 65, 65, 100, 30, 64, 66], 256, 4224),          # 128 rows
    ([130, 0, 65, 65, 100, 30, 64, 66], 384, 4224),
    ([65] * 30 + [0] * 5 + [130] * 5, 4096, 128),            # cuts
    ([300, 0, 257, 13, 130, 1, 32, 307], 256, 4224),         # 256 rows, half a column tile at the end
    ([300, 0, 257, 13, 130, 1, 32, 307], 384, 4224),         # 256 rows, an odd number of K pairs
    ([513, 256, 300], 384, 384),
    ([900, 0, 64, 2000], 896, 1152),
    ([700] * 12, 512, 512),
]


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts,K,N", PRODUCTS)
def test_matmul(counts, K, N, out_dtype):
    rng = np.random.default_rng(len(counts) + K + N)
    G, M = len(counts), int(np.sum(counts))
    E = min(G + 2, 1000)
    expert = rng.permutation(max(E, G))[:G].astype(np.int32) % E
    rows, w = _codes(rng, M, K), _codes(rng, E, K, N)
    rs, wsc = _scale(rng, M), _scale(rng, E, N)
    off = _offsets(counts)
    print(f"[int8 matmul] {counts[:6]} K={K} N={N}", flush=True)
    out = mel.grouped_matmul_int8(*_dev(rows, rs, off, expert, w, wsc), out_dtype=out_dtype)
    torch.cuda.synchronize()
    r = np.concatenate([ref.matmul(rows[a:b], rs[a:b], w[e], wsc[e]) for a, b, e in zip(off, off[1:], expert)]) \
        if M else np.zeros((0, N))
    tol = (4 * U + (BF if out_dtype == torch.bfloat16 else 0)) * np.abs(r)
    assert np.all(np.abs(_host(out) - r) <= tol)


@pytest.mark.parametrize("K", [256, 640])
def test_matmul_of_many_tasks(K):
    """256-row tiles, more than four tasks per workgroup (claimed two ahead); sampled rows of every tile."""
    rng = np.random.default_rng(K)
    counts, N = [5000, 3000, 0, 1, 4099, 2900, 6000, 3000], 4224
    M, off = sum(counts), _offsets(counts)
    rows, w, rs, wsc = _codes(rng, M, K), _codes(rng, 8, K, N), _scale(rng, M), _scale(rng, 8, N)
    out = mel.grouped_matmul_int8(*_dev(rows, rs, off, np.arange(8, dtype=np.int32), w, wsc))
    for a, b, e in zip(off, off[1:], range(8)):
        at = np.unique(np.concatenate([np.arange(a, b, 37), np.arange(max(a, b - 3), b)]))
        if at.size:
            r = ref.matmul(rows[at], rs[at], w[e], wsc[e])
            got = _host(out[torch.from_numpy(at).cuda()])
            assert np.all(np.abs(got - r) <= (4 * U + BF) * np.abs(r))


def test_matmul_largest_codes():
    """All codes -128: the largest sums that K allows here, beyond 2^24."""
    K, N = 4096, 128
    rows, w = np.full((70, K), -128, np.int8), np.full((1, K, N), -128, np.int8)
    one = np.ones(70, np.float32)
    out = mel.grouped_matmul_int8(*_dev(rows, one, np.array([0, 70], np.int32), np.zeros(1, np.int32), w,
                                        np.ones((1, N), np.float32)), out_dtype=torch.float32)
    assert torch.all(out == 16384.0 * K)


@pytest.mark.parametrize("counts", [[20, 30], [200, 90], [600, 333]])
def test_matmul_leaves_other_rows_alone_and_skips_bad_experts(counts):
    """Rows before the first and after the last group, and those of a group whose expert does not
    exist, keep what `out` held; the status word tells of the expert."""
    rng = np.random.default_rng(8)
    K, N, gap = 256, 256, 5
    M = sum(counts) + gap + 7 + 11
    off = _offsets(counts + [7], gap)
    expert = np.array([1, 0, 9], np.int32)
    rows, w, rs, wsc = _codes(rng, M, K), _codes(rng, 2, K, N), _scale(rng, M), _scale(rng, 2, N)
    out = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    mel.grouped_matmul_int8(*_dev(rows, rs, off, expert, w, wsc), out=out, workspace=ws)
    assert mel.device_status(ws) == 4
    got = _host(out)
    a, b = gap, gap + sum(counts)
    assert np.all(got[:a] == 7.0) and np.all(got[b:] == 7.0)
    for g in range(2):
        r = ref.matmul(rows[off[g]:off[g + 1]], rs[off[g]:off[g + 1]], w[expert[g]], wsc[expert[g]])
        assert np.all(np.abs(got[off[g]:off[g + 1]] - r) <= (4 * U + BF) * np.abs(r))


@pytest.mark.parametrize("rows,groups", [(90, 3), (90, 1500), (700, 64), (2000, 3000)])
def test_matmul_offsets_that_fall(rows, groups):
    """Offsets 0, M, 0, M, ...: every second group would hold all rows.  The first keeps them."""
    rng = np.random.default_rng(rows + groups)
    K, N = 256, 256
    off = np.array([rows * (g % 2) for g in range(groups + 1)], np.int32)
    a, w, rs, wsc = _codes(rng, rows, K), _codes(rng, 2, K, N), _scale(rng, rows), _scale(rng, 2, N)
    out = mel.grouped_matmul_int8(*_dev(a, rs, off, np.arange(groups, dtype=np.int32) % 2, w, wsc))
    r = ref.matmul(a, rs, w[0], wsc[0])
    assert np.all(np.abs(_host(out) - r) <= (4 * U + BF) * np.abs(r))


def test_matmul_of_thousands_of_groups():
    """Three passes of the tile builder, empty groups at their borders."""
    rng = np.random.default_rng(77)
    counts = rng.integers(0, 3, 2100)
    counts[[0, 1023, 1024, 2047, 2048, 2099]] = 0
    counts[[1022, 1025, 2049]] = [70, 130, 65]
    K, N, E = 128, 128, 9
    off, M = _offsets(counts), int(counts.sum())
    expert = rng.integers(0, E, len(counts)).astype(np.int32)
    a, w, rs, wsc = _codes(rng, M, K), _codes(rng, E, K, N), _scale(rng, M), _scale(rng, E, N)
    out = _host(mel.grouped_matmul_int8(*_dev(a, rs, off, expert, w, wsc)))
    row_expert = np.repeat(expert, counts)
    for e in range(E):
        at = row_expert == e
        r = ref.matmul(a[at], rs[at], w[e], wsc[e])
        assert np.all(np.abs(out[at] - r) <= (4 * U + BF) * np.abs(r))


@pytest.mark.parametrize("groups,rows", [(480, 1920), (481, 1920), (510, 1), (511, 1), (8, 32000), (1, 32512), (3, 65000)])
def test_matmul_about_the_largest_own_table(groups, rows):
    """Row tiles about the most that a workgroup lists for itself, few and many to a group; K one step."""
    rng = np.random.default_rng(groups + rows)
    K, N, E = 128, 128, 5
    off = np.concatenate([[0], np.sort(rng.integers(0, rows + 1, groups - 1)), [rows]]).astype(np.int32)
    expert = rng.integers(0, E, groups).astype(np.int32)
    a, w, rs, wsc = _codes(rng, rows, K), _codes(rng, E, K, N), _scale(rng, rows), _scale(rng, E, N)
    out = _host(mel.grouped_matmul_int8(*_dev(a, rs, off, expert, w, wsc)))
    row_expert = np.repeat(expert, np.diff(off))
    for e in range(E):
        at = row_expert == e
        r = ref.matmul(a[at], rs[at], w[e], wsc[e])
        assert np.all(np.abs(out[at] - r) <= (4 * U + BF) * np.abs(r))


def test_matmul_nan_scale_marks_its_row_alone():
    rng = np.random.default_rng(12)
    rows, w = _codes(rng, 70, 128), _codes(rng, 1, 128, 128)
    rs, wsc = _scale(rng, 70), _scale(rng, 1, 128)
    rs[3] = np.nan
    out = _host(mel.grouped_matmul_int8(*_dev(rows, rs, np.array([0, 70], np.int32), np.zeros(1, np.int32), w, wsc)))
    assert np.all(np.isnan(out[3])) and np.all(np.isfinite(np.delete(out, 3, 0)))


# ------------------------------------------------------------------------------------------- FFN, layer

def _weights(rng, E, H, F):
    return (_codes(rng, E, H, F), _scale(rng, E, F, level=3e-4), _codes(rng, E, H, F), _scale(rng, E, F, level=3e-4),
            _codes(rng, E, F, H), _scale(rng, E, H, level=3e-4))


FFNS = [
    ([1], 128, 128), ([3, 0, 5], 256, 384), ([60, 64, 1], 128, 640), ([150, 129], 384, 256), ([300, 0, 270], 256, 512),
    ([2000], 128, 128), ([1, 1], 2048, 256), ([400, 290], 128, 384), ([512, 31, 600], 384, 640),
    ([33], 1024, 4096),                                      # 64 rows, both products cut
    ([130, 0, 66, 1, 63] + [65] * 9 + [195, 0], 256, 1152),  # 128 rows
    ([200, 0, 190], 256, 4096),                              # 128 rows, the second product cut
    ([65] * 38 + [130, 0], 2048, 256),                       # 128 rows, the first product cut
    ([260, 0, 257, 3] + [130] * 36, 256, 640),               # 256 rows
    ([260, 0, 257, 3] + [130] * 36, 384, 640),               # 256 rows, odd numbers of K pairs
]


@pytest.mark.parametrize("counts,H,F", FFNS)
def test_ffn(counts, H, F):
    rng = np.random.default_rng(H + F + len(counts))
    G, M = len(counts), sum(counts)
    w = _weights(rng, G, H, F)
    rows, rs = _codes(rng, M, H), _scale(rng, M, level=0.02)
    off, expert = _offsets(counts), rng.permutation(G).astype(np.int32)
    print(f"[int8 ffn] {counts} H={H} F={F}", flush=True)
    out = _host(mel.grouped_ffn_int8(*_dev(rows, rs, off, expert, *w)))
    for a, b, e in zip(off, off[1:], expert):
        if b > a:
            y, slack = ref.ffn(rows[a:b], rs[a:b], *[t[e] for t in w])
            assert np.all(np.abs(out[a:b] - y) <= slack + BF * (np.abs(y) + slack))


LAYERS = [(2600, 256, 640, 40, 2), (2600, 384, 640, 40, 2), (520, 256, 1152, 16, 2), (1, 2048, 1024, 8, 2), (64, 256, 256, 16, 4), (65, 256, 256, 16, 4), (32, 128, 256, 1023, 8), (256, 128, 128, 3, 1),
          (1, 256, 384, 4, 2), (3, 128, 128, 1, 1), (40, 256, 256, 8, 3), (150, 128, 384, 3, 3), (900, 256, 256, 5, 2),
          (64, 128, 128, 100, 8)]


def _layer_ref(x_codes, x_scale, w, ids, probs):
    T, k = ids.shape
    H = w[4].shape[2]
    r, tol = np.zeros((T, H)), np.zeros((T, H))
    for e in range(w[0].shape[0]):
        t, j = np.nonzero(ids == e)
        if t.size:
            y, slack = ref.ffn(x_codes[t], x_scale[t], *[a[e] for a in w])
            p = probs[t, j].astype(np.float64)[:, None]
            np.add.at(r, t, p * y)
            np.add.at(tol, t, p * (slack + (BF + 2 * k * U) * (np.abs(y) + slack)))
    return r, tol + BF * (np.abs(r) + tol)


@pytest.mark.parametrize("T,H,F,E,k", LAYERS)
def test_layer(T, H, F, E, k):
    rng = np.random.default_rng(T + H + E)
    w = _weights(rng, E, H, F)
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).bfloat16()
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    probs = rng.dirichlet(np.ones(k), T).astype(np.float32)
    q, s = ref.quantize(x.float().numpy())
    r, tol = _layer_ref(q, s, w, ids, probs)
    wd, idd, pd = _dev(*w), *_dev(ids), *_dev(probs)
    print(f"[int8 layer] T={T} H={H} F={F} E={E} k={k}", flush=True)
    out = mel.expert_forward_int8(x.cuda(), None, *wd, idd, pd)
    assert np.all(np.abs(_host(out) - r) <= tol + 4 * U * np.abs(r))
    # the same from codes the caller quantised, and again on a workspace the caller keeps: bitwise
    codes, scales = mel.int8_quantize(x.cuda())
    prob = mel.problem(T, H, F, E, k, mel.INT8, 0, mel.FLAG_QUANTIZE_X)
    ws = torch.full((mel.workspace_size(prob),), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(mel.expert_forward_int8(codes, scales, *wd, idd, pd, workspace=ws), out)
    assert torch.equal(mel.expert_forward_int8(x.cuda(), None, *wd, idd, pd, workspace=ws), out)


def test_no_tokens_and_no_rows():
    rng = np.random.default_rng(0)
    w = _dev(*_weights(rng, 2, 128, 256))
    i32 = dict(dtype=torch.int32, device="cuda")
    x = torch.empty((0, 128), dtype=torch.bfloat16, device="cuda")
    out = mel.expert_forward_int8(x, None, *w, torch.empty((0, 2), **i32), torch.empty((0, 2), device="cuda"))
    assert out.shape == (0, 128)
    off, ex = torch.zeros(3, **i32), torch.arange(2, **i32)
    y = mel.grouped_ffn_int8(torch.empty((0, 128), dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda"), off, ex, *w)
    assert y.shape == (0, 128)
    # rows, but no group holds any
    y = torch.full((5, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    mel.grouped_ffn_int8(torch.ones((5, 128), dtype=torch.int8, device="cuda"), torch.ones(5, device="cuda"), off, ex, *w, out=y)
    assert torch.all(y == 3.0)


def test_one_expert_in_every_slot_of_a_token():
    """A token may name an expert twice: both slots count."""
    rng = np.random.default_rng(5)
    T, H, F, E, k = 30, 128, 128, 3, 2
    w = _weights(rng, E, H, F)
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).bfloat16()
    ids = np.full((T, k), 1, np.int32)
    ids[::3] = [[0, 2]]
    probs = rng.dirichlet(np.ones(k), T).astype(np.float32)
    q, s = ref.quantize(x.float().numpy())
    r, tol = _layer_ref(q, s, w, ids, probs)
    out = _host(mel.expert_forward_int8(x.cuda(), None, *_dev(*w), *_dev(ids, probs)))
    assert np.all(np.abs(out - r) <= tol + 4 * U * np.abs(r))


def test_two_streams_at_once():
    """Two layer calls in flight on two streams, each on its own workspace."""
    rng = np.random.default_rng(7)
    T, H, F, E, k = 400, 512, 512, 4, 2
    w = _dev(*_weights(rng, E, H, F))
    xs = [torch.randn((T, H), device="cuda").bfloat16() for _ in range(2)]
    ids = torch.from_numpy(np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)).cuda()
    probs = torch.softmax(torch.randn((T, k), device="cuda"), 1)
    alone = [mel.expert_forward_int8(x, None, *w, ids, probs) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    outs = []
    for _ in range(3):
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                outs.append(mel.expert_forward_int8(x, None, *w, ids, probs))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, alone[i % 2])


def test_layer_drops_bad_ids_and_marks_nan_tokens():
    rng = np.random.default_rng(6)
    T, H, F, E, k = 50, 128, 256, 4, 2
    w = _weights(rng, E, H, F)
    x = torch.randn((T, H), dtype=torch.float32).bfloat16()
    x[9, 3] = float("nan")
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    ids[4] = [E, -1]
    probs = np.full((T, k), 0.5, np.float32)
    prob = mel.problem(T, H, F, E, k, mel.INT8, 0, mel.FLAG_QUANTIZE_X)
    ws = torch.empty(mel.workspace_size(prob), dtype=torch.uint8, device="cuda")
    out = _host(mel.expert_forward_int8(x.cuda(), None, *_dev(*w), *_dev(ids, probs), workspace=ws))
    assert mel.device_status(ws) == 4
    assert np.all(out[4] == 0) and np.all(np.isnan(out[9])) and np.all(np.isfinite(np.delete(out, 9, 0)))


@pytest.mark.parametrize("T", [1, 5, 100])
def test_layer_rows_do_not_depend_on_the_batch(T):
    """A token's output is the same alone (partial sums, one launch of preparation), in a small batch and
    in a large one (another tile height and another cut of K): the sums are exact."""
    rng = np.random.default_rng(T)
    H, F, E, k = 512, 384, 4, 2
    w = _dev(*_weights(rng, E, H, F))
    x = torch.randn((700, H), device="cuda").bfloat16()
    ids = torch.from_numpy(np.stack([rng.permutation(E)[:k] for _ in range(700)]).astype(np.int32)).cuda()
    probs = torch.softmax(torch.randn((700, k), device="cuda"), 1)
    whole = mel.expert_forward_int8(x, None, *w, ids, probs)
    part = mel.expert_forward_int8(x[:T].contiguous(), None, *w, ids[:T].contiguous(), probs[:T].contiguous())
    assert torch.equal(part, whole[:T])


def test_gate_then_int8_layer_in_a_graph():
    """The serving step: gate on the logits, the layer on int8 weights; captured, and replayed on other
    tokens with eager calls and synchronizations between."""
    rng = np.random.default_rng(3)
    T, H, F, E, k = 96, 256, 256, 16, 4
    w = _dev(*_weights(rng, E, H, F))
    bias = torch.linspace(-0.05, 0.05, E, device="cuda")
    x = torch.randn((T, H), device="cuda").bfloat16()
    logits = torch.randn((T, E), device="cuda")

    def step():
        ids, probs = mel.router_gate(logits, k, score="sigmoid", bias=bias, groups=4, topk_groups=2, scale=1.5)
        return mel.expert_forward_int8(x, None, *w, ids, probs)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for _ in range(3):
        x.copy_(torch.randn((T, H), device="cuda"))
        logits.copy_(torch.randn((T, E), device="cuda"))
        eager = step()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


def test_train_step_of_the_gate_through_the_layer():
    """Gate, layer, backward, gate backward: the gradient of sum(dout * out) with respect to the logits
    against float64 differences of the plain form (bf16 layer: 2e-2 of the largest gradient)."""
    import oracle
    import synth
    from synth import device as dv
    oracle.build()
    T, H, F, E, k = 24, 128, 128, 6, 2
    inp = synth.make_layer(T=T, H=H, F=F, E=E, k=k, dtype="bf16", seed=4)
    d = dv.layer(inp)
    rng = np.random.default_rng(2)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    kw = dict(score="sigmoid", renormalize=True, scale=2.0)
    ids, probs = mel.router_gate(torch.from_numpy(logits).cuda(), k, bias=torch.zeros(E, device="cuda"), **kw)
    dout = synth.make_dout(inp)
    grads = mel.expert_backward(d.x, d.w_gate, d.w_up, d.w_down, ids, probs, dv.tensor(dout))
    dl = mel.router_gate_backward(torch.from_numpy(logits).cuda(), ids, grads[4], **kw)
    inp.expert_ids, inp.probs = ids.cpu().numpy(), probs.cpu().numpy()
    ref_dprobs = oracle.backward(inp, dout)[4]
    r = ref.gate_backward(logits, inp.expert_ids, ref_dprobs, "sigmoid", True, 2.0)
    assert np.abs(_host(dl) - r).max() <= 2e-2 * np.abs(r).max()


def test_refusals():
    rows, w = torch.zeros((4, 128), dtype=torch.int8, device="cuda"), torch.zeros((2, 128, 128), dtype=torch.int8, device="cuda")
    rs, wsc = torch.ones(4, device="cuda"), torch.ones((2, 128), device="cuda")
    off, ex = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda"), torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        mel.grouped_matmul_int8(rows, rs, off, ex, w, wsc, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        mel.grouped_matmul_int8(rows, rs[:3], off, ex, w, wsc)
    with pytest.raises(ValueError):
        mel.grouped_matmul_int8(rows, rs, off, ex, w.transpose(1, 2), wsc)
    with pytest.raises(mel.MoeError):
        mel.grouped_matmul_int8(rows[:, :64].contiguous(), rs, off, ex, w[:, :64].contiguous(), wsc)
    with pytest.raises(mel.MoeError):
        mel.grouped_matmul_int8(rows, rs, off, ex, torch.zeros(2 * 128 * 128 + 4, dtype=torch.int8, device="cuda")[4:].view(2, 128, 128), wsc)
    with pytest.raises(ValueError):
        mel.grouped_matmul_int8(rows, rs, off, ex, w, wsc, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        mel.int8_quantize(torch.zeros((2, 8), dtype=torch.float16, device="cuda"))
    x = torch.zeros((2, 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        mel.expert_forward_int8(x, torch.ones(2, device="cuda"), w, wsc, w, wsc, w, wsc,
                                torch.zeros((2, 1), dtype=torch.int32, device="cuda"), torch.ones((2, 1), device="cuda"))


# ------------------------------------------------------------------------------------------- offsets that fall

def _row_experts(off, expert, E, M):
    """Each row's expert, -1 for none: a group begins no earlier than any offset before it."""
    held, reached = np.full(M, -1), 0
    for g in range(len(expert)):
        reached = max(reached, min(max(off[g], 0), M))
        if 0 <= expert[g] < E:
            held[reached:max(reached, min(max(off[g + 1], 0), M))] = expert[g]
    return held


FALLING = [
    ([40, 10, 60], [1, 0], 60),
    ([5, 0, 10], [0, 1], 12),
    ([5, 3, 30, 8, 50], [0, 1, 0, 1], 55),                   # falls twice
    ([0, 20, 5, 30], [9, 0, 1], 33),                         # the first group's expert does not exist
    ([30, 2, 40, 33, 64], [1, 9, 0, 1], 70),                 # a later one's does not
    ([-3, 6, 2, 500], [1, 0, 1], 50),                        # offsets outside the rows
    ([64, 64, 0, 64], [0, 1, 0], 64),                        # no row is held
]


# 8192 values of K are cut for so few rows (the sums are joined by a launch of their own), 256 are not.
@pytest.mark.parametrize("K", [256, 2048, 8192])
@pytest.mark.parametrize("off,expert,M", FALLING)
def test_matmul_rows_of_offsets_that_fall(off, expert, M, K):
    rng = np.random.default_rng(K + M)
    N = 256
    rows, w, rs, wsc = _codes(rng, M, K), _codes(rng, 2, K, N), _scale(rng, M), _scale(rng, 2, N)
    held = _row_experts(off, expert, 2, M)
    for dtype in (torch.bfloat16, torch.float32):
        print(f"[int8 matmul] offsets {off} K={K} {dtype}", flush=True)
        out = torch.full((M, N), 7.0, dtype=dtype, device="cuda")
        ws = torch.full((64 << 20,), 85, dtype=torch.uint8, device="cuda")
        mel.grouped_matmul_int8(*_dev(rows, rs, np.array(off, np.int32), np.array(expert, np.int32), w, wsc), out=out,
                                out_dtype=dtype, workspace=ws)
        got = _host(out)
        assert np.all(got[held < 0] == 7.0)
        for e in range(2):
            at = held == e
            r = ref.matmul(rows[at], rs[at], w[e], wsc[e])
            assert np.all(np.abs(got[at] - r) <= (4 * U + (BF if dtype == torch.bfloat16 else 0)) * np.abs(r))


@pytest.mark.parametrize("H,F", [(256, 256), (1024, 4096)])      # whole products, both products cut
@pytest.mark.parametrize("off,expert,M", FALLING)
def test_ffn_rows_of_offsets_that_fall(off, expert, M, H, F):
    rng = np.random.default_rng(H + M)
    w = _weights(rng, 2, H, F)
    rows, rs = _codes(rng, M, H), _scale(rng, M, level=0.02)
    held = _row_experts(off, expert, 2, M)
    print(f"[int8 ffn] offsets {off} H={H} F={F}", flush=True)
    out = torch.full((M, H), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((256 << 20,), 85, dtype=torch.uint8, device="cuda")
    mel.grouped_ffn_int8(*_dev(rows, rs, np.array(off, np.int32), np.array(expert, np.int32), *w), out=out, workspace=ws)
    got = _host(out)
    assert np.all(got[held < 0] == 7.0)
    for e in range(2):
        at = held == e
        if at.any():
            y, slack = ref.ffn(rows[at], rs[at], *[t[e] for t in w])
            assert np.all(np.abs(got[at] - y) <= slack + BF * (np.abs(y) + slack))


@pytest.mark.parametrize("T,H,F,E,k", [(1, 2048, 1024, 8, 8), (64, 256, 256, 16, 8), (2600, 256, 640, 40, 4), (900, 256, 256, 12, 8),
                                       (300, 128, 1152, 8, 3), (520, 384, 4096, 4, 2), (70, 128, 16384, 2, 2), (2100, 3200, 256, 6, 6)])
def test_layer_slots_are_summed_beyond_bfloat16(T, H, F, E, k):
    """A slot's sum keeps float16's 11 bits (2^-11 of probs * y) where a bfloat16 row would keep 8; the rest as in
    test_layer.  Weights of either sign, so that the slots' rows cancel and their roundings show."""
    rng = np.random.default_rng(T + H + E)
    w = _weights(rng, E, H, F)
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).bfloat16()
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    probs = (rng.dirichlet(np.ones(k), T) * rng.choice([-1.0, 1.0], (T, k))).astype(np.float32)
    q, s = ref.quantize(x.float().numpy())
    r, tol = np.zeros((T, H)), np.zeros((T, H))
    for e in range(E):
        t, j = np.nonzero(ids == e)
        y, slack = ref.ffn(q[t], s[t], *[a[e] for a in w])
        p = probs[t, j].astype(np.float64)[:, None]
        np.add.at(r, t, p * y)
        np.add.at(tol, t, np.abs(p) * (slack + (2.0 ** -11 + (2 * k + 8) * U) * (np.abs(y) + slack)))
    print(f"[int8 layer] T={T} H={H} F={F} E={E} k={k}", flush=True)
    out = _host(mel.expert_forward_int8(x.cuda(), None, *_dev(*w), *_dev(ids, probs)))
    tol = tol + BF * (np.abs(r) + tol)
    assert np.all(np.abs(out - r) <= tol)


# Row tiles of 64 (small calls, cut products), 128 and 256 rows; k of both combines.
@pytest.mark.parametrize("T,H,F,E,k", [(3, 2048, 1024, 8, 2), (200, 512, 512, 16, 8), (900, 256, 2048, 4, 2), (4000, 512, 640, 24, 4)])
def test_captured_calls_replayed_on_one_workspace(T, H, F, E, k):
    """Layer, grouped FFN and product captured into two graphs that share each call's workspace, replayed in turn on
    new inputs with eager calls between: every replay bitwise the eager result, which repeats itself."""
    rng = np.random.default_rng(T)
    w = _dev(*_weights(rng, E, H, F))
    x = torch.randn((T, H), device="cuda").bfloat16()
    ids = torch.from_numpy(np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)).cuda()
    probs = torch.softmax(torch.randn((T, k), device="cuda"), 1)
    rows, rs = _dev(_codes(rng, T, H), _scale(rng, T, level=0.02))
    off = _dev(np.concatenate([[0], np.sort(rng.integers(0, T + 1, E - 1)), [T]]).astype(np.int32))[0]
    ex = torch.arange(E, dtype=torch.int32, device="cuda")
    ws = [torch.full((256 << 20,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]

    def step(spaces):
        return (mel.expert_forward_int8(x, None, *w, ids, probs, workspace=spaces[0]),
                mel.grouped_ffn_int8(rows, rs, off, ex, *w, workspace=spaces[1]),
                mel.grouped_matmul_int8(rows, rs, off, ex, w[0], w[1], workspace=spaces[2]))

    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = step(ws)
        graphs.append((g, outs))
    for i in range(4):
        x.copy_(torch.randn((T, H), device="cuda"))
        rows.copy_(torch.randint(-127, 128, (T, H), device="cuda"))
        off[1:-1] = torch.randint(0, T + 1, (E - 1,), device="cuda").sort().values
        eager = step([None] * 3)
        assert all(torch.equal(a, b) for a, b in zip(eager, step(ws)))
        for g, outs in graphs:
            for o in outs:
                o.fill_(3.0)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(eager, outs))
