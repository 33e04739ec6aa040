"""The shared expert's operators on the CPU: the generator's known answers, and every refusal of the C ABI before
anything is enqueued (the pointers are never read)."""
import ctypes
import os

import pytest

import shared_expert_reference as ref

torch = pytest.importorskip("torch")

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def mel():
    import moe_expert_layer_amd as m
    if not os.path.exists(m.lib_path):
        from moe_expert_layer_amd.build import build
        build(verbose=False)
    m.library()
    return m


def test_philox_known_answers():
    """The published test vectors of Philox 4x32-10."""
    assert ref.philox((0, 0, 0, 0), (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    f = 0xFFFFFFFF
    assert ref.philox((f, f, f, f), (f, f)) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert ref.philox((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0)) == \
        [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def _gated(mel, **kw):
    d = dict(T=4, H=16, F=16, dtype=1, activation=0, dropout=0.0)
    d.update(kw)
    return mel.MoeGated(*[d[k] for k in ("T", "H", "F", "dtype", "activation", "dropout")])


NAN = float("nan")


@pytest.mark.parametrize("kw,expected", [
    (dict(), 0), (dict(T=0), 0), (dict(H=1, F=1), 0), (dict(H=1001, F=7), 0), (dict(dtype=0), 0),
    (dict(T=-1), 1), (dict(H=0), 1), (dict(F=-5), 1), (dict(activation=3), 1), (dict(activation=-1), 1),
    (dict(dropout=-0.1), 1), (dict(dropout=1.1), 1), (dict(dropout=NAN), 1), (dict(dropout=1.0), 0),
    (dict(dtype=2), 2), (dict(dtype=3), 2), (dict(T=1 << 31), 2), (dict(H=(1 << 22) + 1), 2), (dict(F=(1 << 22) + 1), 2),
    (dict(T=(1 << 31) - 1, H=512, F=512), 2), (dict(T=1 << 28, H=512, F=512), 0), (dict(T=(1 << 28) + 1), 2),
    (dict(T=1 << 28, H=513), 2), (dict(H=1 << 22, F=1 << 19), 2),
])
def test_gated_sizes(mel, kw, expected):
    lib = mel.library()
    g = _gated(mel, **kw)
    n = ctypes.c_size_t()
    for backward in (0, 1):
        assert lib.moe_gated_workspace_size(ctypes.byref(g), backward, ctypes.byref(n)) == expected, lib.moe_last_error()
    assert lib.moe_gated_workspace_size(None, 0, ctypes.byref(n)) == 1
    if expected == 0:
        assert lib.moe_gated_workspace_size(ctypes.byref(g), 0, None) == 1


def test_gated_refusals(mel):
    lib = mel.library()
    ok = P(0x10000)

    def forward(g, x=ok, wg=ok, wu=ok, rng=None, h=ok, saved=None, ws=ok, n=1 << 40):
        return lib.moe_gated_projection(ctypes.byref(g), x, wg, wu, rng, h, saved, ws, n, None)

    def backward(g, x=ok, wg=ok, wu=ok, dh=ok, rng=None, saved=None, dx=ok, dwg=ok, dwu=ok, ws=ok, n=1 << 40):
        return lib.moe_gated_projection_backward(ctypes.byref(g), x, wg, wu, dh, rng, saved, dx, dwg, dwu, ws, n, None)

    g = _gated(mel)
    for name in ("x", "wg", "wu", "h"):
        assert forward(g, **{name: None}) == 1
    for name in ("x", "wg", "wu", "dh", "dx", "dwg", "dwu"):
        assert backward(g, **{name: None}) == 1
    # bfloat16 pointers to half an element; rows of whole chunks that start between two
    assert forward(g, h=P(0x10001)) == 1 and forward(g, saved=P(0x10001)) == 1 and backward(g, dh=P(0x10001)) == 1
    for name in ("x", "wg", "wu"):
        assert forward(g, **{name: P(0x10008)}) == 1 and b"aligned" in lib.moe_last_error()
        assert backward(g, **{name: P(0x10008)}) == 1
    # dropout without rng, or with one that is not aligned
    d = _gated(mel, dropout=0.5)
    assert forward(d) == 1 and b"rng" in lib.moe_last_error()
    assert backward(d) == 1 and forward(d, rng=P(0x10004)) == 1
    # workspaces: the backward always needs one, the forward where operands are laid out anew
    assert backward(g, ws=None) == 3 and backward(g, n=1) == 3 and backward(g, ws=P(0x10008)) == 1
    odd = _gated(mel, T=100, H=15)
    assert forward(odd, ws=None) == 3 and forward(odd, n=1) == 3
    # no tokens: nothing to do in the forward
    assert forward(_gated(mel, T=0), x=None, wg=None, wu=None, h=None, ws=None, n=0) == 0


def test_dropout_refusals(mel):
    lib = mel.library()
    ok = P(0x10000)

    def call(x=ok, residual=None, dtype=1, rows=4, cols=16, p=0.5, rng=ok, out=ok):
        return lib.moe_dropout(x, residual, dtype, rows, cols, p, rng, out, None)

    assert call(rows=-1) == 1 and call(cols=0) == 1 and call(p=-0.5) == 1 and call(p=1.5) == 1 and call(p=NAN) == 1
    assert call(dtype=2) == 2 and call(dtype=3) == 2 and call(rows=1 << 31) == 2 and call(cols=(1 << 22) + 1) == 2
    assert call(x=None) == 1 and call(out=None) == 1 and call(rng=None) == 1 and call(rng=P(0x10004)) == 1
    assert call(out=P(0x10001)) == 1 and call(residual=P(0x10001)) == 1 and call(dtype=0, x=P(0x10002)) == 1
    assert call(rows=0, x=None, out=None) == 0


def _adapter(mel, **kw):
    d = dict(T=4, K=16, N=16, L=2, R=8, dtype=1, reserved=0)
    d.update(kw)
    return mel.MoeAdapter(*[d[k] for k in ("T", "K", "N", "L", "R", "dtype", "reserved")])


@pytest.mark.parametrize("kw,expected", [
    (dict(), 0), (dict(T=0), 0), (dict(K=1, N=1, L=1, R=1), 0), (dict(R=128, L=1023), 0), (dict(dtype=0), 0),
    (dict(T=-1), 1), (dict(K=0), 1), (dict(N=0), 1), (dict(L=0), 1), (dict(R=0), 1), (dict(reserved=1), 1),
    (dict(R=129), 2), (dict(L=1024), 2), (dict(dtype=2), 2), (dict(T=(1 << 28) + 1), 2), (dict(K=(1 << 22) + 1), 2),
    (dict(T=1 << 28, K=512, N=512), 0), (dict(T=1 << 28, K=513), 2), (dict(T=1 << 28, N=513), 2),
    (dict(N=(1 << 22) + 1), 2),
])
def test_adapter_sizes(mel, kw, expected):
    lib = mel.library()
    p = _adapter(mel, **kw)
    n = ctypes.c_size_t()
    assert lib.moe_adapter_workspace_size(ctypes.byref(p), ctypes.byref(n)) == expected, lib.moe_last_error()
    assert lib.moe_adapter_workspace_size(None, ctypes.byref(n)) == 1


def test_adapter_refusals(mel):
    lib = mel.library()
    ok = P(0x10000)

    def call(p, base=ok, x=ok, a=ok, b=ok, ids=ok, scale=None, ranks=None, out=ok, ws=ok, n=1 << 40):
        return lib.moe_adapter_add(ctypes.byref(p), base, x, a, b, ids, scale, ranks, out, ws, n, None)

    p = _adapter(mel, T=4000, K=4096, N=4096, R=128)           # sizes that need a workspace
    for name in ("base", "x", "a", "b", "ids", "out"):
        assert call(p, **{name: None}) == 1
    for name in ("scale", "ranks", "ids"):
        assert call(p, **{name: P(0x10002)}) == 1
    assert call(p, out=P(0x10001)) == 1
    assert call(p, ws=None) == 3 and call(p, n=0) == 3 and call(p, ws=P(0x10008)) == 1
    assert call(_adapter(mel, T=0), base=None, x=None, a=None, b=None, ids=None, out=None, ws=None, n=0) == 0


def test_binding_refuses(mel):
    x = torch.zeros((2, 16), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="on a GPU"):
        mel.dropout(x, 0.5)
    with pytest.raises(ValueError, match="on a GPU"):
        mel.gated_projection(x, x, x)
    with pytest.raises(ValueError, match="activation"):
        mel._gated(1, 8, 8, mel.BF16, "relu", 0.0, 0)
    with pytest.raises(mel.MoeError):
        mel.gated_workspace_size(1, 0, 8, mel.BF16)
    with pytest.raises(mel.MoeError):
        mel.adapter_workspace_size(1, 8, 8, 1, 1000, mel.BF16)
    assert mel.gated_workspace_size(4, 16, 16, mel.BF16) == 0
