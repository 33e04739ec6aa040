"""CPU checks of the int8 and gate entry points' argument checks (they return before any HIP call), and
of the plain forms the GPU tests use."""
import ctypes

import numpy as np
import pytest

import int8_gate_reference as ref


@pytest.fixture(scope="module")
def mel():
    import os

    import moe_expert_layer_amd as m
    if not os.path.exists(m.lib_path):
        from moe_expert_layer_amd.build import build
        build(verbose=False)
    m.library()
    return m


@pytest.mark.parametrize("kw,expected", [
    (dict(), 0), (dict(T=0), 0),
    (dict(H=192), 2), (dict(F=64), 2), (dict(H=131072), 2), (dict(H=130944), 0),
    (dict(E=0), 1), (dict(E=1024), 2), (dict(k=5), 1), (dict(T=-1), 1), (dict(head=256), 2),
    (dict(T=1 << 26, H=128), 2),                       # T * H = 2^33
    (dict(T=1 << 31, k=1), 2), (dict(flags=4), 1), (dict(flags=2), 0), (dict(flags=1), 0),
])
def test_int8_problem(mel, kw, expected):
    v = dict(T=64, H=256, F=384, E=4, k=2, head=0, flags=0)
    v.update(kw)
    prob = mel.problem(v["T"], v["H"], v["F"], v["E"], v["k"], mel.INT8, v["head"], v["flags"])
    n = ctypes.c_size_t()
    assert mel.library().moe_workspace_size(ctypes.byref(prob), ctypes.byref(n)) == expected
    if expected == 0:
        assert n.value >= v["T"] * v["k"] * (v["F"] + 2 * v["H"])


def test_int8_calls_refuse_before_enqueue(mel):
    lib = mel.library()
    n = ctypes.c_size_t()
    p, q = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008)
    size = lib.moe_grouped_matmul_int8_workspace_size
    assert size(100, 4, 256, 128, ctypes.byref(n)) == 0
    assert size(-1, 4, 256, 128, ctypes.byref(n)) == 1 and size(1, 0, 256, 128, ctypes.byref(n)) == 1
    assert size(1, 1, 64, 128, ctypes.byref(n)) == 2 and size(1, 1, 128, 130, ctypes.byref(n)) == 2
    assert size(1, (1 << 24) + 1, 128, 128, ctypes.byref(n)) == 2
    # 2^24 row tiles x 2^14 column tiles: more tasks than 32 bits number
    assert size((1 << 31) - 1, 1 << 24, 128, 1 << 22, ctypes.byref(n)) == 2
    assert size(1, 1, 131072, 128, ctypes.byref(n)) == 2 and size(1 << 31, 1, 128, 128, ctypes.byref(n)) == 2
    size(100, 4, 256, 128, ctypes.byref(n))
    call = lib.moe_grouped_matmul_int8
    args = [p, p, 100, p, p, 4, p, p, 2, 256, 128, p, mel.BF16, p, n.value, None]

    def with_(i, v):
        a = list(args)
        a[i] = v
        return call(*a)
    assert with_(13, None) == 3 and with_(14, n.value - 1) == 3
    assert with_(0, None) == 1 and with_(3, None) == 1 and with_(11, None) == 1
    assert with_(0, q) == 1 and b"aligned" in lib.moe_last_error()
    assert with_(12, mel.MXFP8) == 2 and with_(8, 1024) == 2 and with_(8, 0) == 1
    prob = mel.problem(0, 256, 256, 2, 1, mel.INT8)
    assert lib.moe_grouped_ffn_workspace_size(ctypes.byref(prob), 10, 2, ctypes.byref(n)) == 0
    assert lib.moe_grouped_ffn_int8(ctypes.byref(prob), *([None] * 2), 10, None, None, 2, *([None] * 8), n.value, None) == 3
    bf = mel.problem(8, 256, 256, 2, 1, mel.BF16)
    assert lib.moe_expert_forward_int8(ctypes.byref(bf), *([None] * 12), 0, None) == 1
    i8 = mel.problem(8, 256, 256, 2, 1, mel.INT8)
    assert lib.moe_expert_forward_int8(ctypes.byref(i8), *([None] * 12), 0, None) == 3
    # the other dtypes' calls do not take int8 problems
    assert lib.moe_expert_forward(ctypes.byref(i8), *([None] * 8), 0, None) == 2
    assert lib.moe_backward_workspace_size(ctypes.byref(i8), ctypes.byref(n)) == 2
    assert lib.moe_int8_quantize(None, mel.F32, 4, 8, None, None, None) == 1
    assert lib.moe_int8_quantize(None, mel.F32, 0, 8, None, None, None) == 0
    assert lib.moe_int8_quantize(p, mel.MXFP8, 4, 8, p, p, None) == 2
    assert lib.moe_int8_quantize(p, mel.F32, 4, 0, p, p, None) == 1


def test_gate_refuses_before_enqueue(mel):
    lib = mel.library()
    p = ctypes.c_void_p(0x1000)

    def call(T=4, E=8, k=2, dtype=0, logits=p, **kw):
        v = dict(score=0, renormalize=1, groups=1, topk_groups=1, group_top=2, scale=1.0)
        v.update(kw)
        g = mel.MoeGate(*v.values())
        a = lib.moe_router_gate(ctypes.byref(g), logits, dtype, None, T, E, k, p, p, None)
        b = lib.moe_router_gate_backward(ctypes.byref(g), logits, dtype, T, E, k, p, p, p, None)
        assert a == b
        return a
    assert call(T=0) == 0
    for kw in (dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=9), dict(E=128, k=65), dict(logits=None),
               dict(score=2), dict(renormalize=2), dict(groups=3), dict(groups=0), dict(groups=2, topk_groups=3),
               dict(groups=4, topk_groups=0), dict(groups=8, topk_groups=1), dict(group_top=0), dict(scale=float("nan")),
               dict(T=1 << 40)):
        assert call(**kw) == 1, kw
    assert call(dtype=2) == 2
    assert lib.moe_router_gate(None, p, 0, None, 4, 8, 2, p, p, None) == 1


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_plain_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(0)
    l = rng.standard_normal((5, 9))
    ids = np.stack([rng.permutation(9)[:4] for _ in range(5)])
    dp = rng.standard_normal((5, 4))
    g = ref.gate_backward(l, ids, dp, score, renorm, 1.5)

    def loss(v):
        w = np.take_along_axis(ref.scores(v, score), ids, 1)
        return 1.5 * (dp * (w / w.sum(1, keepdims=True) if renorm else w)).sum(1)
    for e in range(9):
        h = np.zeros(9)
        h[e] = 1e-5
        np.testing.assert_allclose((loss(l + h) - loss(l - h)) / 2e-5, g[:, e], rtol=1e-6, atol=1e-9)


def test_plain_gate_against_a_sort():
    rng = np.random.default_rng(1)
    l = rng.standard_normal((30, 24)).astype(np.float32)
    ids, w, s = ref.gate(l, 5)
    assert np.array_equal(ids, np.argsort(-l, 1, kind="stable")[:, :5])
    np.testing.assert_allclose(w.sum(1), 1.0)
    ids, _, _ = ref.gate(l, 6, groups=4, topk_groups=1, group_top=1)
    assert np.array_equal(ids[:, 0], l.argmax(1)) and np.all(ids // 6 == ids[:, :1] // 6)


@pytest.mark.parametrize("place", [2, 3, 4])
def test_gate_settings_that_do_not_fit(mel, place):
    """Group settings of more than 32 bits are refused, not cut to their low bits."""
    args = ["softmax", 1, 1, 1, 1, 1.0]
    assert mel._gate(*args).groups == 1
    for v in (2 ** 32 + 1, -2 ** 32 + 1, 2 ** 31):
        args[place] = v
        with pytest.raises(ValueError):
            mel._gate(*args)
