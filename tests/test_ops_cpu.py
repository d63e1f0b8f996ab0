"""Host-side checks of the routing and 4-bit operators: refusals before anything is enqueued, the stored
order of 4-bit codes, and the generator's weights. No GPU."""
import ctypes

import numpy as np
import pytest
import torch

from fine_grained_sparse_fp32_b200 import _build, kmoe
from fine_grained_sparse_fp32_b200.inputs import LayerConfig, make_inputs, pack_w4, unpack_w4
import plain_ops

A = ctypes.c_void_p(1 << 20)
OFF = ctypes.c_void_p((1 << 20) + 4)
OK, BAD, UNSUP = kmoe.KMOE_OK, kmoe.KMOE_ERR_INVALID_ARG, kmoe.KMOE_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return kmoe.load()


def rule(**kw):
    f = dict(score=0, n_groups=8, topk_groups=4, group_score=1, renormalise=1, scale=1.0)
    f.update(kw)
    return ctypes.byref(kmoe._RoutingStruct(**f))


@pytest.mark.parametrize("kw,code,word", [
    (dict(score=2), BAD, b"score"), (dict(score=-1), BAD, b"score"), (dict(group_score=5), BAD, b"group_score"),
    (dict(n_groups=0), UNSUP, b"n_groups"), (dict(n_groups=7), UNSUP, b"n_groups"),
    (dict(n_groups=48), UNSUP, b"n_groups"), (dict(topk_groups=0), BAD, b"topk_groups"),
    (dict(topk_groups=9), BAD, b"topk_groups"), (dict(renormalise=2), BAD, b"renormalise"),
    (dict(scale=float("nan")), BAD, b"scale"), (dict(scale=float("inf")), BAD, b"scale")])
def test_routing_rules_are_checked(lib, kw, code, word):
    assert lib.moe_route(A, 0, None, 4, 384, 6, rule(**kw), A, A, None) == code and word in lib.moe_last_error()
    ex = kmoe.Experts(A, A, A, None, None, None, kmoe.KMOE_BF16)
    st = lib.moe_forward_routed(A, kmoe.KMOE_BF16, 4, 2560, 384, 6, 512, rule(**kw), A, None, ctypes.byref(ex), None, A,
                                kmoe.KMOE_BF16, None, None, None, A, 1 << 40, None)
    assert st == code
    st = lib.moe_block_forward_routed(A, 4, 2560, 384, 6, 512, rule(**kw), A, A, 1e-6, A, None, ctypes.byref(ex), None,
                                      A, None, None, None, None, A, 1 << 40, None)
    assert st == code


def test_route_refuses_groups_that_hold_too_few_experts_and_bad_pointers(lib):
    assert lib.moe_route(A, 0, None, 4, 8, 6, rule(n_groups=4, topk_groups=2), A, A, None) == BAD
    assert lib.moe_route(A, 0, None, 4, 384, 9, rule(), A, A, None) == UNSUP
    assert lib.moe_route(A, 0, None, 4, 2048, 6, rule(), A, A, None) == UNSUP
    assert lib.moe_route(A, 2, None, 4, 384, 6, rule(), A, A, None) == UNSUP
    assert lib.moe_route(A, 0, None, 4, 384, 6, None, A, A, None) == BAD
    for args in ((None, A, A), (A, None, A), (A, A, None), (OFF, A, A)):
        assert lib.moe_route(args[0], 0, None, 4, 384, 6, rule(), args[1], args[2], None) == BAD
    assert lib.moe_route(A, 0, OFF, 4, 384, 6, rule(), A, A, None) == BAD
    assert lib.moe_route(None, 0, None, 0, 384, 6, rule(), None, None, None) == OK
    assert lib.moe_forward_routed(A, 1, 4, 2560, 384, 6, 512, None, A, None, None, None, A, 1, None, None, None, A, 0,
                                  None) == BAD


def w4(group=128, codes=A, scales=A, zeros=None):
    v = lambda p: None if p is None else p.value
    return kmoe._W4Struct(v(codes), v(scales), v(zeros), group)


def linear(lib, w=None, x_dtype=1, N=4, P=4, rows=16, cols=256, E=1, perm=None, off=None, x=A, y=A, y_dtype=1):
    w = w4() if w is None else w
    return lib.moe_linear_w4(x, x_dtype, N, P, rows, cols, E, perm, off, ctypes.byref(w), y, y_dtype, A, 1 << 40, None)


def test_linear_w4_checks_its_arguments(lib):
    assert linear(lib, P=0, x=None, y=None) == OK
    for kw, code in ((dict(x_dtype=0), UNSUP), (dict(y_dtype=3), UNSUP), (dict(N=-1), BAD), (dict(P=-1), BAD),
                     (dict(rows=0), UNSUP), (dict(rows=65537), UNSUP), (dict(cols=200), UNSUP), (dict(cols=0), UNSUP),
                     (dict(cols=8192 + 128), UNSUP), (dict(E=0, off=A), UNSUP), (dict(E=1025, off=A), UNSUP),
                     (dict(E=2), BAD), (dict(N=3), BAD), (dict(x=None), BAD), (dict(y=None), BAD), (dict(y=OFF), BAD),
                     (dict(perm=OFF), BAD), (dict(off=OFF), BAD), (dict(w=w4(group=48)), UNSUP),
                     (dict(w=w4(codes=None)), BAD), (dict(w=w4(scales=OFF)), BAD), (dict(w=w4(zeros=OFF)), BAD)):
        assert linear(lib, **kw) == code, kw
    assert lib.moe_linear_w4(A, 1, 4, 4, 16, 256, 1, None, None, None, A, 1, A, 0, None) == BAD
    need = kmoe.moe_linear_w4_workspace_size(5000, 5000, 16, 256)
    assert need >= 5000 * (256 * 2 + 4)
    assert kmoe.moe_linear_w4_workspace_size(5000, 5000, 16, 256, y_dtype=torch.float32) == 0
    assert kmoe.moe_linear_w4_workspace_size(4, 4, 16, 256) == 0
    assert kmoe.moe_linear_w4_workspace_size(1 << 19, 1 << 19, 4096, 8192) > 1 << 33        # more than 32 bits
    assert kmoe.moe_linear_w4_workspace_size((1 << 22) - 1, 1 << 22, 16, 8192) > 1 << 35
    assert kmoe.moe_linear_w4_workspace_size(1 << 22, 1 << 22, 16, 8192) == 0                 # beyond 64 GiB of x: the other kernel
    w = w4()
    call = lambda ws, n: lib.moe_linear_w4(A, 1, 5000, 5000, 16, 256, 1, None, None, ctypes.byref(w), A, 1, ws, n, None)
    assert call(A, need - 1) == kmoe.KMOE_ERR_WORKSPACE and call(None, need) == BAD


def test_quant_w4_checks_its_arguments(lib):
    q = lambda w=A, dt=0, rows=4, cols=256, g=64, c=A, s=A, z=None: lib.moe_quant_w4(w, dt, rows, cols, g, c, s, z, None)
    assert q(rows=0, w=None, c=None, s=None) == OK
    for kw, code in ((dict(dt=2), UNSUP), (dict(rows=-1), BAD), (dict(cols=192), UNSUP), (dict(g=16), UNSUP),
                     (dict(w=None), BAD), (dict(c=OFF), BAD), (dict(s=None), BAD), (dict(z=OFF), BAD)):
        assert q(**kw) == code, kw
    d = lambda w=w4(), rows=4, cols=256, out=A, dt=0: lib.moe_dequant_w4(ctypes.byref(w), rows, cols, out, dt, None)
    assert d(rows=0) == OK
    for kw, code in ((dict(w=w4(group=8)), UNSUP), (dict(rows=-1), BAD), (dict(cols=64), UNSUP), (dict(out=None), BAD),
                     (dict(dt=2), UNSUP)):
        assert d(**kw) == code, kw


def test_4_bit_experts_are_checked(lib):
    def ffn(gate=None, up=None, down=None, shared=None, x_dtype=1, null=False):
        arr = (kmoe._W4Struct * 3)(gate or w4(), up or w4(), down or w4())
        ex = kmoe.Experts(dtype=kmoe.KMOE_W4, w4=None if null else arr)
        st = lib.moe_grouped_ffn(A, x_dtype, 4, 256, 128, 8, 2, A, A, ctypes.byref(ex),
                                 None if shared is None else ctypes.byref(shared), A, A, A, 16, None)
        return st
    assert ffn() == kmoe.KMOE_ERR_WORKSPACE            # everything else was accepted
    assert ffn(null=True) == BAD
    assert ffn(x_dtype=0) == UNSUP
    assert ffn(gate=w4(group=64)) == UNSUP             # gate and up differ
    assert ffn(up=w4(zeros=A)) == UNSUP
    assert ffn(down=w4(group=32)) == kmoe.KMOE_ERR_WORKSPACE
    assert ffn(down=w4(codes=None)) == BAD
    other = kmoe.Experts(dtype=kmoe.KMOE_W4, w4=(kmoe._W4Struct * 3)(w4(64), w4(64), w4()))
    assert ffn(shared=other) == UNSUP
    assert ffn(shared=kmoe.Experts(A, A, A, None, None, None, kmoe.KMOE_BF16)) == UNSUP
    bf = kmoe.moe_workspace_size(32, 2560, 384, 6, 512, kmoe.KMOE_BF16, kmoe.KMOE_BF16)
    assert kmoe.moe_workspace_size(32, 2560, 384, 6, 512, kmoe.KMOE_BF16, kmoe.KMOE_W4) >= bf
    assert kmoe.moe_block_workspace_size(32, 2560, 384, 6, 512, kmoe.KMOE_W4) > 0


def test_python_calls_refuse_tensors_the_library_would_misread():
    x = torch.zeros((2, 256), dtype=torch.bfloat16)
    codes, s = torch.zeros((16, 128), dtype=torch.uint8), torch.ones((16, 2), dtype=torch.bfloat16)
    w = kmoe.W4(codes, s)
    assert (w.rows, w.cols, w.group, w.E) == (16, 256, 128, 1)
    for bad in (lambda: kmoe.W4(codes.short(), s), lambda: kmoe.W4(codes.t(), s), lambda: kmoe.W4(codes, s.float()),
                lambda: kmoe.W4(codes, s[:8]), lambda: kmoe.W4(codes, s, torch.zeros((16, 2))),
                lambda: kmoe.moe_linear_w4(x, w), lambda: kmoe.moe_linear_w4(x[0], w),
                lambda: kmoe.moe_route(torch.zeros((2, 8)), 2), lambda: kmoe.moe_quant_w4(torch.zeros((2, 128))),
                lambda: kmoe.moe_dequant_w4(w), lambda: kmoe.Routing(score="tanh"),
                lambda: kmoe.Routing(group_score="mean")):
        with pytest.raises(ValueError):
            bad()
    cfg = LayerConfig("w4", 4, 256, 4, 2, 128, "bf16", "w4")
    layer = make_inputs(cfg)
    kmoe.experts_of(layer)
    with pytest.raises(ValueError):
        kmoe.experts_of(dict(layer, w_down=layer["w_down"][:, :, :32].contiguous(), s_down=layer["s_down"]))
    with pytest.raises(ValueError):
        kmoe.experts_of(dict(layer, w_up=layer["w_up"][:2]))


def test_stored_order_of_codes():
    gen = torch.Generator().manual_seed(0)
    q = torch.randint(0, 16, (3, 384), dtype=torch.uint8, generator=gen)
    packed = pack_w4(q)
    assert torch.equal(packed, plain_ops.w4_bytes(q))
    assert torch.equal(unpack_w4(packed), q)
    assert torch.equal(plain_ops.w4_codes(packed).to(torch.uint8), q)
    one = torch.zeros((1, 128), dtype=torch.uint8)
    one[0, 32 + 8 + 3] = 5              # word 5 (columns 40..47), stored at 4 * 1 + 1 = 5; column 3: bits 20..23
    b = pack_w4(one)
    assert int(b[0, 5 * 4 + 2]) == 0x50 and int(b.sum()) == 0x50


@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, False), (128, True)])
def test_generated_4_bit_layer(group, zeros):
    cfg = LayerConfig("w4", 4, 256, 4, 2, 128, "bf16", "w4", w4_group=group, w4_zeros=zeros)
    layer = make_inputs(cfg, seed=3)
    ref = make_inputs(LayerConfig("f", 4, 256, 4, 2, 128, "bf16", "f32"), seed=3)
    for m in ("gate", "up", "down"):
        v = plain_ops.w4_values(layer["w_" + m], layer["s_" + m], layer["z_" + m])
        step = layer["s_" + m].double().repeat_interleave(group, -1)
        w = ref["w_" + m].double()
        # half a step, plus what the scale's BF16 rounding (2^-8) can cost at the largest of 7 or 15 steps
        assert (v - w).abs().max() <= (step * (0.5 + (15 if zeros else 7) * 2.0 ** -8 + 1e-6)).max()
        assert ((v - w).abs() <= step * (0.5 + (15 if zeros else 7) * 2.0 ** -8 + 1e-6) + (step * 0.5 if zeros else 0)).all()


def test_plain_routing_by_hand():
    """Two groups of two: group scores decide before experts do, and masked experts come last."""
    l = torch.tensor([[0.0, 2.0, 1.0, 1.5]])
    idx, w = plain_ops.route(l, 2, n_groups=2, topk_groups=1, group_score="top2")
    assert idx.tolist() == [[3, 2]]                     # s(1) + s(1.5) > s(0) + s(2)
    sig = lambda v: 1 / (1 + np.exp(-v))
    np.testing.assert_allclose(w[0], [sig(1.5) / (sig(1.5) + sig(1.0)), sig(1.0) / (sig(1.5) + sig(1.0))], rtol=1e-14)
    assert plain_ops.route(l, 2, n_groups=2, topk_groups=1, group_score="max")[0].tolist() == [[1, 0]]
    l[0, 3] = -float("inf")
    idx, w = plain_ops.route(l, 2, n_groups=2, topk_groups=1, group_score="max", renormalise=False, scale=2.0)
    assert idx.tolist() == [[1, 0]] and abs(float(w[0, 0]) - 2 * sig(2.0)) < 1e-14
    idx, w = plain_ops.route(torch.full((1, 4), -float("inf")), 3, score="softmax")
    assert idx.tolist() == [[0, 1, 2]] and float(w.abs().sum()) == 0
