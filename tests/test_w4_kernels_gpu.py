"""Each of the two kernels for 4-bit products against the bound of its own, and both at the layer's full width.

Tolerances as in test_w4_range_gpu.py: the few-row kernel takes weights exactly and x to 2^-22 of the largest value of
its 128 columns, the tensor-core kernel weights to 2^-11 and x to 2^-39 of its row's largest value.
"""
import os
import subprocess
import sys
import textwrap

import pytest
import torch

from fine_grained_sparse_fp32_b200 import _build, kmoe
from fine_grained_sparse_fp32_b200.inputs import CONFIGS, LayerConfig, make_inputs
import plain_ops
from test_w4_range_gpu import BF16, check, gen, randn, runs_on_tensor_cores, sums_bound, values

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    kmoe.load()


@pytest.mark.parametrize("N", [7, 8, 24, 33, 70, 129, 300])
@pytest.mark.parametrize("rows,cols", [(16, 640), (100, 2560), (515, 256), (17, 8192), (1300, 384)])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True)])
def test_linear_w4_within_the_bound_of_its_kernel(N, rows, cols, group, zeros):
    g = gen(N + rows)
    x = randn(g, N, cols).bfloat16()
    w = kmoe.moe_quant_w4(randn(g, rows, cols) * 0.02 + 0.01, group=group, zeros=zeros)
    for y_dtype in (torch.bfloat16, torch.float32):
        check(kmoe.moe_linear_w4(x, w, y_dtype=y_dtype), x, values(w), runs_on_tensor_cores(N, w, y_dtype))


def ffn_uses_tensor_cores(cfg):
    # gate and up are dealt out in units of 128 rows each, a matrix alone in units of 256
    return kmoe.moe_linear_w4_workspace_size(cfg.N, cfg.N * cfg.K, 2 * cfg.I, cfg.d, cfg.E, cfg.w4_group) > 0


def check_experts(layer, y, ys, x, perm, offsets, tensor_cores):
    """Errors of both sums go through SiLU(g) * u, whose slopes are |dh/dg| <= 1.1 |u| and |dh/du| = |SiLU(g)|;
    exponential and reciprocal are off by less than 2^-20 together; H is rounded to FP16 on the tensor cores (2^-11)."""
    off, E = offsets.tolist(), layer["cfg"].E
    for e in range(E + 1):
        rows, got = (x, ys) if e == E else (x[perm[off[e]:off[e + 1]].long()], y[off[e]:off[e + 1]])
        if not rows.shape[0]:
            continue
        v = [plain_ops.w4_values(layer["w_" + m][e], layer["s_" + m][e], None if layer.get("z_" + m) is None else layer["z_" + m][e])
             for m in ("gate", "up", "down")]
        rows = rows.double()
        a, u = rows @ v[0].t(), rows @ v[1].t()
        silu = a * torch.sigmoid(a)
        h = silu * u
        dh = 1.1 * u.abs() * sums_bound(rows, v[0], tensor_cores) + silu.abs() * sums_bound(rows, v[1], tensor_cores) + 2.0 ** -20 * h.abs()
        if tensor_cores:
            dh = dh + 2.0 ** -11 * (h.abs() + dh)
        ref = h @ v[2].t()
        tol = dh @ v[2].abs().t() + sums_bound(h.abs() + dh, v[2], tensor_cores) + BF16 * ref.abs() + 1e-37
        off_by = ((got.double() - ref).abs() / tol).max()
        assert off_by <= 1, (e, float(off_by))


@pytest.mark.parametrize("N", [9, 60, 130, 260, 700])
@pytest.mark.parametrize("d,I,E,K,group,zeros", [(256, 128, 8, 2, 128, False), (384, 256, 5, 3, 32, True),
                                                 (1280, 128, 16, 6, 64, True)])
def test_experts_within_the_bound_of_their_kernel(N, d, I, E, K, group, zeros):
    cfg = LayerConfig("w4", N, d, E, K, I, "bf16", "w4", w4_group=group, w4_zeros=zeros)
    layer = make_inputs(cfg, seed=N, device="cuda")
    g = gen(N + d)
    x = randn(g, N, d).bfloat16()
    idx = torch.rand((N, E), device="cuda", generator=g).topk(K, 1).indices.int()
    _, offsets, perm, _ = kmoe.moe_permute(idx, E)
    y, ys = kmoe.Layer(layer, N).grouped_ffn(x, perm, offsets)
    check_experts(layer, y, ys, x, perm, offsets, ffn_uses_tensor_cores(cfg))


def test_prefill_at_full_width():
    """4096 tokens through 384 experts and a shared one, alone and in a layer call."""
    cfg = CONFIGS["w4_prefill"]
    layer = make_inputs(cfg, seed=2, device="cuda")
    assert ffn_uses_tensor_cores(cfg)
    handle = kmoe.Layer(layer, cfg.N)
    idx = torch.empty((cfg.N, cfg.K), dtype=torch.int32, device="cuda")
    w = torch.empty((cfg.N, cfg.K), device="cuda")
    out = torch.empty((cfg.N, cfg.d), device="cuda")
    handle.forward(layer["x"], y=out, topk_idx=idx, topk_w=w)
    assert kmoe.moe_device_status(handle.ws) == 0
    _, offsets, perm, inv = kmoe.moe_permute(idx, cfg.E)
    y, ys = handle.grouped_ffn(layer["x"], perm, offsets)
    assert kmoe.moe_device_status(handle.ws) == 0
    check_experts(layer, y, ys, layer["x"], perm, offsets, True)
    # the layer's result is their weighted sum, in FP32 and slot order: K + 1 roundings of 2^-24 a term
    terms = w.double()[..., None] * y.double()[inv.long()]
    ref, size = ys.double() + terms.sum(1), ys.double().abs() + terms.abs().sum(1)
    assert ((out.double() - ref).abs() <= (2 * cfg.K + 2) * 2.0 ** -24 * size).all()


CHILD = textwrap.dedent('''
    import sys
    sys.path.insert(0, {root!r}); sys.path.insert(0, {tests!r})
    import torch
    from fine_grained_sparse_fp32_b200 import kmoe
    from fine_grained_sparse_fp32_b200.inputs import LayerConfig, make_inputs
    import plain_ops
    from test_w4_kernels_gpu import check_experts, ffn_uses_tensor_cores, gen, randn
    for N, group, zeros in ((20, 64, True), (900, 32, True), (900, 128, False)):
        cfg = LayerConfig("w4", N, 512, 8, 2, 256, "bf16", "w4", w4_group=group, w4_zeros=zeros)
        layer = make_inputs(cfg, seed=N, device="cuda")
        assert ffn_uses_tensor_cores(cfg) == (N == 900)
        rule = dict(score="sigmoid", n_groups=4, topk_groups=2)
        logits = layer["x"].float() @ layer["w_router"].t()
        idx, w = kmoe.moe_route(logits, cfg.K, layer["bias"], kmoe.Routing(**rule))
        assert torch.equal(idx.cpu(), plain_ops.route(logits, cfg.K, layer["bias"], **rule)[0])
        _, offsets, perm, _ = kmoe.moe_permute(idx, cfg.E)
        handle = kmoe.Layer(layer, N, routing=kmoe.Routing(**rule))
        y, ys = handle.grouped_ffn(layer["x"], perm, offsets)
        assert kmoe.moe_device_status(handle.ws) == 0
        check_experts(layer, y, ys, layer["x"], perm, offsets, N == 900)
        handle.forward(layer["x"])
        assert kmoe.moe_device_status(handle.ws) == 0
    print("DEBUG-BUILD-OK")
''')


def test_debug_build_routes_and_takes_4_bit_weights():
    """libkmoe_debug.so: the same kernels with index checks, in a child process."""
    lib = _build.build(debug=True)
    child = CHILD.format(root=ROOT, tests=os.path.join(ROOT, "tests"))
    r = subprocess.run([sys.executable, "-c", child], env=dict(os.environ, KMOE_LIBRARY=lib), capture_output=True, text=True, timeout=900)
    assert r.returncode == 0 and "DEBUG-BUILD-OK" in r.stdout, r.stdout[-2000:] + r.stderr[-3000:]
