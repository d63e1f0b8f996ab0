"""4-bit products whose weights, scales or tokens span wide ranges, against plain 64-bit forms.

Tolerances. y is rounded to BF16 once (half a step, 2^-8 of the value). On the tensor cores a weight is rounded to
FP16 at most once, 2^-11 of its own value, and x is held to 2^-39 of its row's largest value. The sums follow in
FP32: at most cols / 16 partial sums and cols / 32 scaled ones, each with two roundings of 2^-24, and eight more, all
relative to S = sum |W| |x|. Nothing is allowed for a group whose weights, or whose x, are zero: its scale, however large,
must not cost the others a bit. The few-row kernel takes weights exactly and x to within 2^-22 of the largest value
of its 128 columns.
"""
import pytest
import torch

from fine_grained_sparse_fp32_b200 import _build, kmoe
from fine_grained_sparse_fp32_b200.inputs import LayerConfig, make_inputs
import plain_ops

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    kmoe.load()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(shape, device="cuda", generator=g)


def values(w):
    return plain_ops.w4_values(w.codes, w.scales, w.zeros)


def sums_bound(x, w, tensor_cores):
    """Error of the sums before they are rounded to y; x [n, cols], w [rows, cols] in FP64."""
    cols = x.shape[1]
    each = (cols / 16 + cols / 32 + 8) * 2.0 ** -23
    if tensor_cores:
        top, each, x_off = x.abs().amax(-1, keepdim=True).expand_as(x), each + 2.0 ** -11, 2.0 ** -39
    else:
        top, x_off = x.abs().unflatten(-1, (-1, 128)).amax(-1).repeat_interleave(128, -1), 2.0 ** -22
    return (each * x.abs() + x_off * top) @ w.abs().t()


def check(y, x, w, tensor_cores):
    """y of BF16 or FP32 x [n, cols] and FP64 weights [rows, cols]."""
    x = x.double()
    ref = x @ w.t()
    tol = sums_bound(x, w, tensor_cores) + (BF16 * ref.abs() if y.dtype == torch.bfloat16 else 0) + 1e-37
    assert torch.isfinite(y).all()
    off = (y.double() - ref).abs() / tol
    assert off.max() <= 1, float(off.max())


def runs_on_tensor_cores(N, w, y_dtype=torch.bfloat16):
    return kmoe.moe_linear_w4_workspace_size(N, N, w.rows, w.cols, w.E, w.group, y_dtype) > 0


# ------------------------------------------------- scales of a row that differ widely
@pytest.mark.parametrize("N", [8, 2500])
@pytest.mark.parametrize("group,zeros", [(32, False), (32, True), (64, True), (128, False), (128, True)])
@pytest.mark.parametrize("std", [0.02, 1e-3, 1e-4, 1e-5])
@pytest.mark.parametrize("where", ["padded", "pruned"])
def test_groups_of_zeros_cost_the_others_nothing(N, group, zeros, std, where):
    """The quantiser gives a group of zeros the scale 1: columns padded with zeros, and pruned groups."""
    g = gen(N + group)
    w = randn(g, 256, 1280) * std
    if where == "padded":
        w[:, -128:] = 0.0
    else:
        w.unflatten(1, (-1, group))[torch.rand((256, 1280 // group), device="cuda", generator=g) < 0.2] = 0.0
    q = kmoe.moe_quant_w4(w, group=group, zeros=zeros)
    x = randn(g, N, 1280).bfloat16()
    assert runs_on_tensor_cores(N, q) == (N == 2500)
    y = kmoe.moe_linear_w4(x, q)
    check(y, x, values(q), N == 2500)
    assert torch.equal(y, kmoe.moe_linear_w4(x, q))


def wide_w4(g, lead, rows, cols, group, zeros, binades):
    """Any codes, scales over `binades` powers of two, some of them 0 or negative."""
    shape = (lead, rows, cols // group)
    codes = torch.randint(0, 256, (lead, rows, cols // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.exp2((torch.rand(shape, device="cuda", generator=g) - 0.5) * binades) * 0.01
    pick = torch.rand(shape, device="cuda", generator=g)
    scales = torch.where(pick < 0.05, torch.zeros_like(scales), torch.where(pick > 0.9, -scales, scales))
    z = torch.randint(0, 16, shape, dtype=torch.uint8, device="cuda", generator=g) if zeros else None
    return kmoe.W4(codes, scales.bfloat16(), z)


@pytest.mark.parametrize("binades", [6, 20, 60])
@pytest.mark.parametrize("group,zeros", [(32, False), (32, True), (64, False), (64, True), (128, False), (128, True)])
@pytest.mark.parametrize("N,rows,cols", [(2500, 256, 1280), (2000, 301, 128), (3000, 130, 384)])
def test_scales_over_many_powers_of_two(N, rows, cols, group, zeros, binades):
    """x is zero in some groups of 32 columns and large in others, so that any of a row's groups decides its sum."""
    g = gen(rows + group + binades)
    w = wide_w4(g, 1, rows, cols, group, zeros, binades)
    w = kmoe.W4(w.codes[0], w.scales[0], None if w.zeros is None else w.zeros[0])
    shape = (N, cols // 32, 1)
    x = randn(g, N, cols).unflatten(1, (-1, 32)) * torch.exp2(torch.randint(-9, 10, shape, device="cuda", generator=g))
    x = (x * (torch.rand(shape, device="cuda", generator=g) < 0.3)).flatten(1).bfloat16()
    assert runs_on_tensor_cores(N, w)
    y = kmoe.moe_linear_w4(x, w)
    check(y, x, values(w), True)
    assert torch.equal(y, kmoe.moe_linear_w4(x, w))


@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True)])
@pytest.mark.parametrize("cols", [128, 640])
def test_wide_and_ordinary_units_in_turn(group, zeros, cols):
    """Experts of 0 to 1500 rows, some with scales that differ widely, whose units a CTA takes one after another."""
    g = gen(cols + group)
    N, E, rows = 1500, 7, 900
    w = wide_w4(g, E, rows, cols, group, zeros, 40)
    w.scales[::2] = (torch.rand(w.scales[::2].shape, device="cuda", generator=g) * 0.02 + 0.001).bfloat16()
    w.scales[1, 300:] = 0.01                                # of its tiles, one or two
    x = randn(g, N, cols).bfloat16()
    counts = torch.tensor([40, 1500, 17, 0, 700, 129, 64])
    offsets = torch.cat((counts.new_zeros(1), counts.cumsum(0))).int().cuda()
    P = int(counts.sum())
    perm = torch.randint(0, N, (P,), dtype=torch.int32, device="cuda", generator=g)
    assert kmoe.moe_linear_w4_workspace_size(N, P, rows, cols, E, group) > 0
    y = kmoe.moe_linear_w4(x, w, perm, offsets)
    v, off = values(w), offsets.tolist()
    for e in range(E):
        at = slice(off[e], off[e + 1])
        if off[e] < off[e + 1]:
            check(y[at], x[perm[at].long()], v[e], True)
    assert torch.equal(y, kmoe.moe_linear_w4(x, w, perm, offsets))


@pytest.mark.parametrize("N", [8, 2500])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("binades", [0, 4, 30])
def test_a_weight_of_zero_stays_zero_for_every_zero_point(N, group, binades):
    """Codes equal to their zero point (0 to 15) in columns where x is large, and one place away from it elsewhere,
    with scales of every mantissa."""
    g = gen(group + binades)
    rows, cols = 256, 640
    shape = (rows, cols // group)
    z = torch.randint(0, 16, shape, dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.randint(128, 256, shape, device="cuda", generator=g) * 2.0 ** -15
    scales = scales * torch.exp2((torch.rand(shape, device="cuda", generator=g) * binades).round())
    q = z.repeat_interleave(group, 1).short()
    large = torch.arange(cols, device="cuda") % 5 == 0
    step = torch.where(q == 0, 1, torch.where(q == 15, -1, torch.randint(0, 2, q.shape, device="cuda", generator=g) * 2 - 1))
    q = torch.where(large, q, q + step).to(torch.uint8)
    w = kmoe.W4(plain_ops.w4_bytes(q.cpu()).cuda(), scales.bfloat16(), z)
    x = randn(g, N, cols)
    x[:, large] *= 4000
    x = x.bfloat16()
    assert runs_on_tensor_cores(N, w) == (N == 2500)
    check(kmoe.moe_linear_w4(x, w), x, values(w), N == 2500)


@pytest.mark.parametrize("N", [40, 1500])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, False)])
def test_experts_with_groups_of_zeros(N, group, zeros):
    """The FFN with weights of spread 1e-4 and 1e-3 and zeros at the end of every row. For the result the errors of
    both sums go through SiLU(g) * u, whose slopes are |dh/dg| <= 1.1 |u| and |dh/du| = |SiLU(g)|; exponential and
    reciprocal are off by less than 2^-20 together; H is rounded to FP16 on the tensor cores (2^-11)."""
    d, I, E, K = 512, 256, 4, 2
    cfg = LayerConfig("w4", N, d, E, K, I, "bf16", "w4", w4_group=group, w4_zeros=zeros)
    layer = make_inputs(cfg, seed=N, device="cuda")
    g = gen(N)
    for m, (r, c, std) in dict(gate=(I, d, 1e-4), up=(I, d, 1e-3), down=(d, I, 1e-4)).items():
        w = randn(g, E + 1, r, c) * std
        w[..., -128:] = 0.0
        q = kmoe.moe_quant_w4(w, group=group, zeros=zeros)
        layer.update({"w_" + m: q.codes, "s_" + m: q.scales, "z_" + m: q.zeros})
    x = randn(g, N, d).bfloat16()
    x[:, ::7] *= 30
    idx = torch.rand((N, E), device="cuda", generator=g).topk(K, 1).indices.int()
    _, offsets, perm, _ = kmoe.moe_permute(idx, E)
    y, ys = kmoe.Layer(layer, N).grouped_ffn(x, perm, offsets)
    off, tc = offsets.tolist(), N == 1500
    for e in range(E + 1):
        rows, got = (x, ys) if e == E else (x[perm[off[e]:off[e + 1]].long()], y[off[e]:off[e + 1]])
        v = [plain_ops.w4_values(layer["w_" + m][e], layer["s_" + m][e], layer["z_" + m][e] if zeros else None)
             for m in ("gate", "up", "down")]
        rows = rows.double()
        a, u = rows @ v[0].t(), rows @ v[1].t()
        silu = a * torch.sigmoid(a)
        h = silu * u
        dh = 1.1 * u.abs() * sums_bound(rows, v[0], tc) + silu.abs() * sums_bound(rows, v[1], tc) + 2.0 ** -20 * h.abs()
        if tc:
            dh = dh + 2.0 ** -11 * (h.abs() + dh)
        ref = h @ v[2].t()
        tol = dh @ v[2].abs().t() + sums_bound(h.abs() + dh, v[2], tc) + BF16 * ref.abs() + 1e-37
        off_by = ((got.double() - ref).abs() / tol).max()
        assert off_by <= 1, (e, float(off_by))


@pytest.mark.parametrize("large", [1000.0, 30000.0])
@pytest.mark.parametrize("N", [1, 3, 21, 2000])
@pytest.mark.parametrize("group,zeros,y_dtype", [(32, True, torch.bfloat16), (64, False, torch.bfloat16),
                                                 (128, False, torch.bfloat16), (128, True, torch.float32)])
def test_one_large_channel_costs_the_others_nothing(large, N, group, zeros, y_dtype):
    """One x of 128 columns far above the rest, in a column whose weights are zero in many rows."""
    g = gen(N + group)
    rows, cols = 200, 512
    w = randn(g, rows, cols) * 0.02
    w[:, 77::128] = 0.0
    w[::3, 77::128] = 0.01
    q = kmoe.moe_quant_w4(w, group=group, zeros=zeros)
    x = randn(g, N, cols)
    x[:, 77::128] = large
    x = x.bfloat16()
    check(kmoe.moe_linear_w4(x, q, y_dtype=y_dtype), x, values(q), runs_on_tensor_cores(N, q, y_dtype))


@pytest.mark.parametrize("N", [8, 2500])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, False)])
@pytest.mark.parametrize("w_size,x_size", [(1e37, 1e-30), (1e37, 1e-8), (1e-36, 1e30), (1e-30, 1e37)])
def test_large_weights_and_small_tokens_meet_in_range(N, group, zeros, w_size, x_size):
    g = gen(N + group)
    q = kmoe.moe_quant_w4((randn(g, 200, 256).clamp(-6, 6) * w_size), group=group, zeros=zeros)
    x = (randn(g, N, 256) * x_size).bfloat16()
    check(kmoe.moe_linear_w4(x, q), x, values(q), N == 2500)


@pytest.mark.parametrize("N", [8, 2500])
def test_the_largest_scales(N):
    """Scales up to the largest finite one, with codes at most one place from their zero point."""
    g = gen(N)
    codes = torch.randint(7, 10, (200, 256), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.tensor([2.0 ** 127 * 1.9921875, 2.0 ** 127, -2.0 ** 126.5, 2.0 ** 120], device="cuda")
    scales = scales[torch.randint(0, 4, (200, 4), device="cuda", generator=g)].bfloat16()
    w = kmoe.W4(plain_ops.w4_bytes(codes.cpu()).cuda(), scales)
    x = (randn(g, N, 256) * 1e-25).bfloat16()
    check(kmoe.moe_linear_w4(x, w), x, values(w), N == 2500)
