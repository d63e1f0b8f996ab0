"""Routing and 4-bit operators on the GPU against plain 64-bit forms.

Tolerances. A rounding to BF16 is off by at most 2^-8 of the value. A product with 4-bit weights takes x in
fixed point, for each 128 columns off by at most 2^-14 of their largest |x| (2^-22 for FP32 results, which take
one digit more); the sums of a group are exact, and in FP32 follow, for each digit group of x, one scaled sum
per group of weights (at most cols / 32, each two roundings of 2^-24 and the addition's) and the joining of
digits and of at most 16 column shares, all relative to S = sum |W| |x| (a digit's own sum of magnitudes is
below 2 S): in all less than (cols / 16 + cols / 32 + 8) * 2^-23 * S plus sum |W| 2^-14 (or 2^-22) max|x|.
Batches on the tensor cores (BF16 results) round each weight to FP16, 2^-11 S, have x exact to 2^-39 of a row's
largest value, and FP32 sums of cols / 16 partial sums. (There a zero point's product z s is rounded apart, by
2^-11 at worst and for odd z above 8 only; no allowance is made for it.) For the FFN the errors of both sums go through
SiLU(g) * u, whose slopes are |dh/dg| <= 1.1 |u| and |dh/du| = |SiLU(g)|; the hardware exponential and reciprocal are off by less than 2^-20 together; H is rounded to BF16 at worst;
all of it goes through |W_d|.
"""
import numpy as np
import pytest
import torch

from fine_grained_sparse_fp32_b200 import _build, kmoe
from fine_grained_sparse_fp32_b200.inputs import CONFIGS, LayerConfig, make_block_inputs, make_inputs
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


# ------------------------------------------------------------------ quantiser
@pytest.mark.parametrize("rows,cols", [(1, 128), (7, 384), (513, 256), (3, 2560)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quant_w4_is_bit_exact(rows, cols, group, zeros, dtype):
    w = randn(gen(rows + cols), rows, cols) * 0.02
    w[0, :32] = 0.0                                        # a group of zeros (where the group is 32)
    w[-1, -32:] = torch.linspace(0.5, 3.0, 32)             # one sign only
    if rows > 2:
        w[1, :group] *= 1e-38                              # denormal values, a scale that rounds to a denormal
        w[2, :group] *= 1e30
    w = w.to(dtype)
    got = kmoe.moe_quant_w4(w, group=group, zeros=zeros)
    q, s, z = plain_ops.quant_w4(w, group, zeros)
    assert torch.equal(plain_ops.w4_codes(got.codes).cpu().to(torch.uint8), q)
    assert torch.equal(got.scales.cpu(), s)
    assert (got.zeros is None) == (z is None) and (z is None or torch.equal(got.zeros.cpu(), z))
    ref = plain_ops.w4_values(got.codes, got.scales, got.zeros)
    assert torch.equal(kmoe.moe_dequant_w4(got, dtype=torch.float32).double(), ref)
    assert torch.equal(kmoe.moe_dequant_w4(got), ref.float().to(torch.bfloat16))


def test_quant_w4_stacks_overwrites_and_takes_no_rows():
    w = randn(gen(1), 3, 20, 256)
    a = kmoe.moe_quant_w4(w, group=64)
    for e in range(3):
        b = kmoe.moe_quant_w4(w[e], group=64)
        assert torch.equal(a.codes[e], b.codes) and torch.equal(a.scales[e], b.scales)
    c = kmoe.moe_quant_w4(w * 2, group=64, out=a)
    assert c is a and torch.equal(c.scales[0], kmoe.moe_quant_w4(w[0] * 2, group=64).scales)
    with pytest.raises(ValueError):
        kmoe.moe_quant_w4(w, group=64, zeros=True, out=a)
    with pytest.raises(ValueError):
        kmoe.moe_quant_w4(w.transpose(0, 1), group=64)
    none = kmoe.moe_quant_w4(torch.empty((0, 256), device="cuda"))
    assert none.codes.shape == (0, 128) and kmoe.moe_dequant_w4(none).shape == (0, 256)


# -------------------------------------------------------------------- routing
def check_route(logits, K, bias, **kw):
    idx, w = kmoe.moe_route(logits, K, bias=bias, routing=kmoe.Routing(**kw))
    ri, rw = plain_ops.route(logits, K, bias, **kw)
    assert torch.equal(idx.cpu(), ri)
    # FP32 arithmetic of an exponential, a sum and quotients: under 16 roundings of 2^-24
    assert torch.allclose(w.cpu().double(), rw, rtol=16 * 2.0 ** -24, atol=1e-37)


@pytest.mark.parametrize("N,E,K,groups,keep", [
    (1, 384, 6, 1, 1), (33, 384, 6, 8, 4), (9, 384, 8, 8, 1), (5, 1024, 8, 3 - 1, 1), (17, 61, 5, 1, 1), (4, 8, 8, 1, 1),
    (3, 1, 1, 1, 1), (12, 63, 4, 3, 2), (40, 256, 8, 32, 4), (6, 96, 2, 6, 5), (8, 1023, 7, 11, 2), (5, 200, 3, 25, 25),
    (300, 64, 6, 16, 4)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("by", ["max", "top2"])
def test_route_matches_the_definition(N, E, K, groups, keep, score, by):
    g = gen(N + E)
    logits = randn(g, N, E) * 2
    bias = torch.rand(E, device="cuda", generator=g) * 0.2 - 0.1
    for renorm, scale, b, l in ((True, 2.5, bias, logits), (False, 1.0, None, logits), (True, 1.0, bias, logits.bfloat16()),
                                (False, 0.5, None, logits.bfloat16())):
        check_route(l.contiguous(), K, b, score=score, n_groups=groups, topk_groups=keep, group_score=by,
                    renormalise=renorm, scale=scale)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_ties_masks_and_non_finite_logits(score):
    inf, nan = float("inf"), float("nan")
    E, K = 64, 6
    g = gen(5)
    logits = randn(g, 14, E)
    logits[0] = 0.25                                         # all equal: lowest indices
    logits[1] = -inf                                         # nothing left: experts 0.., weight 0
    logits[2, 3:] = -inf                                     # fewer than K left
    logits[3, ::2] = nan
    logits[4] = torch.randint(0, 3, (E,), device="cuda", generator=g).float()
    logits[5, 10] = inf
    logits[6] = 40.0 + torch.arange(E, device="cuda")        # sigmoid is 1 in FP64: ties
    logits[7] = 17.0 + torch.arange(E, device="cuda") * 1e-5     # sigmoid is 1 in FP32, not in FP64
    logits[8] = -200.0 - torch.arange(E, device="cuda")      # scores that are 0 in FP32
    logits[9] = 1.0 + torch.randint(0, 3, (E,), device="cuda", generator=g) * 2.0 ** -23   # neighbours in FP32
    logits[10, :60] = -inf
    logits[11] = -88.0 - torch.rand(E, device="cuda", generator=g)
    logits[12] = -700.0 - torch.arange(E, device="cuda")     # scores that are 0 in FP64 from somewhere on
    logits[13] = -torch.arange(E, device="cuda") * 40.0
    bias = torch.rand(E, device="cuda", generator=g) * 0.1
    off = bias.clone()
    off[torch.arange(0, E, 3)] = -inf
    off[7] = nan
    up = bias.clone()
    up[[50, 20]] = inf
    for b in (None, bias, off, up):
        for groups, keep in ((1, 1), (8, 2), (8, 1), (4, 3)):
            for by in ("max", "top2"):
                check_route(logits, K, b, score=score, n_groups=groups, topk_groups=keep, group_score=by)


def test_route_large_batch_is_deterministic_and_empty_batch_returns():
    logits = randn(gen(9), 30000, 384)
    bias = torch.rand(384, device="cuda") * 0.1
    r = kmoe.Routing(n_groups=8, topk_groups=4)
    a, b = kmoe.moe_route(logits, 6, bias, r), kmoe.moe_route(logits, 6, bias, r)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    at = torch.randperm(30000)[:64]
    ri, _ = plain_ops.route(logits[at.cuda()], 6, bias, n_groups=8, topk_groups=4)
    assert torch.equal(a[0].cpu()[at], ri)
    idx, w = kmoe.moe_route(logits[:0], 6)
    assert idx.shape == (0, 6) and w.shape == (0, 6)


# ------------------------------------------------------------- 4-bit products
def make_w4(g, lead, rows, cols, group, zeros):
    shape = (lead, rows, cols // group)
    codes = torch.randint(0, 256, (lead, rows, cols // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = (torch.rand(shape, device="cuda", generator=g) * 0.02 + 0.001).to(torch.bfloat16)
    z = torch.randint(0, 16, shape, dtype=torch.uint8, device="cuda", generator=g) if zeros else None
    return kmoe.W4(codes, scales, z)


def sums_bound(x, w, cols, tensor_cores=False, y_dtype=torch.bfloat16):
    top = x.abs().unflatten(-1, (-1, 128)).amax(-1).repeat_interleave(128, -1)
    each = (cols / 16 + cols / 32 + 8) * 2.0 ** -23 + (2.0 ** -11 if tensor_cores else 0)
    return (each * x.abs() + (2.0 ** -22 if y_dtype == torch.float32 else 2.0 ** -14) * top) @ w.abs().t()


def check_linear(y, x, w, cols, rows=None):
    """rows: rows of the call (those of y, unless y is a part of them). From seven rows on it may run on
    the tensor cores."""
    ref = x @ w.t()
    tc = y.dtype == torch.bfloat16 and (rows or y.shape[0]) >= 7
    tol = sums_bound(x, w, cols, tc, y.dtype) + (BF16 * ref.abs() if y.dtype == torch.bfloat16 else 0) + 1e-30
    assert torch.isfinite(y).all()
    off = (y.double() - ref).abs() / tol
    assert off.max() <= 1, float(off.max())


@pytest.mark.parametrize("N", [1, 3, 8, 9, 17, 32, 33, 70, 129, 300])
@pytest.mark.parametrize("rows,cols", [(1, 128), (15, 384), (16, 640), (100, 2560), (515, 256), (17, 8192)])
def test_linear_w4_one_matrix(N, rows, cols):
    g = gen(N * 1000 + rows + cols)
    x = randn(g, N, cols).bfloat16()
    for group, zeros, y_dtype in ((128, False, torch.float32), (128, True, torch.bfloat16), (64, True, torch.float32),
                                  (64, False, torch.bfloat16), (32, False, torch.float32), (32, True, torch.bfloat16)):
        w = make_w4(g, 1, rows, cols, group, zeros)
        w = kmoe.W4(w.codes[0], w.scales[0], None if w.zeros is None else w.zeros[0])
        y = kmoe.moe_linear_w4(x, w, y_dtype=y_dtype)
        check_linear(y, x.double(), plain_ops.w4_values(w.codes, w.scales, w.zeros), cols)
        assert torch.equal(y, kmoe.moe_linear_w4(x, w, y_dtype=y_dtype))


@pytest.mark.parametrize("N,E,K", [(1, 16, 4), (5, 16, 4), (64, 7, 3), (300, 3, 2), (130, 61, 8), (2500, 3, 2), (1300, 16, 5)])
@pytest.mark.parametrize("group,zeros", [(32, True), (128, False)])
@pytest.mark.parametrize("y_dtype", [torch.float32, torch.bfloat16])
def test_linear_w4_grouped_by_expert(N, E, K, group, zeros, y_dtype):
    g = gen(N + E)
    rows, cols = 72, 384
    x = randn(g, N, cols).bfloat16()
    w = make_w4(g, E, rows, cols, group, zeros)
    idx = torch.rand((N, E), device="cuda", generator=g).topk(K, 1).indices.int()
    counts, offsets, perm, inv = kmoe.moe_permute(idx, E)
    y = kmoe.moe_linear_w4(x, w, perm, offsets, y_dtype=y_dtype)
    v = plain_ops.w4_values(w.codes, w.scales, w.zeros)
    off = offsets.tolist()
    for e in range(E):
        at = slice(off[e], off[e + 1])
        if off[e] < off[e + 1]:
            check_linear(y[at], x.double()[perm[at].long()], v[e], cols, rows=N * K)


def test_linear_w4_leaves_uncovered_rows_and_reads_no_foreign_token():
    g = gen(2)
    N, cols, rows = 6, 256, 40
    x = randn(g, N, cols).bfloat16()
    w = make_w4(g, 3, rows, cols, 64, True)
    perm = torch.tensor([0, 5, 2, 6, -1, 3, 1, 1, 2, 0], dtype=torch.int32, device="cuda")    # 6 and -1: no such token
    offsets = torch.tensor([1, 5, 5, 8], dtype=torch.int32, device="cuda")                    # rows 0, 8, 9: no expert
    out = torch.full((10, rows), 7.0, device="cuda")
    y = kmoe.moe_linear_w4(x, w, perm, offsets, out=out)
    assert y is out and (out[[0, 8, 9]] == 7).all()
    assert (out[[3, 4]] == 0).all()
    v = plain_ops.w4_values(w.codes, w.scales, w.zeros)
    check_linear(out[1:3], x.double()[[5, 2]], v[0], cols)
    check_linear(out[5:8], x.double()[[3, 1, 1]], v[2], cols)
    # ranges that reach outside the batch are cut to it
    out.fill_(7.0)
    kmoe.moe_linear_w4(x, w, perm, torch.tensor([-3, 2, 1, 99], dtype=torch.int32, device="cuda"), out=out)
    assert torch.isfinite(out).all()
    assert kmoe.moe_linear_w4(x[:0], w, perm[:0], offsets).shape == (0, rows)
    assert (kmoe.moe_linear_w4(x[:0], w, perm, torch.tensor([0, 4, 7, 10], dtype=torch.int32, device="cuda")) == 0).all()


def test_linear_w4_many_rows_uncovered_and_foreign():
    """As above, at a size that runs on the tensor cores (and an odd number of weight rows)."""
    g = gen(12)
    N, cols, rows, P = 50, 256, 301, 4000
    x = randn(g, N, cols).bfloat16()
    w = make_w4(g, 3, rows, cols, 128, True)
    assert kmoe.moe_linear_w4_workspace_size(N, P, rows, cols, 3, 128) > 0
    perm = torch.randint(0, N, (P,), dtype=torch.int32, device="cuda", generator=g)
    perm[[100, 2000]] = torch.tensor([-1, N], dtype=torch.int32, device="cuda")
    offsets = torch.tensor([70, 150, 150, 3900], dtype=torch.int32, device="cuda")
    out = torch.full((P, rows), 7.0, device="cuda", dtype=torch.bfloat16)
    kmoe.moe_linear_w4(x, w, perm, offsets, out=out)
    assert (out[:70] == 7).all() and (out[3900:] == 7).all() and (out[[100, 2000]] == 0).all()
    xs = x.double()[perm.clamp(0, N - 1).long()]
    xs[[100, 2000]] = 0
    v = plain_ops.w4_values(w.codes, w.scales, w.zeros)
    check_linear(out[70:150], xs[70:150], v[0], cols, rows=P)
    check_linear(out[150:3900], xs[150:3900], v[2], cols, rows=P)
    again = torch.full_like(out, 7.0)
    kmoe.moe_linear_w4(x, w, perm, offsets, out=again)
    assert torch.equal(out, again)


@pytest.mark.parametrize("N,y_dtype", [(5, torch.float32), (5, torch.bfloat16), (2500, torch.bfloat16)])
def test_linear_w4_takes_wide_ranges_of_values(N, y_dtype):
    """Large and tiny x and scales: sums stay in FP32 range and keep their relative accuracy."""
    g = gen(3)
    x = randn(g, N, 512) * torch.tensor([1e-20, 1e-3, 1.0, 1e4, 1e15], device="cuda").repeat(N // 5)[:, None]
    x = x.bfloat16()
    w = make_w4(g, 1, 33, 512, 128, False)
    w.scales.mul_(torch.logspace(-12, 10, 33, device="cuda")[None, :, None])
    w.scales[0, :, 1] *= 2.0 ** -9                         # groups of one row that differ widely
    w.scales[0, ::2, 2] *= 2.0 ** 7
    y = kmoe.moe_linear_w4(x, kmoe.W4(w.codes[0], w.scales[0]), y_dtype=y_dtype)
    check_linear(y, x.double(), plain_ops.w4_values(w.codes[0], w.scales[0]), 512)


@pytest.mark.parametrize("N", [6, 2500])
def test_linear_w4_keeps_non_finite_rows_to_themselves(N):
    g = gen(6)
    x = randn(g, N, 384).bfloat16()
    x[1, 7], x[N - 1, 300] = float("nan"), float("inf")
    w = make_w4(g, 1, 40, 384, 128, True)
    y = kmoe.moe_linear_w4(x, kmoe.W4(w.codes[0], w.scales[0], w.zeros[0]))
    fine = torch.ones(N, dtype=torch.bool, device="cuda")
    fine[[1, N - 1]] = False
    check_linear(y[fine], x[fine].double(), plain_ops.w4_values(w.codes[0], w.scales[0], w.zeros[0]), 384, rows=N)
    assert not torch.isfinite(y[1]).any() and not torch.isfinite(y[N - 1]).all()


@pytest.mark.parametrize("N,E,y_dtype", [(300000, 1, torch.bfloat16), (140000, 3, torch.bfloat16), (20000, 1, torch.float32),
                                         (9000, 3, torch.float32)])
def test_linear_w4_long_batches(N, E, y_dtype):
    """More blocks of tokens than the kernels' tables name: each row's result, and each expert's last row."""
    g = gen(N)
    rows, cols = 72, 128
    x = randn(g, 4096, cols).bfloat16()
    w = make_w4(g, E, rows, cols, 64, True)
    perm = torch.randint(0, 4096, (N,), dtype=torch.int32, device="cuda", generator=g)
    off = [0, N] if E == 1 else [0, N // 2 + 5, N // 2 + 5 + N // 3, N]
    y = kmoe.moe_linear_w4(x, w, perm, torch.tensor(off, dtype=torch.int32, device="cuda"), y_dtype=y_dtype)
    v = plain_ops.w4_values(w.codes, w.scales, w.zeros)
    for e in range(E):
        check_linear(y[off[e]:off[e + 1]], x.double()[perm[off[e]:off[e + 1]].long()], v[e], cols, rows=N)


def test_products_on_the_tensor_cores_give_up_and_report():
    """Waits run out (a limit of 100 clocks; a wait asleep in hardware looks again after 20 us, and the sums of
    8192 or 6144 columns of 256 rows and 128 tokens take longer): the kernels return, the status word says so,
    and the next call is right."""
    g = gen(21)
    x = randn(g, 1500, 8192).bfloat16()
    w = kmoe.moe_quant_w4(randn(g, 700, 8192) * 0.03)
    need = kmoe.moe_linear_w4_workspace_size(1500, 1500, 700, 8192)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    layer = make_inputs(LayerConfig("w4", 1500, 6144, 8, 2, 256, "bf16", "w4"), seed=3, device="cuda")
    idx = torch.rand((1500, 8), device="cuda", generator=g).topk(2, 1).indices.int()
    _, offsets, perm, _ = kmoe.moe_permute(idx, 8)
    handle = kmoe.Layer(layer, 1500)
    try:
        kmoe.moe_set_wait_limit(100)
        kmoe.moe_linear_w4(x, w, ws=ws)
        handle.grouped_ffn(layer["x"], perm, offsets)
        assert kmoe.moe_device_status(ws) == 1 and kmoe.moe_device_status(handle.ws) == 1
    finally:
        kmoe.moe_set_wait_limit(0)
    y = kmoe.moe_linear_w4(x, w, ws=ws)
    assert kmoe.moe_device_status(ws) == 0
    check_linear(y, x.double(), plain_ops.w4_values(w.codes, w.scales), 8192)
    check_ffn(layer, 1500, 2, 8, 77, handle=handle)
    assert kmoe.moe_device_status(handle.ws) == 0


# ------------------------------------------------------------- experts' FFN
def ffn_ref(x, layer, e, tc):
    """FP64 result and bound of expert e on rows x; tc: on the tensor cores."""
    z = lambda m: None if layer.get("z_" + m) is None else layer["z_" + m][e]
    wg, wu, wd = (plain_ops.w4_values(layer["w_" + m][e], layer["s_" + m][e], z(m)) for m in ("gate", "up", "down"))
    d, I = wg.shape[1], wg.shape[0]
    a, u = x @ wg.t(), x @ wu.t()
    h = a * torch.sigmoid(a) * u
    dh = 1.1 * u.abs() * sums_bound(x, wg, d, tc) + (a * torch.sigmoid(a)).abs() * sums_bound(x, wu, d, tc) \
        + 2.0 ** -20 * h.abs()
    dh = dh + BF16 * (h.abs() + dh)
    y = h @ wd.t()
    hh = h.abs() + dh
    return y, dh @ wd.abs().t() + sums_bound(hh, wd, I, tc) + BF16 * y.abs() + 1e-30


def check_ffn(layer, N, K, E, seed, with_shared=True, handle=None):
    cfg = layer["cfg"]
    g = gen(seed)
    x = randn(g, N, cfg.d).bfloat16()
    idx = torch.rand((N, E), device="cuda", generator=g).topk(K, 1).indices.int()
    _, offsets, perm, _ = kmoe.moe_permute(idx, E)
    handle = handle or kmoe.Layer(layer, N)
    y, ys = handle.grouped_ffn(x, perm, offsets, with_shared=with_shared)
    off = offsets.tolist()
    for e in range(E + 1):
        rows, got = (x, ys) if e == E else (x[perm[off[e]:off[e + 1]].long()], y[off[e]:off[e + 1]])
        if e == E and not with_shared:
            assert ys is None
            continue
        if rows.shape[0]:
            ref, tol = ffn_ref(rows.double(), layer, e, N * K >= 7 * E)
            off_by = ((got.double() - ref).abs() / tol).max()
            assert off_by <= 1, (e, float(off_by))
    return x, perm, offsets, y, ys


@pytest.mark.parametrize("N", [1, 2, 9, 40, 130, 260, 700, 1500])
@pytest.mark.parametrize("d,I,E,K,group,zeros", [(256, 128, 8, 2, 128, False), (384, 256, 5, 3, 32, True),
                                                 (1280, 128, 16, 6, 64, True), (512, 384, 4, 4, 64, False)])
def test_grouped_ffn_w4(N, d, I, E, K, group, zeros):
    cfg = LayerConfig("w4", N, d, E, K, I, "bf16", "w4", w4_group=group, w4_zeros=zeros)
    layer = make_inputs(cfg, seed=N, device="cuda")
    check_ffn(layer, N, K, E, N + d)
    check_ffn(layer, N, K, E, N + d, with_shared=False)


@pytest.mark.parametrize("name", ["w4_decode"])
def test_grouped_ffn_w4_full_width(name):
    cfg = CONFIGS[name]
    layer = make_inputs(cfg, seed=1, device="cuda")
    handle = kmoe.Layer(layer, cfg.N)
    x, perm, offsets, y, ys = check_ffn(layer, cfg.N, cfg.K, cfg.E, 4, handle=handle)
    y2, ys2 = handle.grouped_ffn(x, perm, offsets)
    assert torch.equal(y, y2) and torch.equal(ys, ys2)


# ------------------------------------------------- the operators in one layer
def route_agrees(idx, logits, K, bias, margin, **kw):
    """Tokens whose choice by FP64 logits is the same for every logit within `margin`."""
    ri, _ = plain_ops.route(logits, K, bias, **kw)
    return (idx.cpu() == ri).all(1).float().mean() >= 1 - margin


@pytest.mark.parametrize("N", [1, 20, 300, 600])
@pytest.mark.parametrize("w_dtype", ["w4", "bf16"])
def test_layer_with_the_new_routing(N, w_dtype):
    """Route, dispatch, experts and combine in one call: the choice follows the router's logits, and the
    result is the weighted sum of the experts' outputs for that choice."""
    cfg = LayerConfig("l", N, 512, 64, 6, 128, "bf16", w_dtype, w4_group=64, w4_zeros=True)
    layer = make_inputs(cfg, seed=7, device="cuda")
    kw = dict(score="sigmoid", n_groups=8, topk_groups=3, group_score="top2", renormalise=True, scale=2.5)
    y, idx, w, counts = kmoe.moe_forward(layer["x"], layer, with_outputs=True, y_dtype=torch.float32,
                                         routing=kmoe.Routing(**kw))
    logits = layer["x"].double() @ layer["w_router"].double().t()
    # logits in FP32 are off by some 1e-6, so only near-ties may fall the other way
    assert route_agrees(idx, logits, cfg.K, layer["bias"], 0.02, **kw)
    assert torch.equal(counts.cpu(), torch.bincount(idx.cpu().flatten().long(), minlength=cfg.E).int())
    s = torch.sigmoid(logits).gather(1, idx.long())
    rw = 2.5 * s / s.sum(1, keepdim=True)
    assert torch.allclose(w.double(), rw, rtol=1e-4, atol=0)
    handle = kmoe.Layer(layer, N)
    _, offsets, perm, inv = kmoe.moe_permute(idx, cfg.E)
    yp, ys = handle.grouped_ffn(layer["x"], perm, offsets)
    ref = ys.double() + (w.double()[..., None] * yp.double()[inv.long()]).sum(1)
    assert torch.allclose(y.double(), ref, rtol=1e-5, atol=1e-5 * float(ref.abs().max()))
    # the sandwich block takes the same rule
    b = make_block_inputs(cfg, 3, "cuda")
    out, x, bidx, bw, _ = kmoe.moe_block_forward(b["h"], layer, b["gamma_pre"], b["gamma_post"], 1e-6, with_outputs=True,
                                                 routing=kmoe.Routing(**kw))
    m, midx, mw, _ = kmoe.moe_forward(x, layer, with_outputs=True, y_dtype=torch.float32, routing=kmoe.Routing(**kw))
    assert torch.equal(bidx, midx) and torch.equal(bw, mw)
    m = m.double()
    post = m / (m.square().mean(1, keepdim=True) + 1e-6).sqrt() * b["gamma_post"].double()
    want = b["h"].double() + post
    assert ((out.double() - want).abs() <= BF16 * want.abs() + 1e-4 * post.abs() + 1e-6).all()


def test_layer_without_a_bias_and_old_rule_unchanged():
    cfg = LayerConfig("l", 40, 512, 64, 6, 128, "bf16", "w4")
    layer = make_inputs(cfg, seed=8, device="cuda")
    plain = dict(layer, bias=None)
    y, idx, w, _ = kmoe.moe_forward(layer["x"], plain, with_outputs=True, routing=kmoe.Routing(score="softmax"))
    zero = dict(layer, bias=torch.zeros(64, device="cuda"))
    y0, idx0, w0, _ = kmoe.moe_forward(layer["x"], zero, with_outputs=True, routing=kmoe.Routing(score="softmax"))
    assert torch.equal(y, y0) and torch.equal(idx, idx0) and torch.equal(w, w0)
    # the rule of `score` still selects on logits + bias and leaves the weights as they are
    _, idx1, w1, _ = kmoe.moe_forward(layer["x"], layer, with_outputs=True)
    logits = layer["x"].double() @ layer["w_router"].double().t()
    assert torch.allclose(w1.double(), torch.sigmoid(logits).gather(1, idx1.long()), atol=1e-5)


def test_a_stream_of_its_own_and_graphs_that_run_at_once():
    cfg = LayerConfig("l", 24, 512, 64, 6, 128, "bf16", "w4", w4_group=32)
    layer = make_inputs(cfg, seed=9, device="cuda")
    r = kmoe.Routing(n_groups=4, topk_groups=2)
    handles = [kmoe.Layer(layer, cfg.N, routing=r) for _ in range(2)]
    xs = [layer["x"].clone(), (layer["x"] * 0.5).contiguous()]
    want = [handles[0].forward(x).clone() for x in xs]
    w = kmoe.moe_quant_w4(randn(gen(4), 130, 512))
    lin = kmoe.moe_linear_w4(xs[0], w).clone()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs, ys = [], []
    for h, x, st in zip(handles, xs, streams):
        y = torch.empty_like(x)
        with torch.cuda.stream(st):
            h.forward(x, y=y)                                     # the current stream is this one
            z = kmoe.moe_linear_w4(x, w, stream=st)
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            h.forward(x, y=y)
            z = kmoe.moe_linear_w4(x, w)
        graphs.append(g)
        ys.append((y, z))
    for rep in range(3):
        for y, z in ys:
            y.zero_()
            z.zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        assert torch.equal(ys[0][0], want[0]) and torch.equal(ys[1][0], want[1])
        assert torch.equal(ys[0][1], lin)
    # new values in the captured input
    xs[0].copy_(xs[1])
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(ys[0][0], want[1])
