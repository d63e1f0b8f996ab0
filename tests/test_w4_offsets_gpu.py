"""Grouped 4-bit products of so many rows that blocks of rows and their cost come near 32 bits."""
import pytest
import torch

from fine_grained_sparse_fp32_b200 import _build, kmoe
import plain_ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    kmoe.load()


def matrices(E):
    g = torch.Generator(device="cuda").manual_seed(E)
    return g, kmoe.moe_quant_w4(torch.randn((E, 1, 128), device="cuda", generator=g)), \
        torch.randn((4, 128), device="cuda", generator=g).bfloat16()


@pytest.mark.parametrize("y_dtype", [torch.float32, torch.bfloat16])
def test_many_rows_of_many_experts(y_dtype):
    E, P = 1024, (1 << 25) + 3
    g, w, x = matrices(E)
    perm = torch.randint(0, 4, (P,), dtype=torch.int32, device="cuda", generator=g)
    cuts = torch.randint(0, P, (E - 1,), device="cuda", generator=g).sort().values
    offsets = torch.cat((cuts.new_tensor([0]), cuts, cuts.new_tensor([P]))).int()
    y = kmoe.moe_linear_w4(x, w, perm, offsets, y_dtype=y_dtype)
    v = plain_ops.w4_values(w.codes, w.scales)[:, 0]
    expert = torch.searchsorted(offsets[1:].long(), torch.arange(P, device="cuda"), right=True)
    at = expert * 4 + perm
    ref, size = (v @ x.double().t()).flatten()[at, None], (v.abs() @ x.double().abs().t()).flatten()[at, None]
    # one rounding to BF16 (2^-8); in FP32 cols / 16 partial sums, cols / 32 scaled ones and 8 more, two roundings of
    # 2^-24 of the sum of magnitudes each
    tol = (2.0 ** -8 * ref.abs() if y_dtype == torch.bfloat16 else 0) + (128 / 16 + 128 / 32 + 8) * 2.0 ** -23 * size
    assert ((y.double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("y_dtype", [torch.float32, torch.bfloat16])
def test_nothing_is_done_for_descending_offsets_of_that_size(y_dtype):
    """Every second expert's range holds all rows: together more blocks than 32 bits count."""
    E, P = 1024, 1 << 28
    _, w, x = matrices(E)
    perm = torch.zeros(P, dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, P] * (E // 2) + [0], dtype=torch.int32, device="cuda")
    y = torch.full((P, 1), 7.0, dtype=y_dtype, device="cuda")
    kmoe.moe_linear_w4(x, w, perm, offsets, out=y)
    assert (y == 7).all()
