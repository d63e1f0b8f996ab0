"""4-bit products on the tensor cores whose waits run out."""
import pytest
import torch

from fine_grained_sparse_fp32_b200 import _build, kmoe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    kmoe.load()


@pytest.mark.parametrize("cols", [384, 512, 8192])
def test_calls_after_one_that_gave_up_are_right(cols):
    """Few blocks of columns a unit, so that the loads are all asked for when the other warps give up: a call
    with the usual limit right behind it, and the next ones, are not disturbed by what was still in flight."""
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.randn((1200, cols), device="cuda", generator=g).bfloat16()
    w = kmoe.moe_quant_w4(torch.randn((1500, cols), device="cuda", generator=g) * 0.03)
    assert kmoe.moe_linear_w4_workspace_size(1200, 1200, 1500, cols) > 0
    want = kmoe.moe_linear_w4(x, w)
    try:
        for _ in range(20):
            kmoe.moe_set_wait_limit(1)
            kmoe.moe_linear_w4(x, w)
            kmoe.moe_set_wait_limit(0)
            assert torch.equal(kmoe.moe_linear_w4(x, w), want)
    finally:
        kmoe.moe_set_wait_limit(0)


def test_every_call_that_gave_up_says_so():
    """Many short products whose waits all run out: the word that reports it is cleared before any CTA can write it."""
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((1300, 8192), device="cuda", generator=g).bfloat16()
    w = kmoe.moe_quant_w4(torch.randn((700, 8192), device="cuda", generator=g) * 0.03)
    ws = torch.empty(kmoe.moe_linear_w4_workspace_size(1300, 1300, 700, 8192), dtype=torch.uint8, device="cuda")
    ws[:256] = 0
    try:
        for _ in range(30):
            kmoe.moe_set_wait_limit(1)
            kmoe.moe_linear_w4(x, w, ws=ws)
            assert kmoe.moe_device_status(ws) == 1
            kmoe.moe_set_wait_limit(0)
            kmoe.moe_linear_w4(x, w, ws=ws)
            assert kmoe.moe_device_status(ws) == 0
    finally:
        kmoe.moe_set_wait_limit(0)
