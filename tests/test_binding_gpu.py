"""The binding's handling of streams and of tensors that the library would misread."""
import pytest
import torch

from fine_grained_sparse_fp32_b200 import _build, kmoe
from fine_grained_sparse_fp32_b200.inputs import LayerConfig, make_block_inputs, make_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    kmoe.load()


def small(w_dtype="w4", N=24):
    cfg = LayerConfig("l", N, 512, 64, 6, 128, "bf16", w_dtype, w4_group=64)
    return cfg, make_inputs(cfg, seed=3, device="cuda"), kmoe.Routing(n_groups=8, topk_groups=3)


@pytest.mark.parametrize("with_outputs", [False, True])
@pytest.mark.parametrize("routed", [False, True])
def test_memory_of_a_call_on_a_stream_is_that_streams(with_outputs, routed, monkeypatch):
    """Workspace and outputs come from the memory of the stream that the call is given: what is freed on return is
    reused by that stream alone, behind the call's kernels."""
    cfg, layer, rule = small()
    b = make_block_inputs(cfg, 3, "cuda")
    rule = rule if routed else None
    want = kmoe.moe_forward(layer["x"], layer, routing=rule)
    block = kmoe.moe_block_forward(b["h"], layer, b["gamma_pre"], b["gamma_post"], 1e-6, routing=rule)
    torch.cuda.synchronize()
    st, seen = torch.cuda.Stream(), []
    for name in ("empty", "empty_like"):
        def made(*a, _f=getattr(torch, name), **kw):
            seen.append(torch.cuda.current_stream())
            return _f(*a, **kw)
        monkeypatch.setattr(torch, name, made)
    got = kmoe.moe_forward(layer["x"], layer, routing=rule, stream=st, with_outputs=with_outputs)
    got2 = kmoe.moe_block_forward(b["h"], layer, b["gamma_pre"], b["gamma_post"], 1e-6, routing=rule, stream=st, with_outputs=with_outputs)
    handle_forward = len(seen)
    monkeypatch.undo()
    assert handle_forward >= 4 and all(s == st for s in seen)
    assert torch.cuda.current_stream() != st
    st.synchronize()
    assert torch.equal(got[0] if with_outputs else got, want)
    assert torch.equal(got2[0] if with_outputs else got2, block)


def test_outputs_of_a_handle_on_a_stream(monkeypatch):
    cfg, layer, rule = small()
    handle, st, seen = kmoe.Layer(layer, cfg.N, routing=rule), torch.cuda.Stream(), []
    want = handle.forward(layer["x"])
    torch.cuda.synchronize()

    def made(*a, _f=torch.empty, **kw):
        seen.append(torch.cuda.current_stream())
        return _f(*a, **kw)
    monkeypatch.setattr(torch, "empty", made)
    y = handle.forward(layer["x"], stream=st)
    monkeypatch.undo()
    st.synchronize()
    assert seen == [st] and torch.equal(y, want)


def test_a_workspace_elsewhere_is_refused():
    g = torch.Generator(device="cuda").manual_seed(1)
    w = kmoe.moe_quant_w4(torch.randn((700, 256), device="cuda", generator=g))
    x = torch.randn((2500, 256), device="cuda", generator=g).bfloat16()
    need = kmoe.moe_linear_w4_workspace_size(2500, 2500, 700, 256)
    assert need > 0
    for bad in (torch.empty(need, dtype=torch.uint8), torch.empty(need, dtype=torch.int16, device="cuda"),
                torch.empty(2 * need, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            kmoe.moe_linear_w4(x, w, ws=bad)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert torch.equal(kmoe.moe_linear_w4(x, w, ws=ws), kmoe.moe_linear_w4(x, w))
