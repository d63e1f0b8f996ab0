"""What a layer call with a routing rule refuses before the library is called. No GPU."""
import pytest
import torch

from fine_grained_sparse_fp32_b200 import _build, kmoe
from fine_grained_sparse_fp32_b200.inputs import LayerConfig, make_inputs


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    kmoe.load()


def handles():
    cfg = LayerConfig("l", 4, 256, 8, 2, 128, "bf16", "w4")
    layer = make_inputs(cfg, seed=1)
    return cfg, layer, kmoe.Layer(layer, 4, routing=kmoe.Routing()), kmoe.Layer(layer, 4, block=True, routing=kmoe.Routing())


def refuses(call, word):
    with pytest.raises(ValueError, match=word):
        call()


def test_routed_layer_calls_refuse_tensors_the_library_would_misread(monkeypatch):
    cfg, layer, plain, block = handles()
    x, g = layer["x"], torch.ones(256, dtype=torch.bfloat16)
    monkeypatch.setattr(kmoe, "_on_gpu", lambda t, name: None)      # (these tensors are on the CPU)
    monkeypatch.setattr(kmoe, "_call", lambda *a: None)
    plain.forward(x)
    block.block_forward(x, g, g, 1e-6)
    wrong = [(dict(x=x[:, :128].contiguous()), "x"), (dict(x=x.t().contiguous().t()), "x"), (dict(x=x.half()), "x"),
             (dict(y=x[:2]), "y"), (dict(topk_idx=torch.empty((4, 2), dtype=torch.int64)), "topk_idx"),
             (dict(topk_w=torch.empty((4, 3))), "topk_w"), (dict(counts=torch.empty(7, dtype=torch.int32)), "counts")]
    for kw, word in wrong:
        refuses(lambda: plain.forward(**dict(dict(x=x), **kw)), word)
    wrong = [(dict(h=x[:, :128].contiguous()), "h"), (dict(h=x.float()), "h"), (dict(gamma_pre=g.float()), "gamma_pre"),
             (dict(gamma_post=g[:128]), "gamma_post"), (dict(h_out=x[:2]), "h_out"), (dict(x_out=x.float()), "x_out"),
             (dict(counts=torch.empty(8)), "counts")]
    for kw, word in wrong:
        refuses(lambda: block.block_forward(**dict(dict(h=x, gamma_pre=g, gamma_post=g, eps=1e-6), **kw)), word)
    for name, t in (("w_router", layer["w_router"].bfloat16()), ("bias", layer["bias"][:4])):
        bad = kmoe.Layer(dict(layer, **{name: t}), 4, routing=kmoe.Routing())
        refuses(lambda: bad.forward(x), name)


def test_routed_layer_calls_refuse_tensors_of_the_host():
    cfg, layer, plain, block = handles()
    g = torch.ones(256, dtype=torch.bfloat16)
    refuses(lambda: plain.forward(layer["x"]), "CUDA")
    refuses(lambda: block.block_forward(layer["x"], g, g, 1e-6), "CUDA")


def test_rules_and_4_bit_weights_cannot_be_changed_behind_their_struct():
    rule = kmoe.Routing(n_groups=2, topk_groups=1, scale=2.0)
    w = kmoe.W4(torch.zeros((16, 128), dtype=torch.uint8), torch.ones((16, 2), dtype=torch.bfloat16))
    for thing, name, value in ((rule, "scale", 1.0), (rule, "topk_groups", 2), (w, "scales", w.scales.clone()), (w, "zeros", None)):
        with pytest.raises(AttributeError, match=name):
            setattr(thing, name, value)
    assert rule.scale == 2.0 and rule._struct.scale == 2.0
    w.scales.fill_(0.5)                       # values are the caller's to change
