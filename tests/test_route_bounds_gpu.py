"""Choices of moe_route that lie next to what FP32 scores can tell apart, against the plain FP64 form."""
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


def check_route(logits, K, bias, **kw):
    idx, w = kmoe.moe_route(logits, K, bias=bias, routing=kmoe.Routing(**kw))
    ri, rw = plain_ops.route(logits, K, bias, **kw)
    assert torch.equal(idx.cpu(), ri)
    # FP32 arithmetic of an exponential, a sum and quotients: under 16 roundings of 2^-24 (a sum of many terms
    # next to 2^-24 of the first adds as many more)
    assert torch.allclose(w.cpu().double(), rw, rtol=(16 + logits.shape[1] / kw.get("n_groups", 1)) * 2.0 ** -24, atol=1e-37)


@pytest.mark.parametrize("E,groups", [(1020, 17), (1008, 18), (512, 16), (720, 9)])
@pytest.mark.parametrize("term", [-16.64, -16.63])
@pytest.mark.parametrize("by", ["max", "top2"])
def test_softmax_with_many_terms_next_to_the_last_place(E, groups, term, by):
    """The first expert's group holds terms just below (-16.64) or above (-16.63) half of the last place of 1, which
    an FP32 sum loses or doubles one by one, and a bias brings another group's expert within that of the first. Every
    other choice is far from the next."""
    size = E // groups
    logits = torch.full((1, E), -60.0)
    logits[0, :size] = term
    logits[0, 0] = 0.0
    other = E - size + 2
    s = torch.softmax(logits[0].double(), 0)
    for gap in torch.linspace(-6e-6, 6e-6, 121).tolist():
        bias = -0.01 * (torch.arange(E) // size + 1.0) - 0.01 * (torch.arange(E) % size != 0)
        bias[0] = 0.0
        bias[other] = float(s[0] - s[other] + gap)
        check_route(logits.cuda(), 2, bias.cuda(), score="softmax", n_groups=groups, topk_groups=3, group_score=by,
                    renormalise=False)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups,keep,by", [(1, 1, "max"), (8, 3, "max"), (8, 3, "top2"), (32, 9, "top2")])
@pytest.mark.parametrize("large", [-1e9, 100.0, 1e9, -3e38])
def test_experts_with_a_bias_far_from_the_others(score, groups, keep, by, large):
    """A large finite bias: experts switched off by it (of some groups all, or all but one), and experts it prefers."""
    g = torch.Generator(device="cuda").manual_seed(groups)
    E, K = 64, 6
    logits = torch.randn((40, E), device="cuda", generator=g)
    logits[1] = logits[1].round()                            # ties
    logits[2] = 1.0 + torch.randint(0, 3, (E,), device="cuda", generator=g) * 2.0 ** -23
    for n in (1, 5, 20, 61):
        bias = torch.rand(E, device="cuda", generator=g) * 0.1
        bias[torch.randperm(E, device="cuda", generator=g)[:n]] = large
        check_route(logits, K, bias, score=score, n_groups=groups, topk_groups=keep, group_score=by, renormalise=n < 20)
    bias = torch.rand(E, device="cuda", generator=g) * 0.1
    bias[:24] = large                                        # whole groups
    bias[3] = 0.05
    check_route(logits, K, bias, score=score, n_groups=groups, topk_groups=keep, group_score=by)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("by", ["max", "top2"])
def test_scores_next_to_each_other_among_large_biases(score, by):
    """Biases of 1, 100 and 1e6 that differ by a few FP32 places, where s decides below those places or not."""
    g = torch.Generator(device="cuda").manual_seed(3)
    E = 48
    logits = torch.randn((64, E), device="cuda", generator=g) * 3
    for at in (1.0, 100.0, 1e6):
        bias = at * (1 + torch.randint(-3, 4, (E,), device="cuda", generator=g) * 2.0 ** -23)
        for groups, keep in ((1, 1), (6, 2), (12, 7)):
            check_route(logits, 4, bias, score=score, n_groups=groups, topk_groups=keep, group_score=by)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("low", [-40.0, -60.0, -75.0, -100.0])
def test_renormalised_weights_of_scores_far_below_the_largest(score, low):
    """The bias chooses experts whose scores lie down to e^-105 below the largest one (or 1): their shares of the sum
    do not lose places to FP32's smallest numbers. Each logit's distance from the largest choice, 40 at most, is off by
    one rounding, which its exponential multiplies: 40 more roundings than check_route allows."""
    g = torch.Generator(device="cuda").manual_seed(int(-low))
    E, K = 64, 6
    logits = low - torch.rand((50, E), device="cuda", generator=g) * 5
    logits[:, ::7] -= 35
    logits[:, 3] = 2.0
    bias = torch.zeros(E, device="cuda")
    bias[torch.randperm(E, device="cuda", generator=g)[:12]] = 3.0 + 0.1 * torch.arange(12, device="cuda")
    bias[3] = -1.0
    for groups, keep in ((1, 1), (8, 5)):
        kw = dict(score=score, n_groups=groups, topk_groups=keep, group_score="max", renormalise=True)
        idx, w = kmoe.moe_route(logits, K, bias=bias, routing=kmoe.Routing(**kw))
        ri, rw = plain_ops.route(logits, K, bias, **kw)
        assert torch.equal(idx.cpu(), ri)
        assert torch.allclose(w.cpu().double(), rw, rtol=56 * 2.0 ** -24, atol=1e-37)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_equal_logits_at_the_end_of_the_choice_hide_no_third(score, dtype):
    """The last choice and the first that goes are equal, and an expert of a lower index has another logit but the same
    FP64 score: saturated sigmoids, scores that are 0, and logits whose places are below those of their scores."""
    E = 42
    rows = []
    for pair, third, rest in ((82.0, 56.0, -1.0), (40.0, 39.0, 3.0), (-760.0, -800.0, -900.0), (1e-9, 1e-9 - 1.1e-16, -2.0)):
        l = torch.full((E,), rest)
        l[[17, 19, 35]] = pair
        l[10] = third
        if pair < 0:
            l[5] = 1.0                                       # the largest, which is chosen first
        rows.append(l)
    logits = torch.stack(rows).to(dtype).cuda()
    for K in (1, 2, 3):
        for groups, keep in ((1, 1), (2, 1), (6, 1), (6, 2), (21, 1), (21, 3)):
            if keep * E // groups >= K:
                for by in ("max", "top2"):
                    check_route(logits, K, None, score=score, n_groups=groups, topk_groups=keep, group_score=by, renormalise=False)


@pytest.mark.parametrize("renormalise", [False, True])
def test_sigmoids_down_to_the_smallest_numbers(renormalise):
    """Scores of logits below -88.7, where e^-l is infinite in FP32, are not 0 yet: each is off by at most a half of
    2^-149, and a share of a sum of 0.01 or more by 2^-143."""
    logits = torch.full((60, 8), -200.0, device="cuda")
    logits[:, 0] = -4.0
    logits[:, 1] = -86.0 - torch.arange(60, device="cuda") * 0.3
    bias = torch.tensor([2.0, 1.0, 0.0, 0, 0, 0, 0, 0], device="cuda")
    kw = dict(score="sigmoid", renormalise=renormalise)
    idx, w = kmoe.moe_route(logits, 2, bias=bias, routing=kmoe.Routing(**kw))
    ri, rw = plain_ops.route(logits, 2, bias, **kw)
    assert torch.equal(idx.cpu(), ri)
    assert torch.allclose(w.cpu().double(), rw, rtol=16 * 2.0 ** -24, atol=2.0 ** -143)
