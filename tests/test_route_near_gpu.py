"""Routing with a bias where equal choice values cross the topk-th place and a different
one that FP32 cannot tell from them stands behind them."""

import pytest
import torch

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(scope="module")
def nvm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import nvfp4_weight_quantized_moe_b200 as nvm
    return nvm


def _route(nvm, logits, bias, topk, score, groups=1, keep=1):
    m = logits.shape[0]
    ids = torch.empty(m, topk, dtype=torch.int32, device="cuda")
    weights = torch.empty(m, topk, device="cuda")
    nvm.route_topk(logits, ids, weights, score=score, bias=bias, num_groups=groups, topk_groups=keep)
    torch.cuda.synchronize()
    return ids


def _by_definition(logits, bias, topk, score, groups=1, keep=1):
    l = logits.double()
    if score == "softmax":
        p = (l - l.amax(dim=1, keepdim=True)).exp()
        p = p / p.sum(dim=1, keepdim=True)
    else:
        p = 1.0 / (1.0 + (-l).exp())
    choice = p + bias.double()
    if groups > 1:
        best = choice.view(l.shape[0], groups, -1).amax(dim=2)
        order = best.sort(dim=1, descending=True, stable=True).indices[:, :keep]
        kept = torch.zeros_like(best, dtype=torch.bool).scatter_(1, order, True)
        choice = choice.masked_fill(~kept.repeat_interleave(l.shape[1] // groups, dim=1), -INF)
    return choice.sort(dim=1, descending=True, stable=True).indices[:, :topk].to(torch.int32)


@pytest.mark.parametrize("experts", [16, 33, 64, 128, 256, 1000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_saturated_scores(nvm, experts, dtype):
    """Sigmoids that are 1 in FP32: a run of equal logits, then larger ones."""
    for topk in (1, 2, 7, 8):
        for equal in (topk, topk + 1, min(experts - 3, 20)):
            logits = torch.zeros(4, experts, device="cuda")
            logits[:, :equal] = 20.0
            logits[0, equal] = 30.0
            logits[1, equal:equal + 3] = 25.0
            logits[2, experts - 1] = 22.0
            logits = logits.to(dtype)
            bias = torch.zeros(experts, device="cuda")
            got = _route(nvm, logits, bias, topk, "sigmoid")
            assert torch.equal(got, _by_definition(logits, bias, topk, "sigmoid")), (topk, equal)


@pytest.mark.parametrize("groups,keep", [(1, 1), (16, 5), (8, 3)])
def test_vanishing_scores(nvm, groups, keep):
    """Softmax scores under the FP32 range: equal ones first, larger ones behind them."""
    g = torch.Generator(device="cuda").manual_seed(1)
    logits = (torch.randn(20000, 64, generator=g, device="cuda") * 2).round() * 50.0
    bias = torch.zeros(64, device="cuda")
    got = _route(nvm, logits, bias, 3, "softmax", groups, keep)
    assert torch.equal(got, _by_definition(logits, bias, 3, "softmax", groups, keep))


@pytest.mark.parametrize("score,amp", [("sigmoid", 4.0), ("sigmoid", 8.0), ("softmax", 2.5)])
def test_scores_of_few_values_with_whole_biases(nvm, score, amp):
    """Many equal choice values, and values that a bias of 1 brings next to others."""
    g = torch.Generator(device="cuda").manual_seed(2)
    logits = (torch.randn(50000, 128, generator=g, device="cuda") * 2).round() * amp
    bias = torch.randn(128, generator=g, device="cuda").round()
    got = _route(nvm, logits, bias, 8, score)
    want = _by_definition(logits, bias, 8, score)
    # Where 64 bits cannot tell two values apart either, any of them is right: both
    # choices' values in 64 bits, in order.
    p = torch.softmax(logits.double(), 1) if score == "softmax" else 1.0 / (1.0 + (-logits.double()).exp())
    c = p + bias.double()
    off = (c.gather(1, got.long()) - c.gather(1, want.long())).abs()
    assert bool((off <= 8 * 2.0 ** -53 * (c.abs().amax() + 1)).all())
