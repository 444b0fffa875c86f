"""Group choice of the routing where a group's score is a sum of values of opposite signs.

The score of a group is then small and its parts are not: FP32 rounds each part by up to
2^-24 of the part's size, so scores that differ by more than the sum's own rounding may
still be in the wrong order.  ids have to be those of the definition in 64 bits.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu

LOWEST, LARGEST = torch.finfo(torch.float32).min, torch.finfo(torch.float32).max
INF = float("inf")


@pytest.fixture(scope="module")
def nvm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import nvfp4_weight_quantized_moe_b200 as nvm
    return nvm


def _ids_by_definition(logits, bias, topk, score, groups, keep):
    """Group score: the sum of the best two; ties to the lower index (stable sorts)."""
    l = logits.double()
    m, e = l.shape
    if score == "softmax":
        p = (l - l.amax(dim=1, keepdim=True)).exp()
        p = p / p.sum(dim=1, keepdim=True)
    else:
        p = 1.0 / (1.0 + (-l).exp())
    choice = p + bias.double()
    best = choice.view(m, groups, -1).sort(dim=2, descending=True, stable=True).values[:, :, :2].sum(dim=2)
    order = best.sort(dim=1, descending=True, stable=True).indices[:, :keep]
    kept = torch.zeros(m, groups, dtype=torch.bool, device="cuda").scatter_(1, order, True)
    choice = choice.masked_fill(~kept.repeat_interleave(e // groups, dim=1), -INF)
    return choice.sort(dim=1, descending=True, stable=True).indices[:, :topk].to(torch.int32)


def _route(nvm, logits, bias, topk, score, groups, keep):
    m = logits.shape[0]
    ids = torch.empty(m, topk, dtype=torch.int32, device="cuda")
    weights = torch.empty(m, topk, device="cuda")
    nvm.route_topk(logits, ids, weights, score=score, bias=bias, num_groups=groups, topk_groups=keep, group_top=2)
    torch.cuda.synchronize()
    return ids


# Groups of 8, 32, 2 and 32 experts in whole lanes, and groups that are not.
@pytest.mark.parametrize("score,experts,groups,keep", [
    ("softmax", 256, 32, 16), ("softmax", 256, 8, 4), ("sigmoid", 32, 16, 8), ("sigmoid", 256, 8, 4),
    ("softmax", 60, 20, 9), ("sigmoid", 66, 6, 3)])
@pytest.mark.parametrize("size", [2.0, 8.0, 64.0, 256.0])
def test_one_expert_of_each_group_against_the_others(nvm, score, experts, groups, keep, size):
    """100000 rows of near-equal groups: one expert of each at bias +size, the rest at -size."""
    g = torch.Generator(device="cuda").manual_seed(int(size) + experts)
    logits = torch.randn(100000, experts, generator=g, device="cuda") * (1.0 if score == "softmax" else 0.05)
    bias = torch.full((groups, experts // groups), -size, device="cuda")
    bias[:, 1] = size
    bias = bias.flatten()
    got = _route(nvm, logits, bias, 8, score, groups, keep)
    want = _ids_by_definition(logits, bias, 8, score, groups, keep)
    assert int((got != want).any(dim=1).sum()) == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_sizes_that_differ_between_the_groups(nvm, score):
    """Some groups' scores are sums of large values, their neighbours' of small ones: the
    error that counts is not the one of the group at the border."""
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.randn(100000, 128, generator=g, device="cuda") * 0.02
    bias = torch.zeros(16, 8, device="cuda")
    bias[:, 2:] = -500.0
    bias[::2, 0], bias[::2, 1] = 200.0, -200.0
    bias = bias.flatten()
    got = _route(nvm, logits, bias, 6, score, 16, 8)
    assert torch.equal(got, _ids_by_definition(logits, bias, 6, score, 16, 8))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_sums_past_the_range_of_fp32(nvm, score):
    """Two biases of the lowest (largest) finite value add up to an infinity in FP32 and to
    a finite score in 64 bits: the first group can be chosen, the second is below one of an
    infinite bias."""
    logits = torch.zeros(3, 8, device="cuda")
    logits[1] = torch.arange(8.0)
    logits[2] = -torch.arange(8.0)
    for values, keep in (([LOWEST] * 8, 2), ([LOWEST] * 6 + [0.0, -1.0], 3), ([LARGEST] * 4 + [INF, 0.0, 1.0, 1.0], 1),
                         ([LARGEST, LARGEST, INF, LOWEST, 1.0, 1.0, LARGEST, 0.0], 2)):
        bias = torch.tensor(values, device="cuda")
        got = _route(nvm, logits, bias, 2, score, 4, keep)
        assert torch.equal(got, _ids_by_definition(logits, bias, 2, score, 4, keep)), values
