"""forward_logits on tensors of another device than the current one: routing and forward
are launched with that device current, so on the same stream.  Fakes; no GPU."""

from types import SimpleNamespace

import pytest
import torch


@pytest.fixture(scope="module")
def nvm():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import nvfp4_weight_quantized_moe_b200 as nvm
    return nvm


def test_routing_and_forward_run_on_the_tensors_device(nvm, monkeypatch):
    current, calls = [torch.device("cuda:0")], []

    class device:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            current.append(self.dev)

        def __exit__(self, *_):
            current.pop()

    monkeypatch.setattr(torch.cuda, "device", device)
    layer = object.__new__(nvm.NVFP4MoE)
    layer.num_experts, layer.topk = 8, 2
    layer.forward = lambda *a, **k: calls.append(("forward", current[-1]))
    router = SimpleNamespace(topk=2, route=lambda *a, **k: calls.append(("route", current[-1])))
    there = torch.device("cuda:1")
    x, logits = SimpleNamespace(shape=(4, 16), device=there), SimpleNamespace(shape=(4, 8), device=there)
    bufs = SimpleNamespace(num_tokens=4, routed_ids=[0] * 4, routed_weights=[0] * 4)
    layer.forward_logits(x, logits, router, bufs)
    assert calls == [("route", there), ("forward", there)] and current == [torch.device("cuda:0")]
