"""The binding's two ways, through the C++ part and through ctypes, make the same call."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def _calls(nvm):
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    logits, bias = rand(9, 64), rand(64) * 0.1
    ids, weights = torch.empty(9, 4, dtype=torch.int32, device="cuda"), torch.empty(9, 4, device="cuda")
    nvm.route_topk(logits, ids, weights, score="sigmoid", bias=bias, num_groups=4, topk_groups=2, group_top=2,
                   renormalize=False, scale=1.5)
    x, res = rand(9, 256).to(torch.bfloat16), rand(9, 256)
    out, r_out = torch.empty_like(x), torch.empty_like(res)
    q, scale = torch.empty(9, 256, dtype=torch.int8, device="cuda"), torch.empty(9, device="cuda")
    nvm.add_rms_norm(x, rand(256), 1e-5, out=out, residual=res, residual_out=r_out, q=q, q_scale=scale)
    w = torch.randint(-127, 128, (48, 256), generator=g, dtype=torch.int8, device="cuda")
    y = torch.empty(9, 48, device="cuda")
    nvm.int8_matmul(q, scale, w, rand(48).abs(), y, bias=rand(48))
    torch.cuda.synchronize()
    return [ids, weights, out, r_out, q, scale, y]


def test_ctypes_and_the_extension_give_the_same(monkeypatch):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import nvfp4_weight_quantized_moe_b200 as nvm
    assert nvm._binding._quick_call is not None
    quick = _calls(nvm)
    monkeypatch.setattr(nvm._binding, "_quick_call", None)
    for a, b in zip(quick, _calls(nvm)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
