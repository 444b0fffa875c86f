"""forward_logits with padding tokens (all logits masked) in layers with and without a
shared expert."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_padding_tokens(shared, dtype):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import nvfp4_weight_quantized_moe_b200 as nvm
    from workloads import make_problem
    from workloads.device import upload_inputs, upload_layer
    from workloads.generators import MoEConfig

    m, pads = 13, [2, 12]
    prob = make_problem(MoEConfig("padded_logits", 256, 512, 8, 2, m, "uniform", 99))
    layer = upload_layer(prob, shared=shared)
    x, _, _ = upload_inputs(prob)
    logits = torch.randn(m, 8, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").to(dtype)
    logits[pads] = float("-inf")
    router = nvm.MoERouter(2, scale=1.5)
    weights = torch.full((m,), 0.5, device="cuda")
    weights[pads[0]] = 0.0
    options = dict(shared_weights=weights) if shared else {}
    for workspace in (None, layer.workspace(m)):
        bufs = layer.forward_logits(x, logits, router, workspace=workspace, **options)
        torch.cuda.synchronize()
        assert bool((bufs.routed_ids[pads] == -1).all()) and bool((bufs.routed_weights[pads] == 0).all())
        # The routing by hand gives the same rows, and the padding tokens' are what their
        # weights say.
        want = layer.forward(x, bufs.routed_ids[:m].clone(), bufs.routed_weights[:m].clone(), workspace=workspace,
                             **options)
        torch.cuda.synchronize()
        assert torch.equal(bufs.out[:m], want.out[:m])
        size = bufs.out[:m].abs().amax(dim=1)
        assert float(size[pads[0]]) == 0.0 and (float(size[pads[1]]) > 0.0) == shared
        assert bool((size[[t for t in range(m) if t not in pads]] > 0).all())
