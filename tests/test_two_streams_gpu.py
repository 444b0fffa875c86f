"""Large and small batches at once, on two streams: every kernel with tensor memory beside
every other one, bit for bit as one after another."""

import pytest
import torch

pytestmark = pytest.mark.gpu


class _Work:
    """A forward of `m` tokens and an int8 product of `pm` x `pn` x `pk` behind it."""

    def __init__(self, nvm, layer, m, pm, pn, pk, seed, **options):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.nvm, self.layer, self.options = nvm, layer, options
        self.x = torch.randn(m, layer.hidden, generator=g, device="cuda").to(torch.bfloat16)
        self.logits = torch.randn(m, layer.num_experts, generator=g, device="cuda")
        self.router = nvm.MoERouter(layer.topk)
        self.bufs, self.ws = layer.buffers(m), layer.workspace(m)
        codes = lambda r, c: torch.randint(-127, 128, (r, c), generator=g, device="cuda", dtype=torch.int8)  # noqa: E731
        self.q, self.w = codes(pm, pk), codes(pn, pk)
        self.qs, self.wscale = torch.rand(pm, generator=g, device="cuda"), torch.rand(pn, generator=g, device="cuda")
        self.y = torch.empty(pm, pn, dtype=torch.bfloat16, device="cuda")

    def run(self):
        self.layer.forward_logits(self.x, self.logits, self.router, self.bufs, workspace=self.ws, **self.options)
        self.nvm.int8_matmul(self.q, self.qs, self.w, self.wscale, self.y)

    def outputs(self):
        return [self.bufs.out, self.y]


def test_large_and_small_batches_at_once():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import nvfp4_weight_quantized_moe_b200 as nvm
    from workloads import make_problem
    from workloads.device import upload_layer
    from workloads.generators import MoEConfig

    layer = upload_layer(make_problem(MoEConfig("streams", 1024, 512, 4, 2, 8, "uniform", 5)))
    pairs = [(_Work(nvm, layer, 2048, 2048, 2048, 1024, 1), _Work(nvm, layer, 32, 256, 1024, 4096, 2, path=nvm.PATH_PREFILL)),
             (_Work(nvm, layer, 2048, 300, 2048, 2048, 3), _Work(nvm, layer, 8, 40, 4096, 1024, 4, path=nvm.PATH_PREFILL))]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for pair in pairs:
        want = []
        for w in pair:
            w.run()
            torch.cuda.synchronize()
            want.append([t.clone() for t in w.outputs()])
            for t in w.outputs():
                t.zero_()
        torch.cuda.synchronize()
        for _ in range(20):
            for w, s in zip(pair, streams):
                with torch.cuda.stream(s):
                    for _ in range(1 if w is pair[0] else 4):
                        w.run()
        torch.cuda.synchronize()
        assert nvm.device_error() == 0
        for w, outs in zip(pair, want):
            for t, u in zip(w.outputs(), outs):
                assert torch.equal(t, u) and float(u.float().abs().max()) > 0
