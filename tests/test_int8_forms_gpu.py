"""The int8 product's kernels, bit for bit: exact integer sums, then the header's FP32
steps, whichever kernel takes the sizes."""

import pytest
import torch

from test_layer_ops_gpu import FORMS

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def nvm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import nvfp4_weight_quantized_moe_b200 as nvm
    return nvm


def _problem(m, n, k):
    g = torch.Generator(device="cuda").manual_seed(m + 3 * n + 7 * k)
    x = torch.randint(-128, 128, (m, k), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-128, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    xs = torch.rand(m, generator=g, device="cuda") + 0.01
    ws = torch.rand(n, generator=g, device="cuda") * 1e-3
    # As large as the products, so that its addition rounds.
    bias = torch.randn(n, generator=g, device="cuda") * 3.0 * k ** 0.5
    return x, xs, w, ws, bias


def _steps(x, xs, w, ws):
    """The sum in FP32 (64 bits hold it exactly before), and two rounded products."""
    return ((x.double() @ w.double().T).float() * xs[:, None]) * ws


@pytest.mark.parametrize("m,n,k", FORMS)
def test_every_kernel_gives_the_same_steps(nvm, m, n, k):
    x, xs, w, ws, bias = _problem(m, n, k)
    want = _steps(x, xs, w, ws)
    for dtype in (F32, BF16):
        for b in (None, bias):
            out = torch.empty(m, n, dtype=dtype, device="cuda")
            nvm.int8_matmul(x, xs, w, ws, out, bias=b)
            assert torch.equal(out, (want if b is None else want + b).to(dtype))
    assert nvm.device_error() == 0


def test_a_row_has_the_same_bits_in_any_batch(nvm):
    x, xs, w, ws, bias = _problem(700, 1536, 1040)
    whole = torch.empty(700, 1536, device="cuda")
    nvm.int8_matmul(x, xs, w, ws, whole, bias=bias)
    for m in (1, 7, 33, 129, 300):
        part = torch.empty(m, 1536, device="cuda")
        nvm.int8_matmul(x[:m], xs[:m], w, ws, part, bias=bias)
        assert torch.equal(part, whole[:m])
