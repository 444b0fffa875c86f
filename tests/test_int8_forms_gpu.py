"""The int8 product's kernels, bit for bit: exact integer sums, then the header's FP32
steps, whichever kernel takes the sizes."""

import math
import random

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


# (channels, tokens, split, deep) of every kernel and cluster size that a product can take.
VARIANTS = [(16, 8, 1, False), (16, 8, 1, True), (16, 16, 1, False), (16, 16, 1, True),
            (64, 128, 1, False), (64, 128, 1, True), (64, 128, 2, True), (64, 128, 4, False), (64, 128, 4, True),
            (64, 128, 8, False), (64, 128, 8, True), (128, 128, 1, False), (128, 128, 1, True),
            (128, 128, 4, False), (128, 128, 4, True), (256, 256, 1, True)]


@pytest.fixture(scope="module")
def shapes(nvm):
    """Up to three shapes for each variant that the choice takes on this device, small ones
    first, from sizes spread over their logarithms."""
    rng = random.Random(5)
    size = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    found = {}
    for _ in range(150000):
        shape = (size(1, 8192), size(1, 8192), 16 * size(1, 512))
        if math.prod(shape) < 5e10:
            found.setdefault(tuple(nvm.int8_form(*shape).values()), []).append(shape)
    return {v: sorted(s, key=math.prod)[:: max(1, len(s) // 3)][:3] for v, s in found.items()}


def test_the_choice_takes_every_variant_and_no_other(shapes):
    assert set(shapes) == set(VARIANTS)


@pytest.mark.parametrize("variant", VARIANTS)
def test_every_variant_gives_the_same_steps(nvm, shapes, variant):
    for m, n, k in shapes[variant]:
        x, xs, w, ws, bias = _problem(m, n, k)
        want = _steps(x, xs, w, ws) + bias
        for dtype in (F32, BF16):
            store = torch.full((m, n + 13), -7.0, dtype=dtype, device="cuda")
            for out in (store[:, :n].clone(), store[:, 5:5 + n]):
                nvm.int8_matmul(x, xs, w, ws, out, bias=bias)
                assert torch.equal(out, want.to(dtype)), (m, n, k)
            assert bool((store[:, :5] == -7.0).all()) and bool((store[:, 5 + n:] == -7.0).all())
    assert nvm.device_error() == 0
