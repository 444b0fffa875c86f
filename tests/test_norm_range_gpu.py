"""RMS norm of rows whose squares pass the FP32 range, and of rows with a NaN or an
infinity: what the header says of out, codes and scale."""

import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
E4M3, INT8 = torch.float8_e4m3fn, torch.int8


@pytest.fixture(scope="module")
def nvm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import nvfp4_weight_quantized_moe_b200 as nvm
    return nvm


def _run(nvm, x, weight, residual, code):
    m, h = x.shape
    out = torch.full((m, h), 7.0, dtype=BF16, device="cuda")
    r_out = None if residual is None else torch.empty(m, h, dtype=residual.dtype, device="cuda")
    q = torch.full((m, h), 7, dtype=torch.uint8, device="cuda").view(code)
    scale = torch.full((m,), 7.0, device="cuda")
    nvm.add_rms_norm(x, weight, 1e-6, out=out, residual=residual, residual_out=r_out, q=q, q_scale=scale)
    torch.cuda.synchronize()
    return out.float(), r_out, q.float(), scale


# Rows of one warp, of a CTA, with single elements at the ends, off 16 bytes, longest.
@pytest.mark.parametrize("h,shift", [(200, 0), (512, 0), (1001, 0), (1001, 1), (4096, 0), (20000, 0), (32768, 0)])
@pytest.mark.parametrize("dtype,rdtype", [(F32, None), (BF16, BF16), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("code", [INT8, E4M3])
def test_squares_past_the_range_give_zeros(nvm, h, shift, dtype, rdtype, code):
    g = torch.Generator(device="cuda").manual_seed(h)
    wide = torch.randn(6, h + shift, generator=g, device="cuda").clamp_(-4, 4)
    x = wide[:, shift:]
    x[1] *= 1e20                       # every square passes
    x[2] *= 2.0 ** 62                  # only their sum does
    x[3, h // 2] = 3e19                # one value alone
    x[4, h - 1] = -3e38
    x = wide.to(dtype)[:, shift:]
    residual = None if rdtype is None else torch.randn(6, h, generator=g, device="cuda").to(rdtype)
    weight = torch.rand(h, generator=g, device="cuda") + 0.1   # r * weight stays in the range
    weight.clamp_(max=1.0)
    out, r_out, q, scale = _run(nvm, x, weight, residual, code)
    for row in (1, 2, 3, 4):
        assert float(out[row].abs().max()) == 0.0 and float(q[row].abs().max()) == 0.0 and float(scale[row]) == 0.0
    for row in (0, 5):
        assert float(out[row].abs().max()) > 0.1 and float(scale[row]) > 0.0
        assert float(q[row].abs().max()) == (127.0 if code == INT8 else 448.0)
    if residual is not None:
        # r in FP32, then the type's rounding, as torch does both.
        assert torch.equal(r_out, (x.float() + residual.float()).to(rdtype))


@pytest.mark.parametrize("h", [64, 300, 4096])
@pytest.mark.parametrize("code", [INT8, E4M3])
def test_rows_with_a_nan_or_an_infinity(nvm, h, code):
    x = torch.ones(3, h, device="cuda")
    x[0, 5] = float("nan")
    x[1, 7] = float("inf")
    out, _, _, scale = _run(nvm, x, torch.ones(h, device="cuda"), None, code)
    assert bool(torch.isnan(out[0]).all()) and bool(torch.isnan(scale[:2]).all())
    elsewhere = torch.arange(h, device="cuda") != 7
    assert bool(torch.isnan(out[1, 7])) and float(out[1, elsewhere].abs().max()) == 0.0
    # 1 / sqrt(1 + 1e-6), within half a step of BF16.
    assert float((out[2] - 1.0).abs().max()) <= 2.0 ** -8
