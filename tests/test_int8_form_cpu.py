"""The query for the int8 product's kernel: its refusals, and that it names a kernel that
exists (without a device it answers for 148 SMs)."""

import pytest

OK, EINVAL, ESHAPE = 0, 1, 2


@pytest.fixture(scope="module")
def B():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import nvfp4_weight_quantized_moe_b200._binding as binding
    return binding


@pytest.mark.parametrize("sizes", [(0, 64, 64), (4, 0, 64), (4, 64, 0), (4, 64, 24), (4, 64, 131072),
                                   (0x7fffff01, 64, 64), (4, 0x7fffff01, 64)])
def test_refuses_what_the_product_refuses(B, sizes):
    form = (B.c_u32 * 4)()
    assert B._lib.nvfp4_moe_int8_form(*sizes, form) == ESHAPE
    with pytest.raises(B.NVFP4MoEError):
        B.int8_form(*sizes)


def test_refuses_no_place_to_write_and_sizes_out_of_range(B):
    assert B._lib.nvfp4_moe_int8_form(4, 64, 64, None) == EINVAL
    for sizes in ((-1, 64, 64), (4, 1 << 32, 64)):
        with pytest.raises(ValueError):
            B.int8_form(*sizes)


@pytest.mark.parametrize("sizes", [(1, 1, 16), (1, 4096, 2048), (32, 5120, 4096), (256, 2048, 7168), (1000, 4099, 2048),
                                   (8192, 8192, 4096), (0x7fffff00, 1, 16), (1, 0x7fffff00, 131056)])
def test_names_a_kernel(B, sizes):
    form = B.int8_form(*sizes)
    assert (form["channels"], form["tokens"]) in ((16, 8), (16, 16), (64, 128), (128, 128), (256, 256))
    assert form["split"] in ((1, 2, 4, 8) if form["channels"] == 64 else (1, 4) if form["channels"] == 128 else (1,))
    assert form["split"] <= (sizes[2] + 127) // 128
