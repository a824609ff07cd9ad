"""Calls of an empty batch through the binding (no GPU needed: nothing is
launched): without tokens the expert-major arrays may be None, with packed and
with fixed regions."""
import pytest

import combine_lds_atomic_amd as moe


@pytest.mark.parametrize("region_rows", [0, 1, 50])
def test_products_without_tokens(region_rows):
    sh = moe.shape(2, 0, 256, 4, 2, region_rows)
    moe.moe_grouped_gemm(sh, None, None, None, None, None, 256, 128, None)
    moe.moe_grouped_gemm_swiglu(sh, None, None, None, None, None, 256, 128, None, None)
    moe.moe_ffn_up(sh, None, None, None, 256, 128, None, None, None)
    moe.moe_grouped_gemm_bf16(sh, None, None, None, 256, 64, False, None)
    moe.moe_ffn_up_grad(sh, None, None, None, None, None, 256, 128, None, None)
    with pytest.raises(moe.MoeError, match="MOE_EINVAL"):      # a bad size is still refused
        moe.moe_ffn_up(sh, None, None, None, 200, 128, None, None, None)


def test_arrays_are_asked_for_with_tokens():
    sh = moe.shape(2, 8, 256, 4, 2, 50)
    with pytest.raises(TypeError, match="x must be a tensor"):
        moe.moe_ffn_up(sh, None, None, None, 256, 128, None, None, None)
    with pytest.raises(TypeError, match="dw must be a tensor"):
        moe.moe_grouped_wgrad(sh, None, None, None, 64, 128, None)
