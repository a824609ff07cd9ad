"""The training operators where they went wrong once, or where a rarer form of a
kernel runs: against the plain float64 forms of tests/training_ref.py."""
import pytest
import torch

import combine_lds_atomic_amd as moe

pytestmark = pytest.mark.gpu

from gpu_harness import log  # noqa: E402

BF = torch.bfloat16


@pytest.mark.parametrize("region_rows", [0, 1, 300])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_wgrad_no_tokens(region_rows, dtype):
    """An empty batch has no exp_off to read, with fixed regions either, and what
    the regions hold is nobody's: the weights' gradients are zeros, or what
    they were when added to."""
    log(f"wgrad without tokens, region_rows={region_rows} {dtype}")
    for N, E, F, K in ((1, 1, 16, 16), (2, 4, 64, 128), (4, 32, 272, 400)):
        sh = moe.shape(N, 0, 256, E, 1, region_rows)
        d, x = (torch.full((N * region_rows, n), float("nan"), dtype=BF, device="cuda") for n in (F, K))
        dw = torch.ones((E, F, K), dtype=dtype, device="cuda")
        moe.moe_grouped_wgrad(sh, d, x, None, F, K, dw, add=True)
        assert (dw == 1).all()
        moe.moe_grouped_wgrad(sh, d, x, None, F, K, dw)
        assert (dw == 0).all()


def test_wgrad_no_tokens_no_arrays():
    """The same with no arrays of rows at all."""
    sh = moe.shape(2, 0, 256, 4, 2, 50)
    dw = torch.ones((4, 64, 128), device="cuda")
    moe.moe_grouped_wgrad(sh, None, None, None, 64, 128, dw, add=True)
    assert (dw == 1).all()
    moe.moe_grouped_wgrad(sh, None, None, None, 64, 128, dw)
    assert (dw == 0).all()
