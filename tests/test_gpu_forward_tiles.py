"""The grouped product's tile kernels on the GPU against the float64 oracle:
single-row tiles, long K, every epilogue, rows by index and in place, more pair
capacity than pairs, offsets out of order.

The shapes go by the launch's rule, the workgroups that a call is expected to
have; error bounds are those of test_gpu_forward.py."""
import pytest
import torch

from oracle import forward_oracle as O
from pruned_expert_backward_amd import lrmoe as L

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from tests.test_gpu_forward import (  # noqa: E402
    ACTS, BF16, DEV, F32, HALF, U, check_linear, gen, linear_inputs, normal)

# name: (segments, columns of y without SwiGLU).  Each holds one-row segments.
TILES = {
    "few rows": ([0, 1, 3, 20, 21], 136),
    "32x256": ([0, 1, 2] + list(range(10, 508, 8)) + [510, 512], 776),
    "32x64": ([0, 1, 120, 121, 300], 1032),
    "64x64": ([0, 1, 600, 601, 1200], 1032),
    "64x128": ([0, 1, 1250, 1251, 2500], 1032),
    # whole 256-row tiles, ends of each class, one row
    "256 rows": ([0, 1500, 1501, 1700, 4200], 2056),
}


def inputs(tile, name, dt, d_in, seed, index, spare=0):
    seg, F = TILES[tile]
    F = F // 16 * 8 if name == "swiglu" else F   # as many rows of W
    return (seg,) + linear_inputs(seg, d_in, 2 * F if name == "swiglu" else F, dt, seed,
                                  spare=spare, index=index, name=name)


@pytest.mark.parametrize("tile", list(TILES))
@pytest.mark.parametrize("name,d_in", [("none", 8), ("swiglu", 776)])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_one_row_tiles_in_place(tile, name, d_in, dt):
    """A tile of one row without a row index reads one row of x: the loads
    ahead of the products go on past the end of K, behind that row."""
    seg, x, W, _, bias, res = inputs(tile, name, dt, d_in, 101, index=False)
    check_linear(seg, x, W, None, bias, res, name, True)
