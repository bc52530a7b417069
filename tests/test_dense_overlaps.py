"""Outputs of the residual step over its inputs, without a GPU: rows that are read after they were written are refused on the
host."""
import pytest

from nvfp4_block_scaled_gather_gb300 import dense as D
from tests.test_dense_abi import INVALID, norm_args

NONE = (0, 0, 0)


@pytest.mark.parametrize("part", ["x", "block"])
@pytest.mark.parametrize("output", ["y", "normed"])
@pytest.mark.parametrize("heads,strides", [(1, (0, 0)), (1, (512, 0)), (4, (1024, 0)), (4, (0, 256)), (4, (2048, 256)), (4, (256, 1024))])
def test_an_output_over_an_input_of_other_strides(native, part, output, heads, strides):
    """One row held along as x and the stream over it, for instance: the first token's y is the others' x."""
    parts = dict(x=(1 << 20, 1024, 256), block=(2 << 20, 1024, 256), y=(3 << 20, 1024, 256), normed=(4 << 20, 1024, 256))
    if heads == 1:
        parts = {n: (p, 256, 0) for n, (p, _, _) in parts.items()}
    parts[part] = (parts[output][0], *strides)
    assert D.load().moe_residual_norm(norm_args(heads=heads, **parts), None) == INVALID
