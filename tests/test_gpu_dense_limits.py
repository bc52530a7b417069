"""The dense operators where fp32 ends: finite rows whose squares do not add up in it."""
import pytest
import torch

from nvfp4_block_scaled_gather_gb300 import _native as N
from nvfp4_block_scaled_gather_gb300 import dense as D
from tests.test_gpu_dense import norm_holds, normal

pytestmark = pytest.mark.gpu


# rows of each of the norm's kernels
ROWS = [(5, 3, 64), (4, 1, 256), (3, 1, 512), (700, 1, 512), (700, 1, 1024), (160, 1, 8208), (155, 1, 14096)]


def kinds_of_gate(t, h, d, seed):
    return {"none": None, "channel": 1 + normal((1, 1, d), "bf16", seed).abs(), "element": 1 + normal((t, h, d), "bf16", seed).abs(),
            "token": 1 + normal((t, h, 1), "bf16", seed).abs()}


@pytest.mark.parametrize("t,h,d", ROWS)
@pytest.mark.parametrize("gate", ["none", "channel", "element", "token"])
def test_a_block_whose_squares_do_not_add_up_adds_nothing(cuda, t, h, d, gate):
    """Its norm is 0, and stays 0 behind weights and gates whose product with its values is past fp32 (3.4e38): y is x, and
    the norm after it x's own."""
    x = normal((t, h, d), "bf16", d)
    b = torch.where(normal((t, h, d), "bf16", d + 1) > 0, 2e38, -1.5e38).bfloat16()
    b[:, :, d // 2:] = 0.0
    kw = dict(gate=kinds_of_gate(t, h, d, d + 2)[gate], pre_weight=normal((d,), "fp32", d + 3))
    y, n, want = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    rows, want_rows = (D.Fp8Rows.empty(t, d) if h == 1 else None for _ in range(2))
    D.moe_residual_norm(x, normed=want, quantized=want_rows, pre_weight=kw["pre_weight"])
    D.moe_residual_norm(x, b, y=y, normed=n, quantized=rows, post_norm=True, post_weight=2 + normal((d,), "fp32", d + 4).abs(),
                        residual_scale=0.5, **kw)
    assert torch.equal(y, x) and torch.equal(n, want)
    if h == 1:
        assert torch.equal(rows.codes.view(torch.uint8), want_rows.codes.view(torch.uint8)) and torch.equal(rows.scales, want_rows.scales)
    assert N.check_status() == 0


@pytest.mark.parametrize("t,h,d", ROWS)
@pytest.mark.parametrize("gate", ["none", "channel", "element", "token"])
def test_a_norms_weights_are_upon_the_norm(cuda, t, h, d, gate):
    """Values of about 1e16 (squares' sum below 2e36) with weights of about 1e23: their product is past fp32, the norm's with
    the weights is not."""
    x, b = normal((t, h, d), "bf16", d), normal((t, h, d), "bf16", d + 1, 1e16)
    kw = dict(gate=kinds_of_gate(t, h, d, d + 2)[gate], post_norm=True, post_weight=normal((d,), "fp32", d + 3, 1e23), residual_scale=0.37,
              eps=1e-6)
    y = torch.empty_like(x)
    D.moe_residual_norm(x, b, y=y, **kw)
    norm_holds(x, b, kw, "bf16", y, None)
    assert N.check_status() == 0
