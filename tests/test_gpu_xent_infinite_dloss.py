"""A dloss that is infinite or NaN stays in its row of dh."""
import pytest
import torch

from compensated_bit_reproducible_gb300 import api
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_other_rows_keep_their_bits(dtype, value):
    d = dev()
    g = torch.Generator(device=d).manual_seed(1)
    h, w = torch.randn(50, 64, device=d, generator=g).to(dtype), (torch.randn(900, 64, device=d, generator=g) * 0.2).to(dtype)
    t = torch.randint(0, 900, (50,), device=d, generator=g)
    lse = api.stable_linear_xent(h, w, t)[1]
    dloss = (0.5 + torch.rand(50, device=d, generator=g)) * 2.0 ** -20
    dloss[3] = 0.0
    want = api.stable_linear_xent_grad(dloss, h, w, t, lse)[0]
    dloss[3] = value
    got = api.stable_linear_xent_grad(dloss, h, w, t, lse)[0]
    rest = torch.arange(50, device=d) != 3
    assert torch.equal(got[rest], want[rest])
    assert not got[3].isfinite().any()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_a_nan_in_a_row_without_a_label(dtype):
    """Its loss, dh and all other rows are as if it were finite; its column of dweight is NaN (0 times it), as the
    header says."""
    d = dev()
    g = torch.Generator(device=d).manual_seed(2)
    h, w = torch.randn(300, 64, device=d, generator=g).to(dtype), (torch.randn(500, 64, device=d, generator=g) * 0.2).to(dtype)
    t = torch.randint(0, 500, (300,), device=d, generator=g)
    t[7] = -1
    ones = torch.ones(300, device=d)
    loss, lse = api.stable_linear_xent(h, w, t)
    dh, dw = api.stable_linear_xent_grad(ones, h, w, t, lse)
    h[7, 5] = float("nan")
    loss2, lse2 = api.stable_linear_xent(h, w, t)
    dh2, dw2 = api.stable_linear_xent_grad(ones, h, w, t, lse2)
    rest, others = torch.arange(300, device=d) != 7, torch.arange(64, device=d) != 5
    assert torch.equal(loss, loss2) and lse2[7].isnan() and torch.equal(lse[rest], lse2[rest])
    assert torch.equal(dh, dh2) and not dh[7].any()
    assert torch.equal(dw[:, others], dw2[:, others]) and dw2[:, 5].isnan().all()
