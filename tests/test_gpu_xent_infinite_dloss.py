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
