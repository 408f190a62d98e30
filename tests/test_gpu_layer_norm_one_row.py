"""The layer norm gradient of a single row too long for a block's shared memory: dweight and dbias are sums of one
term, whatever the workspace held before."""
import pytest
import torch

from compensated_bit_reproducible_gb300 import api
from tests.gpu_util import dev
from tests.model_ref import DTYPES, EPS, TINY

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols,offset", [(40001, 0), (40000, 1)])
def test_sums_of_one_term(dtype, cols, offset):
    d = dev()
    g = torch.Generator(device=d).manual_seed(cols)

    def rows(n, scale):
        t = torch.empty(n * cols + offset, dtype=dtype, device=d)[offset:].view(n, cols)
        t.copy_(torch.randn(n, cols, device=d, generator=g) * scale)
        return t

    # five rows make two blocks' partial rows, of the size that one row's call asks for: the pool hands them out again
    x, dy = rows(5, 1.0), rows(5, 1000.0)
    _, mean, rstd = api.stable_layer_norm(x)
    api.stable_layer_norm_grad(dy, x, None, mean, rstd)
    x, dy = rows(1, 1.0), rows(1, 1.0)
    _, mean, rstd = api.stable_layer_norm(x)
    _, dweight, dbias = api.stable_layer_norm_grad(dy, x, None, mean, rstd)
    assert torch.equal(dbias, dy[0])
    # x - mean, times rstd, times dy: three roundings of float32, one of the type
    want = dy[0].double() * ((x[0].double() - mean.double()) * rstd.double())
    size = dy[0].double().abs() * (x[0].double().abs() + mean.double().abs()) * rstd.double()
    assert torch.all((dweight.double() - want).abs() <= 4 * 2.0 ** -24 * size + EPS[dtype] * want.abs() * 1.001 + TINY[dtype])
