"""Any negative token is padding, whatever its low 32 bits, and none past the table counts."""
import pytest
import torch

from compensated_bit_reproducible_gb300 import api
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu
LEAST, MOST = -(1 << 63), (1 << 63) - 1


@pytest.mark.parametrize("n", [64, 1024, 1025, 5000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_padding_that_looks_like_a_token(dtype, n):
    """Among the positions of every token k there are -2^32 + k, -2^63 + k and 2^32 + k: the gradient's bits and the
    lookup's rows are those with -1 (2^32 + k: NaN in the lookup) in their places."""
    d = dev()
    g = torch.Generator(device=d).manual_seed(n)
    vocab, cols = 11, 96
    tokens = torch.randint(0, vocab, (n,), device=d, generator=g)
    kind = torch.randint(0, 5, (n,), device=d, generator=g)
    dy = torch.randn(n, cols, device=d, generator=g).to(dtype)
    weight = torch.randn(vocab, cols, device=d, generator=g).to(dtype)
    strange = tokens.clone()
    for k, shift in enumerate((-(1 << 32), LEAST, 1 << 32)):
        strange = torch.where(kind == k, tokens + shift, strange)
    # a warp of padding alone, the smallest and the largest value
    strange[:32], strange[32], strange[33] = LEAST, MOST, -(1 << 32) + vocab
    plain = torch.where((strange < 0) | (strange >= vocab), -1, strange)
    want = api.repro_embedding_grad(dy, plain, vocab)
    got = api.repro_embedding_grad(dy, strange, vocab)
    assert torch.equal(got, want) and got.any()
    rows = api.repro_embedding(weight, strange)
    assert torch.equal(rows[strange < vocab], api.repro_embedding(weight, plain)[strange < vocab])
    assert rows[strange >= vocab].isnan().all()
