"""The loss and its gradient over vocabularies of a thousand column tiles and more."""
import numpy as np
import pytest
import torch

from compensated_bit_reproducible_gb300 import api
from tests.test_gpu_linear_xent import check_grad, check_loss, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,vocab,cols", [(1, 261889, 16), (3, 262144, 16), (40, 262144, 8), (5, 262145, 24), (2, 300007, 16),
                                          (2, 524288, 8)])
def test_loss_and_gradient(dtype, n, vocab, cols):
    h, w, labels, t = inputs(n, vocab, cols, dtype, n + cols)
    labels[-1] = vocab - 1
    t[-1] = vocab - 1
    got = api.stable_linear_xent(h, w, t)
    check_loss(h, w, labels, got)
    dloss = torch.from_numpy(np.random.default_rng(n).uniform(-1, 1, n).astype(np.float32)).to(h.device)
    check_grad(dloss, h, w, labels, api.stable_linear_xent_grad(dloss, h, w, t, got[1]), dtype)


def test_gradient_of_512_rows():
    """The most rows whose piece of the vocabulary still has 262,144 columns; a second piece of 37."""
    h, w, labels, t = inputs(512, 262181, 8, torch.bfloat16, 7)
    got = api.stable_linear_xent(h, w, t)
    dloss = torch.ones(512, device=h.device)
    dh, dw = api.stable_linear_xent_grad(dloss, h, w, t, got[1])
    z = h.float() @ w.float().T    # eight exact products: float32 is enough here
    # (a sum of 128 terms in a thread, 2049 tiles' after one another in strands of 8: 2^-23 each, on logits below 32)
    assert torch.all((got[1] - torch.logsumexp(z, 1)).abs() <= 2.0 ** -23 * (128 + 2049 / 4 + 32 * 8))
    p = torch.softmax(z, 1)
    has = (t >= 0).nonzero()[:, 0]
    p[has, t[has]] -= 1.0
    p[t < 0] = 0.0
    for a, want in ((dh, p @ w.float()), (dw, p.T @ h.float())):
        # two roundings to bfloat16 of terms of both signs
        assert (a.float() - want).norm() <= 2 * 2.0 ** -8 * want.norm()
