"""The loss where its exact value is small beside the logits, and logits of any size."""
import numpy as np
import pytest
import torch

from compensated_bit_reproducible_gb300 import api
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu
HALVES = [torch.float16, torch.bfloat16]


def one_dominant(x, vocab, dtype):
    """Rows whose logits are x (the label's) and zeros."""
    d = dev()
    h = torch.zeros(len(x), 8, dtype=dtype, device=d)
    h[:, 0] = torch.from_numpy(x).to(d).to(dtype)
    w = torch.zeros(vocab, 8, dtype=dtype, device=d)
    w[0, 0] = 1.0
    return h, w, torch.zeros(len(x), dtype=torch.int64, device=d), h[:, 0].double().cpu().numpy()


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("vocab", [1, 3, 1000, 5003])
def test_loss_of_confident_rows(dtype, vocab):
    """The label's logit is the largest, so the loss is the log of a sum of at least 1.  The sum's error: an
    exponential's 2^-22 and its argument's rounding, x 2^-24 times 1.45, for all but the label's, which is exactly 1;
    a rounding of 2^-24 of the total for each addition to it that is not too small to change it (64 columns of a
    thread on the label's side, 4 in the tile, the pieces); then the logarithm's two steps."""
    h, w, t, x = one_dominant(np.arange(0, 2000) / 16.0, vocab, dtype)
    loss, lse = (v.double().cpu().numpy() for v in api.stable_linear_xent(h, w, t))
    rest = (vocab - 1) * np.exp(-x)
    want = np.log1p(rest)
    adds = np.where(rest < 2.0 ** -26, 0, min(vocab - 1, 80 + vocab // 64))
    bound = rest * (2.0 ** -22 + (x + 1) * 2.0 ** -23) + adds * 2.0 ** -24 * (1 + rest) / (1 + rest) + want * 2.0 ** -22
    assert np.all(loss >= 0.0)
    assert np.all(np.abs(loss - want) <= bound + 2.0 ** -26)
    assert np.all(np.abs(lse - (x + want)) <= bound + 2.0 ** -24 * (x + want) + 2.0 ** -26)


@pytest.mark.parametrize("dtype", HALVES)
def test_vocabulary_of_one(dtype):
    d = dev()
    g = torch.Generator(device=d).manual_seed(0)
    h = (torch.randn(300, 64, device=d, generator=g) * 20).to(dtype)
    w = torch.randn(1, 64, device=d, generator=g).to(dtype)
    loss, _ = api.stable_linear_xent(h, w, torch.zeros(300, dtype=torch.int64, device=d))
    assert not loss.any()


def large_logits(size):
    """Logits of one float32 product each, up to `size`; a row's largest is a quarter or more above the others."""
    d = dev()
    root = float(torch.tensor(size ** 0.5).bfloat16())
    h = torch.zeros(3, 8, dtype=torch.bfloat16, device=d)
    h[:, 0] = torch.tensor([root, -root, 0.5 * root])
    w = torch.zeros(300, 8, dtype=torch.bfloat16, device=d)
    w[:, 1] = 1.0
    w[:, 0] = (torch.tensor([1.0, 0.75, -1.0, 0.0, 0.5] + [0.25] * 295) * root).to(torch.bfloat16)
    return h, w, torch.tensor([0, 1, 4], device=d)


SIZES = [1e4, 1e7, 3e9, 1e15, 1e30, 1e38]


@pytest.mark.parametrize("size", SIZES)
def test_loss_of_logits_of_any_size(size):
    """The softmax picks the largest: lse is that logit and the loss a difference of two, in float32."""
    h, w, t = large_logits(size)
    loss, lse = api.stable_linear_xent(h, w, t)
    z = h.double() @ w.double().T
    top = z.max(1).values
    assert torch.all((lse.double() - top).abs() <= 2.0 ** -22 * top.abs())
    want = top - z.gather(1, t[:, None])[:, 0]
    assert torch.all((loss.double() - want).abs() <= 2.0 ** -22 * (want.abs() + top.abs()) * (want != 0))


@pytest.mark.parametrize("size", SIZES)
def test_gradient_of_logits_of_any_size(size):
    """One more rounding to 16 bits than the output's own, of terms that do not cancel."""
    h, w, t = large_logits(size)
    lse = api.stable_linear_xent(h, w, t)[1]
    dh, dw = api.stable_linear_xent_grad(torch.ones(3, device=h.device), h, w, t, lse)
    z = h.double() @ w.double().T
    g = torch.softmax(z, 1)
    g[torch.arange(3), t] -= 1.0
    for got, exact in ((dh, g @ w.double()), (dw, g.T @ h.double())):
        assert torch.all((got.double() - exact).abs() <= 2.0 ** -7 * exact.abs() + 2.0 ** -12)
