"""Inputs and outputs that are column slices of one buffer: the bits of separate buffers laid out the same, and
nothing written beside the output."""
import pytest
import torch

from compensated_bit_reproducible_gb300 import api
from tests.gpu_util import dev
from tests.model_ref import DTYPES

pytestmark = pytest.mark.gpu
HALVES = [torch.float16, torch.bfloat16]


class Slices:
    """Two buffers of [rows, left | gap | cols | right]: the input in the first one's left part, the output in its
    right part, or in the second's."""

    def __init__(self, values, rows, cols, gap, fill=7.0):
        self.n, self.left, d = rows, values.shape[1], dev()
        width = self.left + gap + cols + 5
        self.both = torch.full((max(rows, len(values)), width), fill, dtype=values.dtype, device=d)
        self.both[:len(values), :self.left] = values
        self.alone = torch.full_like(self.both, fill)
        self.at = slice(self.left + gap, self.left + gap + cols)
        self.input = self.both[:len(values), :self.left]
        self.before = self.both.clone()

    def out(self, shared):
        return (self.both if shared else self.alone)[:self.n, self.at]

    def check(self):
        assert torch.equal(self.out(True), self.out(False)) and not torch.all(self.out(True) == 7.0)
        self.before[:self.n, self.at] = self.out(True)
        assert torch.equal(self.both, self.before)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols,gap", [(40, 96, 0), (40, 96, 3), (300, 1001, 0), (7, 33, 1), (3, 20001, 2)])
def test_layer_norm(dtype, rows, cols, gap):
    g = torch.Generator(device=dev()).manual_seed(cols)
    x, dy = (torch.randn(rows, cols, device=dev(), generator=g).to(dtype) for _ in range(2))
    s = Slices(x, rows, cols, gap)
    stats = [api.stable_layer_norm(s.input, out=s.out(shared))[1:] for shared in (False, True)]
    assert torch.equal(stats[0][0], stats[1][0]) and torch.equal(stats[0][1], stats[1][1])
    s.check()
    mean, rstd = stats[0]
    for turn in (0, 1):   # dx beside x, dx beside dy
        s = Slices(dy if turn else x, rows, cols, gap)
        sums = [api.stable_layer_norm_grad(*((s.input, x) if turn else (dy, s.input)), None, mean, rstd, out=s.out(shared))
                for shared in (False, True)]
        assert all(torch.equal(a, b) for a, b in zip(sums[0][1:], sums[1][1:]))
        s.check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,cols,gap", [(50, 96, 0), (50, 33, 1), (1500, 301, 0), (1500, 520, 2)])
def test_embedding(dtype, n, cols, gap):
    vocab = 200
    g = torch.Generator(device=dev()).manual_seed(n)
    ids = torch.randint(-1, vocab, (n,), device=dev(), generator=g)
    s = Slices(torch.randn(vocab, cols, device=dev(), generator=g).to(dtype), n, cols, gap)
    for shared in (False, True):
        api.repro_embedding(s.input, ids, out=s.out(shared))
    s.check()
    s = Slices(torch.randn(n, cols, device=dev(), generator=g).to(dtype), vocab, cols, gap)
    for shared in (False, True):
        api.repro_embedding_grad(s.input, ids, vocab, out=s.out(shared))
    s.check()


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("n,vocab,cols,gap", [(70, 300, 96, 0), (70, 300, 77, 1), (600, 700, 64, 3)])
def test_loss_gradient(dtype, n, vocab, cols, gap):
    g = torch.Generator(device=dev()).manual_seed(n)
    h = Slices(torch.randn(n, cols, device=dev(), generator=g).to(dtype), n, cols, gap)
    w = Slices((torch.randn(vocab, cols, device=dev(), generator=g) * 0.3).to(dtype), vocab, cols, gap)
    ids = torch.randint(-1, vocab, (n,), device=dev(), generator=g)
    lse = api.stable_linear_xent(h.input, w.input, ids)[1]
    for shared in (False, True):
        api.stable_linear_xent_grad(torch.ones(n, device=dev()), h.input, w.input, ids, lse,
                                    out=(h.out(shared), w.out(shared)))
    h.check()
    w.check()
