"""The model operators in CUDA graphs."""
import os
import subprocess
import sys

import pytest
import torch

from compensated_bit_reproducible_gb300 import api
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("n,vocab,cols", [(40, 300, 520), (1500, 700, 257)])
def test_replay_sees_new_inputs(n, vocab, cols):
    """A step of all six calls (up to 1024 positions and more; aligned rows and rows that are copied) captured once and
    replayed over new values: the bits of the calls made directly."""
    d = dev()
    g = torch.Generator(device=d).manual_seed(n)
    weight = torch.empty(vocab, cols, dtype=torch.bfloat16, device=d)
    gain, bias = torch.empty(cols, dtype=torch.bfloat16, device=d), torch.empty(cols, dtype=torch.bfloat16, device=d)
    ids, labels = torch.empty(n, dtype=torch.int64, device=d), torch.empty(n, dtype=torch.int64, device=d)
    dloss = torch.empty(n, device=d)

    def new():
        weight.normal_(generator=g).mul_(0.2)
        gain.normal_(1.0, 0.1, generator=g)
        bias.normal_(generator=g)
        ids.random_(-1, vocab, generator=g)
        labels.random_(-1, vocab, generator=g)
        dloss.uniform_(generator=g)

    def step():
        x = api.repro_embedding(weight, ids, scale=3.0)
        h, mean, rstd = api.stable_layer_norm(x, gain, bias)
        loss, lse = api.stable_linear_xent(h, weight, labels)
        dh, dw = api.stable_linear_xent_grad(dloss, h, weight, labels, lse)
        dx, dgain, dbias = api.stable_layer_norm_grad(dh, x, gain, mean, rstd)
        return x, h, mean, rstd, loss, lse, dh, dw, dx, dgain, dbias, api.repro_embedding_grad(dx, ids, vocab, scale=3.0)

    side = torch.cuda.Stream()
    new()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = step()
    for _ in range(3):
        new()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


FIRST_CALL_IN_A_CAPTURE = """
import torch
from compensated_bit_reproducible_gb300 import api
x = torch.randn(70, 520, device="cuda")
side = torch.cuda.Stream()
api.repro_cumsum(x.view(-1), stream=side)       # the environment is checked, the stream's page is there
torch.cuda.synchronize()
refused = False
try:
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        try:
            y = api.stable_layer_norm(x)
        except api.ReproError:
            refused = True
except RuntimeError:
    refused = True
print("refused", refused)
torch.cuda.synchronize()
y, mean, rstd = api.stable_layer_norm(x)
assert torch.allclose(mean, x.mean(1), atol=1e-5)
print("done")
"""


def test_a_first_call_inside_a_capture_does_not_spoil_later_ones():
    dev()
    r = subprocess.run([sys.executable, "-c", FIRST_CALL_IN_A_CAPTURE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "done" in r.stdout, r.stdout + r.stderr
