"""Outputs that a call allocates belong to the stream it runs on: nothing that another stream still has to do to their
memory's earlier or later owner reaches them, nor they it."""
import pytest
import torch

from compensated_bit_reproducible_gb300 import api
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu
DELAY = 200_000_000   # clocks: about 0.1 s


def calls():
    d = dev()
    g = torch.Generator(device=d).manual_seed(3)
    x = torch.randn(70, 520, device=d, generator=g)
    h, w = x.bfloat16(), torch.randn(300, 520, device=d, generator=g).bfloat16()
    ids = torch.randint(-1, 300, (70,), device=d, generator=g)
    ones = torch.ones(70, device=d)
    _, mean, rstd = api.stable_layer_norm(x)
    _, lse = api.stable_linear_xent(h, w, ids)
    state = api.state_new(torch.float32)
    api.state_deposit(state, x.view(-1))
    return {
        "embedding": lambda s: api.repro_embedding(w, ids, stream=s),
        "embedding_grad": lambda s: api.repro_embedding_grad(h, ids, 300, stream=s),
        "layer_norm": lambda s: api.stable_layer_norm(x, stream=s),
        "layer_norm_grad": lambda s: api.stable_layer_norm_grad(x, x, None, mean, rstd, stream=s),
        "xent": lambda s: api.stable_linear_xent(h, w, ids, stream=s),
        "xent_grad": lambda s: api.stable_linear_xent_grad(ones, h, w, ids, lse, stream=s),
        "cumsum": lambda s: api.repro_cumsum(x.view(-1), stream=s),
        "cumsum_from_state": lambda s: api.repro_cumsum_from_state(x.view(-1), state, stream=s),
        "segsum": lambda s: api.repro_segsum(x, stream=s),
        "var": lambda s: api.stable_var(x, stream=s),
        "twoterm_var": lambda s: api.twoterm_var(x, stream=s),
        "compare": lambda s: api.compare_sum(x.view(-1), "pairwise", stream=s),
        "finalize": lambda s: api.state_finalize(state, torch.float32, stream=s),
    }


NAMES = ["embedding", "embedding_grad", "layer_norm", "layer_norm_grad", "xent", "xent_grad", "cumsum",
         "cumsum_from_state", "segsum", "var", "twoterm_var", "compare", "finalize"]


def outputs(y):
    return list(y) if isinstance(y, tuple) else [y]


@pytest.mark.parametrize("name", NAMES)
def test_pending_writes_of_the_current_stream_do_not_reach_an_output(name):
    call = calls()[name]
    want = outputs(call(None))
    side = torch.cuda.Stream()
    call(side)
    torch.cuda.synchronize()
    for y in want:
        for _ in range(3):
            # free memory of this stream with work still to do on it
            freed = [torch.empty_like(y) for _ in range(8)]
            torch.cuda._sleep(DELAY // 10)
            for t in freed:
                t.fill_(1)
            del freed, t
            got = outputs(call(side))
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
            del got


@pytest.mark.parametrize("name", NAMES)
def test_an_output_dropped_while_it_is_pending_is_not_handed_out(name):
    call = calls()[name]
    side = torch.cuda.Stream()
    like = [torch.empty_like(y) for y in outputs(call(side))]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(DELAY)
    call(side)
    mine = [torch.full_like(y, 5) for y in like for _ in range(8)]
    torch.cuda.synchronize()
    assert all(torch.all(t == 5) for t in mine)


def test_an_output_used_on_the_current_stream_is_not_overwritten_by_the_next_call():
    d = dev()
    side, x = torch.cuda.Stream(), torch.randn(70, 520, device=d)
    side.wait_stream(torch.cuda.current_stream())
    y = api.stable_layer_norm(x, stream=side)[0]
    torch.cuda.synchronize()
    want = y.clone()
    torch.cuda._sleep(DELAY)
    kept = y.clone()             # still to come when y is dropped
    del y
    other = torch.zeros_like(x)
    for _ in range(4):
        api.stable_layer_norm(other, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(kept, want)
