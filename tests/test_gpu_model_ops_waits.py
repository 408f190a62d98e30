"""The bounded waits of the layer norm's and the loss's kernels, made to run out: the call ends, the context stays
usable, the next call says so.  Each in a process of its own, as the mark stays for the process."""
import os
import subprocess
import sys

import pytest

from tests.gpu_util import dev

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import os, sys, time
import torch
from compensated_bit_reproducible_gb300 import api
g = torch.Generator(device="cuda").manual_seed(0)
x = torch.randn({rows}, {cols}, device="cuda", generator=g).{kind}()
w = torch.randn(900, {cols}, device="cuda", generator=g).{kind}()
ids = torch.randint(0, 900, ({rows},), device="cuda", generator=g)
ones = torch.ones({rows}, device="cuda")
_, mean, rstd = api.stable_layer_norm(x)
if x.dtype != torch.float32:
    _, lse = api.stable_linear_xent(x, w, ids)
calls = {{
    "layer_norm": lambda: api.stable_layer_norm(x),
    "layer_norm_grad": lambda: api.stable_layer_norm_grad(x, x, None, mean, rstd),
    "xent": lambda: api.stable_linear_xent(x, w, ids),
    "xent_grad": lambda: api.stable_linear_xent_grad(ones, x, w, ids, lse),
}}
table = api.repro_embedding_grad(x, ids, 900)
torch.cuda.synchronize()
os.environ["REPRO_FORCE_WAIT_FAIL"] = "1"
start = time.time()
got = calls["{name}"]()
torch.cuda.synchronize()
assert time.time() - start < 1.5, "the waits ran to their ordinary limit"
if "{name}" == "xent":
    assert got[0].isnan().all() and got[1].isnan().all()
del os.environ["REPRO_FORCE_WAIT_FAIL"]
for name, call in calls.items():
    if x.dtype == torch.float32 and name.startswith("xent"):
        continue
    try:
        call()
        raise SystemExit(name + " did not report the wait that ran out")
    except api.ReproError as e:
        assert e.status == 6, e
# the device and the calls that do not wait are as before
assert torch.equal(api.repro_embedding_grad(x, ids, 900), table)
assert torch.equal(x.float().sum().isfinite(), torch.tensor(True, device="cuda"))
torch.cuda.synchronize()
print("done")
"""


@pytest.mark.parametrize("name,rows,cols,kind", [
    ("layer_norm", 3000, 512, "bfloat16"), ("layer_norm", 3000, 513, "half"), ("layer_norm", 700, 9001, "float"),
    ("layer_norm_grad", 3000, 512, "bfloat16"), ("layer_norm_grad", 3000, 513, "half"), ("layer_norm_grad", 700, 4100, "float"),
    ("xent", 600, 512, "bfloat16"), ("xent", 5, 64, "half"), ("xent_grad", 600, 512, "half"), ("xent_grad", 600, 77, "bfloat16")])
def test_a_wait_that_runs_out(name, rows, cols, kind):
    dev()
    r = subprocess.run([sys.executable, "-c", SCRIPT.format(name=name, rows=rows, cols=cols, kind=kind)], cwd=ROOT,
                       capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "done" in r.stdout, r.stdout + r.stderr
