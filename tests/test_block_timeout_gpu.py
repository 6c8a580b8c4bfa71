"""The dense layer's bounded waits, run out on the GPU without a hang.

The test build of the library (libpkm_waittest.so: a pipeline wait gives up as soon as one try
does not satisfy it) is loaded in a child process. A forward and a backward through the tensor
cores must return, record the timeout in the workspace's status word and leave the context
usable; a small batch, which waits for nothing, must still be right.
"""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
WAITTEST = os.path.join(ROOT, "product_key_memory_b200", "libpkm_waittest.so")

CHILD = r"""
import sys, torch
sys.path.insert(0, ROOT)
import product_key_memory_b200 as P
assert P.LIB_PATH.endswith("libpkm_waittest.so"), P.LIB_PATH
status = []
for kind in (torch.bfloat16, torch.float32):
    x = torch.randn(2000, 1024, device="cuda").to(kind)
    W = torch.randn(1040, 1024, device="cuda").to(kind)
    ws = P.alloc_linear_workspace(P.make_linear_shape(2000, 1040, 1024, kind, kind, "gelu"), False, "cuda")
    y, pre = P.pkm_linear_forward(x, W, activation="gelu", want_pre=True, workspace=ws)
    status.append(P.pkm_device_status(ws))
    ws = P.alloc_linear_workspace(P.make_linear_shape(2000, 1040, 1024, kind, kind, "gelu"), True, "cuda")
    grads = dict(x=torch.empty_like(x), W=torch.empty(1040, 1024, device="cuda"))
    P.pkm_linear_backward(x, W, torch.ones_like(y), grads, pre=torch.ones_like(y), activation="gelu", workspace=ws)
    status.append(P.pkm_device_status(ws))
x = torch.randn(3, 1024, device="cuda")
W = torch.randn(1040, 1024, device="cuda")
y, _ = P.pkm_linear_forward(x, W)
assert bool(((y.double() - x.double() @ W.double().t()).abs() <= 2.0 ** -23 * 1024 * (x.abs().double() @ W.abs().double().t())).all())
torch.cuda.synchronize()
assert float((torch.ones(1000, device="cuda") * 2).sum().item()) == 2000.0
print("STATUS", *status, flush=True)
""".replace("ROOT", repr(ROOT))


@pytest.mark.skipif(not os.path.exists(WAITTEST), reason="test build not built")
def test_waits_of_the_dense_layer_time_out_and_report():
    env = dict(os.environ, PKM_LIBRARY=WAITTEST)
    r = subprocess.run([sys.executable, "-c", CHILD], env=env, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    line = [ln for ln in r.stdout.splitlines() if ln.startswith("STATUS")][-1]
    assert [int(v) for v in line.split()[1:]] == [-5] * 4, line       # PKM_ERR_DEVICE
