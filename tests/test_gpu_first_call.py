"""The first work of a process is a captured call: nothing of the library has been launched before, so every
kernel that the call needs is loaded at the latest while the stream is being captured."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = '''
import sys
import torch
import inputgen
import sparse_expert_ffn_router_b200 as colibri
from tests import gpu_harness as H

kind, T, d, f = sys.argv[1], *map(int, sys.argv[2:])
B = colibri.COLIBRI_BF16
wl = inputgen.custom("first", T=T, d=d, E=4, k=2, f=f, act=inputgen.BF16, wdt=inputgen.I8 if kind == "i8a8" else inputgen.BF16)
p = inputgen.make_problem(wl, seed=3)
t = H.to_device(p)
q, s = torch.zeros(T, d, dtype=torch.int8, device="cuda"), torch.zeros(T, device="cuda")
w, ws = torch.ones(d, d, dtype=torch.int8, device="cuda"), torch.ones(d, device="cuda")
layer = None if kind == "products" else colibri.MoELayer(d, f, 4, 2, 0, B, colibri.COLIBRI_I8A8 if kind == "i8a8" else B, max_tokens=T)
y = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")


def call(stream):
    if kind == "decode":
        layer.decode(t["x"], t["router_w"], None, t["expert_w"], y, stream=stream)
    elif kind == "products":  # the rows of x, and their products in the kernels for few rows and for more
        colibri.colibri_quantize_rows(t["x"], B, T, d, d, q, d, s, stream)
        for rows in (8, T):
            colibri.colibri_int_gemm(q, d, s, w, d, ws, rows, d, d, y, d, B, stream)
    else:
        layer.forward(t["x"], t["router_w"], None, t["expert_w"], y, t["expert_scales"], stream=stream)


torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    call(torch.cuda.current_stream())
g.replay()
torch.cuda.synchronize()
first = y.clone()
assert torch.isfinite(first).all() and first.abs().max() > 0
y.zero_()
call(None)
torch.cuda.synchronize()
if layer:
    layer.sync_status()
colibri.colibri_int_check()
assert torch.equal(y, first)
print("same")
'''


@pytest.mark.gpu
@pytest.mark.parametrize("kind,T,d,f", [("i8a8", 300, 1088, 2112), ("decode", 5, 256, 320), ("products", 20, 256, 320)])
def test_the_first_call_of_a_process_may_be_captured(kind, T, d, f):
    r = subprocess.run([sys.executable, "-c", SCRIPT, kind, str(T), str(d), str(f)], cwd=ROOT,
                       env=dict(os.environ, CUDA_MODULE_LOADING="LAZY"), capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr
