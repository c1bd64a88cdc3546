"""Each call as the first one of its process, inside a stream capture."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import sys, torch
import weight_only_quantized_mlx_b200 as mq
name = sys.argv[1]
d = dict(device="cuda")
torch.manual_seed(1)
def mx4(rows, cols):
    return mq.mx4_view(torch.randint(-2**31, 2**31 - 1, (rows, cols // 8), dtype=torch.int32, **d),
                       torch.randint(115, 123, (rows, cols // 32), dtype=torch.uint8, **d))
def q8(rows, cols):
    keep.append((torch.randint(-2**31, 2**31 - 1, (rows, cols // 4), dtype=torch.int32, **d),
                 torch.full((rows, cols // 64), 2.0 ** -12, dtype=torch.bfloat16, **d),
                 torch.full((rows, cols // 64), -2.0 ** -5, dtype=torch.bfloat16, **d)))
    return mq.weight_view(*keep[-1], 64)
keep = []
m, n, k, e = (20 if name == "gemm_rows" else 200 if name == "gemm8" else 3), 512, 1024, 4
x = torch.randn(m, k, **d).bfloat16()
y = torch.zeros(m, k if "moe" in name else n, dtype=torch.bfloat16, **d)
w, a = mx4(n, k), mx4(m, k)
router = torch.randn(e, k, **d).bfloat16()
weights = [f(r, c) for r, c in ((e * n, k), (e * n, k), (e * k, n)) for f in [q8 if name == "moe8" else mx4]]
w8 = q8(n, k)
ws = torch.empty(1 << 20, dtype=torch.uint8, **d)
out = torch.zeros(n, k, dtype=torch.bfloat16, **d)
calls = {
    "quantize": lambda s: mq.mlxq_mx4_quantize(x, a, s), "dequant": lambda s: mq.mlxq_mx4_dequant(w, out, s),
    "gemm": lambda s: mq.mlxq_mx4_gemm(w, x, y, m, s), "gemm_rows": lambda s: mq.mlxq_mx4_gemm(w, x, y, m, s),
    "matmul": lambda s: mq.mlxq_mx4_matmul(w, a, y, s),
    "moe8": lambda s: mq.mlxq_moe(router, *weights, e, 2, x, y, m, ws, s),
    "moe4": lambda s: mq.mlxq_mx4_moe(router, *weights, e, 2, x, y, m, ws, s),
    "gemm8": lambda s: mq.mlxq_gemm(w8, x, y, m, s),
}
results = {"quantize": lambda: a.tensors[0], "dequant": lambda: out}
s = torch.cuda.Stream()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=s):
    calls[name](s)
graph.replay()
torch.cuda.synchronize()
first = results.get(name, lambda: y)().clone()
results.get(name, lambda: y)().zero_()
calls[name](None)
torch.cuda.synchronize()
assert first.any() and torch.equal(first, results.get(name, lambda: y)())
mq.mlxq_device_status()
print("captured")
"""


@pytest.mark.parametrize("name", ["quantize", "dequant", "gemm", "gemm_rows", "matmul", "moe8", "moe4", "gemm8"])
def test_first_call_of_a_process_can_be_captured(name):
    r = subprocess.run([sys.executable, "-c", PROGRAM, name], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout + r.stderr
