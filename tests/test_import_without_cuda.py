"""The bindings import on a torch without CUDA (whose C module lacks the CUDA functions), as their CPU users need."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
from linear_rnn_b200 import ops
x = torch.empty(2, 3, 5, 8)
print(ops.gla_scan_saved_bytes(ops.make_scan_problem(x)))
"""


def test_ops_imports_without_torchs_cuda_functions():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.split()[-1] == str(4 * 2 * 3 * 8)
