"""The binding on a torch built without CUDA, whose private accessors are absent."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import types
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
torch.cuda.current_device = lambda: 3
torch.cuda.current_stream = lambda i: types.SimpleNamespace(cuda_stream=100 + i)
from block_quantized_weight_qgemm_b200 import qgemm
assert qgemm._current_device() == 3 and qgemm._raw_stream(2) == 102
try:
    qgemm.moe_combine(torch.zeros(2, 8), torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1))
except AssertionError as e:
    assert "CUDA device" in str(e)
else:
    raise SystemExit("host tensors were taken")
print("imported")
"""


def test_import_and_refusal_without_the_private_accessors():
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "imported", r.stderr
