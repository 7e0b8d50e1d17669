"""The package loads where torch has no GPU support; the streams are asked for at a call."""
import os
import subprocess
import sys

import pytest

pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import torch
for name in [n for n in vars(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
import quantized_routed_expert_gemv_amd as qm
assert qm.mx_row_bytes("mxfp6", 64) == 48 and qm.plane_bytes("mxfp4", 16, 32, False) == 256
try:
    qm.mx_quantize(torch.zeros(4, 64))
except ValueError as e:
    assert "device" in str(e)
else:
    raise SystemExit("host tensors were taken")
"""


def test_import_and_sizes():
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr
