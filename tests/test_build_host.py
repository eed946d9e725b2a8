"""The host module belongs to the PyTorch that it was built against."""
import os
import subprocess
import sys

from dora_adapter_linear_gb300 import _lib as L
from dora_adapter_linear_gb300 import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(B.__file__)))
OTHER = """
import torch
torch.__version__ = torch.torch_version.TorchVersion("9.9.9+other")
from dora_adapter_linear_gb300 import _lib, build
assert build._stale(build.sources()), "the other PyTorch's module counts as built"
try:
    _lib.host()
except ImportError as e:
    print("refused:", e)
"""


def test_another_pytorch_neither_takes_the_module_for_built_nor_loads_it():
    B.build()
    assert not B._stale(B.sources()) and L.host()
    done = subprocess.run([sys.executable, "-c", OTHER], cwd=ROOT, capture_output=True, text=True)
    assert done.returncode == 0, done.stderr
    assert "refused:" in done.stdout
