"""The library over a stand-in for the CUDA runtime (fake_cudart.cpp): entry points check their arguments and
come to their launches without a GPU."""
import ctypes
import os
import shutil
import subprocess

import pytest

from dora_adapter_linear_gb300 import _lib as L
from dora_adapter_linear_gb300 import build as B


@pytest.fixture(scope="session")
def fake(tmp_path_factory):
    objects = [os.path.join(B.BUILD, os.path.basename(s) + ".o") for s in B.sources()]
    B.build(force=not all(map(os.path.exists, objects)))
    so = str(tmp_path_factory.mktemp("fake") / "fake.so")
    include = os.path.join(os.path.dirname(os.path.dirname(B.nvcc())), "include")
    source = os.path.join(os.path.dirname(os.path.abspath(__file__)), "fake_cudart.cpp")
    # -Bsymbolic: the library's calls go to the stand-in, whatever runtime the process has loaded
    subprocess.run([shutil.which("g++") or "g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-I", include, source, *objects,
                    "-Wl,-Bsymbolic", "-o", so], check=True)
    lib = ctypes.CDLL(so)
    for name, (res, args) in L._SIGS.items():
        getattr(lib, name).restype, getattr(lib, name).argtypes = res, args
    return lib
