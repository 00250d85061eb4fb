"""When the torch extension module is needed (no GPU): the calls that go through ctypes work without it, the others
say what is missing, and one built against another torch is not loaded but built again."""

import os
import subprocess
import sys

import pytest
import torch

from speculative_decoding_04_b200 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_package_imports_without_the_extension_module():
    code = """
import sys, torch
torch.__version__ = "0.0.1+none"      # a torch that no extension module was built against
from speculative_decoding_04_b200 import dspark as D
assert D.lib.dspark_workspace_size(D.WS_DRAFT, 2, 3, 100, 8) > 0      # a call of the ctypes part
for f in (D.token_logprobs, lambda a, b: D.quantize_q8(a)):
    try:
        f(torch.zeros(2, 5), torch.zeros(2, dtype=torch.int32))
    except ImportError as e:
        assert "speculative_decoding_04_b200.build" in str(e), e
    else:
        sys.exit("no ImportError")
print("ok")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_an_extension_module_of_another_torch_is_not_up_to_date(monkeypatch):
    build.build()
    assert not build.needs_binding()
    here = build.binding_path()
    monkeypatch.setattr(torch, "__version__", "0.0.1+none")
    assert build.needs_binding() and build.binding_path() != here


def test_the_calls_of_the_extension_module_are_those_of_the_library():
    from speculative_decoding_04_b200 import dspark as D

    for name in ("token_logprobs", "token_logprobs_backward", "rmsnorm_q8", "quantize_q8", "matmul_q8"):
        assert callable(getattr(D._binding, name)) and f"dspark_{name}" in D.declared_functions()
    with pytest.raises(AttributeError):
        D._binding.nothing_of_that_name
