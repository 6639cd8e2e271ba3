"""The package, with its build script, imports where torch is not installed
or has no GPU support: torch is loaded by the calls that take tensors."""

import os
import subprocess
import sys

import pytest
import torch

import newton_schulz_matrix_amd as nsmi
from newton_schulz_matrix_amd import operators as ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _python(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)


def test_import_and_build_script_without_torch():
    r = _python("import sys; sys.modules['torch'] = None\n"
                "import newton_schulz_matrix_amd as nsmi, newton_schulz_matrix_amd.build as b\n"
                "print(b.SOURCES != [], callable(nsmi.ns_embedding), nsmi.NS_DT_E4M3)\n")
    assert r.returncode == 0 and r.stdout.split() == ["True", "True", "3"], r.stderr


def test_import_does_not_load_torch():
    r = _python("import sys, newton_schulz_matrix_amd\nprint('torch' in sys.modules)\n")
    assert r.stdout.strip() == "False", r.stderr


@pytest.mark.skipif(not os.path.exists(nsmi.LIB_PATH), reason="libnsmi.so not built")
def test_library_loads_without_torch():
    r = _python("import sys; sys.modules['torch'] = None\n"
                "import newton_schulz_matrix_amd as nsmi\n"
                "print(nsmi.status_string(0), nsmi.ns_rms_norm_grad_workspace_size(5, 64) > 0)\n")
    assert r.returncode == 0 and r.stdout.split()[-1] == "True", r.stderr


def test_import_with_a_torch_that_has_no_stream_getter():
    r = _python("import torch\n"
                "if hasattr(torch._C, '_cuda_getCurrentRawStream'):\n"
                "    del torch._C._cuda_getCurrentRawStream\n"
                "import newton_schulz_matrix_amd as nsmi\n"
                "assert nsmi.ns_adamw_step([], [], [], [], 1, 0.1) is None\n")
    assert r.returncode == 0, r.stderr


def test_the_stream_without_the_getter(monkeypatch):
    class Stream:
        cuda_stream = 1234

    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", None, raising=False)
    monkeypatch.setattr(ops, "_raw_stream", None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream)
    assert ops._stream_of(0) == 1234
