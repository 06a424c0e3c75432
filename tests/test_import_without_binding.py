"""The package without its native torch module (another Python or torch, or a build without their headers): the
product it had before and the C calls work as they did, the torch calls of the operators say what to build."""
from __future__ import annotations

import importlib.util
import os
import subprocess
import sys

import pytest

from _util import ROOT, ensure_lib

ensure_lib()
pytest.importorskip("torch")

PROGRAM = """
import sys
class Block:
    def find_spec(self, name, path=None, target=None):
        if name.endswith("._mnb_ops"):
            raise ImportError("undefined symbol: of_another_torch")
sys.meta_path.insert(0, Block())
import blockwise_bit_quantized_amd as mnb
import torch
assert mnb.mnb_version() == 104 and mnb.mnb_packed_sizes(64, 64, 4, 32, False)[0] == 0
assert mnb.mnb_ops_version() == 100 and mnb.mnb_mx_packed_sizes(64, 64)[0] == 0
x = torch.zeros(4, 64, dtype=torch.float16)
q = mnb.mx_tensor(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8), mnb.MNB_MX_FP8)
w = mnb.MxWeight(torch.zeros(4096, dtype=torch.uint8), torch.zeros(1024, dtype=torch.uint8), 64, 64)
for call in (lambda: mnb.mx_quantize(x), lambda: mnb.mx_dequantize(q), lambda: mnb.mx_matmul(q, w),
             lambda: mnb.rmsnorm(x, x[0]), lambda: mnb.logprobs(x)):
    try:
        call()
    except ImportError as e:
        assert "build.py" in str(e) and "of_another_torch" in str(e), e
    else:
        raise AssertionError("no error")
print("fine")
"""


def test_import_without_the_native_module():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr


def _build_module():
    spec = importlib.util.spec_from_file_location("_mnb_build_test", os.path.join(ROOT, "blockwise_bit_quantized_amd", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_build_without_a_compiler_or_headers_for_the_module(tmp_path, monkeypatch, capsys):
    """The library alone is built then; a module of an earlier build does not stay beside it."""
    b = _build_module()
    for missing in ("compiler", "headers"):
        stale = tmp_path / "_mnb_ops.so"
        stale.write_bytes(b"stale")
        with monkeypatch.context() as m:
            m.setattr(b, "BINDING_LIB", str(stale))
            if missing == "compiler":
                m.setenv("PATH", str(tmp_path))
            else:
                m.setattr(b.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
            b._build_binding(False)
        assert not stale.exists() and "_mnb_ops" in capsys.readouterr().err
