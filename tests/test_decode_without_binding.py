"""The operators of a decoding step without the native torch module: the C calls work, the torch calls say what to build."""
from __future__ import annotations

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
assert mnb.mnb_decode_version() == 100 and mnb.mnb_kv_page_bytes(2, 64, 16) == 2 * 16 * 68
cache, x = mnb.kv_cache(3, 2, 64, page_size=16, device="cpu"), torch.zeros(1, 2, 64, dtype=torch.float16)
pages, lengths = torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
assert mnb.rope_table(4, 32, device="cpu").shape == (4, 32)
for call in (lambda: mnb.kv_append(x, x, x, cache, pages, lengths), lambda: mnb.kv_read(cache, pages, lengths),
             lambda: mnb.kv_attention(x, cache, pages, lengths), lambda: mnb.sample(x[0], torch.zeros(2))):
    try:
        call()
    except ImportError as e:
        assert "build.py" in str(e) and "of_another_torch" in str(e), e
    else:
        raise AssertionError("no error")
print("fine")
"""


def test_decoding_without_the_native_module():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr
