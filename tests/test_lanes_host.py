"""The built kernels' machine code, read for one mistake of the compiler that no result shows reliably.

Where lanes part and meet again (`s_and_saveexec`, a branch past the part when no lane takes it, `s_or exec` at the join, or at an `else`
`s_andn2_saveexec`), nothing may be done for all lanes before the join has brought them back.  With more live registers than a wave has, the register
allocator has put its copies there all the same: in a kernel of 32 rows of 192 elements, copies of lanes' load offsets to
accumulation registers stood before the `s_or exec` behind the loads of the queries, so the lanes of rows that a tile does not
have kept what the registers held before, and their later loads went anywhere."""
from __future__ import annotations

import os
import re
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from _util import ensure_lib

mnb = ensure_lib()
OBJDUMP = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-objdump")


def early(lines):
    """(joins, [(kernel, label, instructions)]) of a listing with labels: vector instructions that stand at a join, or an else, before
    its lanes are set.  (Lanes of scalars kept in a vector register may be read and written whatever the mask is.)"""
    found, joins, kernel, saved, targets = [], 0, None, None, {}
    lines = [s for s in (l.split("//")[0].split(";")[0].strip() for l in lines) if s]
    for i, s in enumerate(lines):
        m = re.search(r"(?:<)?(_Z\w+|\w+)(?:>)?:$", s)
        label = m.group(1) if m else None
        if label and not re.match(r"L(?:BB)?\d", label):
            kernel, saved, targets = label, None, {}
        m = re.match(r"s_\w*saveexec_b64 (\S+),", s)
        if m:
            saved = m.group(1)
        m = re.match(r"s_cbranch_execz \.?(L\w+)", s)
        if m and saved:
            targets.setdefault(m.group(1), set()).add(saved)
        if not label or label not in targets:
            continue
        before = []
        for t in lines[i + 1:i + 400]:
            op = t.split()[0]
            m = re.match(r"s_or_b64 exec, exec, (\S+)|s_(?:or|andn2|xor)_saveexec_b64 [^,]+, (\S+)", t)
            if m:
                if (m.group(1) or m.group(2)) in targets[label]:
                    joins += 1
                    if before:
                        found.append((kernel, label, before))
                break
            if t.endswith(":") or op.startswith(("s_cbranch", "s_branch", "s_endpgm")) or "exec" in t:
                break
            if re.match(r"(v|ds|global|buffer|scratch|flat)_", op) and not re.match(r"v_(readlane|writelane|readfirstlane|nop)", op):
                before.append(t)
    return joins, found


def test_the_reader():
    """It finds what it looks for, and nothing in the same code put right."""
    head = ["0000 <_Zkernel>:", "\ts_and_saveexec_b64 s[8:9], s[14:15]  // 00: 00", "\ts_cbranch_execz L9  // 04: 00", "\tglobal_load_dword v1, v[2:3], off", "",
            "0008 <L9>:"]
    back, copy, scalar = "\ts_or_b64 exec, exec, s[8:9]", "\tv_accvgpr_write_b32 a140, v89", "\tv_writelane_b32 v255, s66, 51"
    assert early(head + [scalar, copy, back]) == (1, [("_Zkernel", "L9", [copy.strip()])])
    assert early(head + [scalar, back, copy]) == (1, [])
    assert early(head + [copy, "\ts_or_b64 exec, exec, s[6:7]"]) == (0, [])          # another join's lanes
    assert early(head + [copy, "\ts_andn2_saveexec_b64 s[4:5], s[8:9]"])[1] == [("_Zkernel", "L9", [copy.strip()])]


@pytest.mark.skipif(not os.path.exists(OBJDUMP) and not shutil.which("llvm-objdump"), reason="no disassembler")
def test_no_vector_instruction_before_the_lanes_are_back(tmp_path):
    tool = OBJDUMP if os.path.exists(OBJDUMP) else shutil.which("llvm-objdump")
    here = shutil.copy(os.path.join(os.path.dirname(mnb.__file__), "libmnb.so"), tmp_path / "lib.so")
    subprocess.run([tool, "--offloading", str(here)], cwd=tmp_path, check=True, capture_output=True)
    objects = sorted(p for p in os.listdir(tmp_path) if "gfx950" in p)
    assert len(objects) >= 10

    def read(name):
        r = subprocess.run([tool, "-d", "--symbolize-operands", "--no-show-raw-insn", name], cwd=tmp_path, check=True, capture_output=True, text=True)
        joins, found = early(r.stdout.splitlines())
        return joins, [(name, *f) for f in found], re.findall(r"<(_Z\w+rows_kernel\w+)>:", r.stdout)
    with ThreadPoolExecutor(4) as pool:
        got = list(pool.map(read, objects))
    assert sum(j for j, _, _ in got) > 1000                   # the listing is read as it is written
    assert any(k for _, _, k in got)
    assert [f for _, found, _ in got for f in found] == []
