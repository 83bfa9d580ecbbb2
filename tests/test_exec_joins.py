"""Joins of the built kernels' branches, read from the library's own machine code (no GPU needed).

Where a branch on an empty execution mask ends, the mask is restored first.  A register that the compiler saves or copies ahead
of that is written in none of the lanes that come there by the branch: a loop whose mask was saved so never ended."""
import os
import re
import shutil
import subprocess

import pytest

LLVM = "/opt/rocm/llvm/bin"
OBJDUMP = os.path.join(LLVM, "llvm-objdump")
VECTOR = re.compile(r"(v_(?!readlane|writelane|readfirstlane)|scratch_|ds_|global_|buffer_|flat_)")
NARROWS = re.compile(r"s_\w+_saveexec|s_\w+ exec|s_xor_b64 .*, exec, ")
ENDS = re.compile(r"(s_cbranch|s_branch|s_endpgm|s_setpc|s_swappc|s_\w+_saveexec)")


def early(lines):
    """(joins that a branch skips to, [(address, instruction)] of vector instructions ahead of their mask) of one object's
    disassembly."""
    code, targets, labels = [], set(), set()
    base = 0
    for line in lines:
        m = re.match(r"([0-9a-f]+) <.*>:", line)
        if m:
            base = int(m.group(1), 16)
            continue
        m = re.match(r"\s+(\S.*?)\s*// ([0-9A-F]+):", line)
        if not m:
            continue
        code.append((int(m.group(2), 16), m.group(1)))
        to = re.match(r"s_c?branch", m.group(1)) and re.search(r"\+0x([0-9a-f]+)>", line)
        if to:
            labels.add(base + int(to.group(1), 16))
            if m.group(1).startswith("s_cbranch_execz") and NARROWS.match(code[-2][1]):
                targets.add(base + int(to.group(1), 16))
    joins, found = 0, []
    for i, (at, _) in enumerate(code):
        if at not in targets:
            continue
        ahead = []
        for a, text in code[i:]:
            if text.startswith(("s_or_b64 exec, exec", "s_mov_b64 exec")):
                joins += 1
                found += ahead
                break
            if ENDS.match(text) or (a != at and a in labels):
                break
            if VECTOR.match(text):
                ahead.append((a, text))
    return joins, found


LISTING = """0000000000001000 <kernel>:
\ts_and_saveexec_b64 s[0:1], vcc                             // 000000001000: BE80206A
\ts_cbranch_execz 2                                          // 000000001004: BF880002 <kernel+0x10>
\tv_and_b32_e32 v1, v3, v1                                   // 000000001008: 26020303
\tv_and_b32_e32 v0, v2, v0                                   // 00000000100C: 26000102
%s\ts_or_b64 exec, exec, s[0:1]                               // 000000001018: 87FE007E
\ts_endpgm                                                   // 00000000101C: BF810000
"""


def test_the_reading_of_a_join():
    store = "\tscratch_store_dwordx2 off, v[0:1], off offset:88           // 000000001010: DC744058 007F0000\n"
    scalar = "\ts_mov_b32 s2, 0                                            // 000000001010: BE820080\n"
    joins, found = early((LISTING % store).splitlines())
    assert joins == 1 and [a for a, _ in found] == [0x1010]
    assert early((LISTING % scalar).splitlines()) == (1, [])


def test_no_join_saves_registers_before_its_mask(tmp_path):
    import precision_moe_expert_mx_amd as m
    lib = os.path.join(os.path.dirname(m.__file__), "libmxmoe.so")
    if not os.path.exists(OBJDUMP) or not os.path.exists(lib):
        pytest.skip("needs the built library and llvm-objdump")
    shutil.copy(lib, tmp_path / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=tmp_path, check=True, capture_output=True)
    objects = [p for p in tmp_path.iterdir() if p.name.endswith("gfx950") and p.stat().st_size]
    assert len(objects) >= 10
    joins = 0
    for p in objects:
        text = subprocess.run([OBJDUMP, "-d", "--no-leading-headers", str(p)], check=True, capture_output=True, text=True).stdout
        n, found = early(text.splitlines())
        joins += n
        assert not found, (p.name, found[:5])
    assert joins > 5000
