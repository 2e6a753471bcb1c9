"""Wait states that the hardware asks of the program, looked for in the built
library's own gfx950 code (no GPU needed).

A scalar write of m0 is followed by at least one other instruction before a
load into LDS reads it: the compiler sees to that where it writes both, not
inside an asm statement.
"""
import os
import re
import shutil
import subprocess

import pytest

from int4_routed_expert_logits_amd import _binding as B

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
LDS_LOAD = re.compile(r"^(global_load_lds_|buffer_load_\w+ .*\blds\b)")
WRITES_M0 = re.compile(r"^s_\w+ m0,")


def early_lds_loads(listing):
    """(loads into LDS, those right behind a write of m0) of a disassembly."""
    loads, early, before, where = 0, [], "", ""
    for line in listing:
        if line.endswith(">:"):
            where, before = line.split("<")[-1][:-2], ""
            continue
        text = line.split("//")[0].strip()
        if not text:
            continue
        if LDS_LOAD.match(text):
            loads += 1
            if WRITES_M0.match(before):
                early.append(f"{where}: {before}; {text}")
        before = text
    return loads, early


def test_the_rule_itself():
    """The two orders, as the disassembler prints them."""
    bad = ["0000 <k>:", "\ts_mov_b32 m0, s4   // 00: BE", "\tglobal_load_lds_dwordx4 v[0:1], off  // 04"]
    good = [bad[0], bad[1], "\ts_nop 0  // 04", bad[2]]
    assert early_lds_loads(bad)[1] and early_lds_loads(good) == (1, [])
    assert early_lds_loads(bad[:2] + ["0100 <l>:"] + bad[2:]) == (1, [])


def test_m0_is_written_a_wait_state_before_loads_into_lds(tmp_path):
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    lib = shutil.copy(B.LIB_PATH, tmp_path)
    subprocess.run([OBJDUMP, "--offloading", lib], cwd=tmp_path, check=True, capture_output=True)
    total, early = 0, []
    for name in sorted(os.listdir(tmp_path)):
        if name.endswith("gfx950"):
            out = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", name], cwd=tmp_path,
                                 check=True, capture_output=True, text=True).stdout
            n, bad = early_lds_loads(out.splitlines())
            total, early = total + n, early + bad
    assert total > 100, "the tiled products fetch into LDS"
    assert not early, f"{len(early)} of {total}, the first: {early[0]}"
