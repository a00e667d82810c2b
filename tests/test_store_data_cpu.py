"""The device code of the built library: what gfx950 needs around wide stores, which
the compiler leaves out for one form of them."""
import os
import re
import shutil
import subprocess

import pytest

from weight_gradient_gemm_amd import _lib

OBJDUMP = shutil.which("llvm-objdump") or "/opt/rocm/llvm/bin/llvm-objdump"


def device_code(folder):
    """The lines of every gfx950 code object in libforge.so, disassembled."""
    copy = shutil.copy(_lib.library_path, folder)
    subprocess.run([OBJDUMP, "--offloading", os.path.basename(copy)], cwd=folder, check=True,
                   capture_output=True)
    for name in sorted(os.listdir(folder)):
        if "gfx950" in name:
            r = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", name], cwd=folder, check=True,
                               capture_output=True, text=True)
            yield from r.stdout.splitlines()


def registers(operand):
    m = re.match(r"v\[(\d+):(\d+)\]$", operand) or re.match(r"v(\d+)()$", operand)
    return set(range(int(m[1]), int(m[2] or m[1]) + 1)) if m else set()


def overwritten(lines):
    """(kernel, store, next instruction) of every buffer store of 12 or 16 bytes a lane with a
    scalar register as its offset whose data the next instruction writes."""
    kernel, store, found = "", None, []
    for line in lines:
        head = re.match(r"[0-9a-f]+ <(\w+)>:", line)
        if head:
            kernel, store = head[1], None
            continue
        code = line.split("//")[0].strip()
        if not code:
            continue
        name, _, rest = code.partition(" ")
        operands = [x.strip() for x in rest.split(",")]
        if store and name.startswith("v_") and registers(operands[0]) & registers(store[1]):
            found.append((kernel, store[0], code))
        store = None
        if re.match(r"buffer_store_dwordx[34]$", name) and re.match(r"s\d+\b|m0\b", operands[3]):
            store = (code, operands[0])
    return found


def test_the_scan_sees_it():
    text = """
0000000000001000 <a_kernel>:
	buffer_store_dwordx4 v[66:69], v227, s[44:47], s65 offen nt// 000000010B40: E07E1000
	v_sub_f32_e32 v66, v214, v71                               // 000000010B48: 04848FD6
	buffer_store_dwordx4 v[66:69], v227, s[44:47], 0 offen nt  // the compiler keeps these apart
	v_sub_f32_e32 v66, v214, v71
	buffer_store_dwordx4 v[66:69], v227, s[44:47], s66 offen nt
	s_nop 0
	v_sub_f32_e32 v66, v214, v71
	buffer_store_dwordx3 v[2:4], v227, s[44:47], s66 offen
	v_mov_b32_e32 v4, v214
	buffer_store_dwordx2 v[2:3], v227, s[44:47], s66 offen
	v_mov_b32_e32 v3, v214
"""
    assert [f[1:] for f in overwritten(text.splitlines())] == [
        ("buffer_store_dwordx4 v[66:69], v227, s[44:47], s65 offen nt", "v_sub_f32_e32 v66, v214, v71"),
        ("buffer_store_dwordx3 v[2:4], v227, s[44:47], s66 offen", "v_mov_b32_e32 v4, v214")]


def test_no_store_has_its_data_overwritten(tmp_path):
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    lines = list(device_code(str(tmp_path)))
    assert sum("buffer_store_dwordx4" in x for x in lines) > 100
    found = overwritten(lines)
    assert not found, (len(found), found[:5])
