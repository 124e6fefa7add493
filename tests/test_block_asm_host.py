"""The built GEMM kernels keep the distance between scalar registers written by vector instructions and the vector memory
instructions that read them.

A vector memory instruction must not read a scalar register in the 5 wait states after a VALU instruction wrote it. The
compiler inserts those states for its own instructions but does not look into the asm blocks that copy and store in the
pipelined GEMM; a resource that it spilled and brings back with v_readlane right before such a block reads wrong, and the copy or
store goes astray. The library's own gfx950 code, as built here, is read back with the ROCm disassembler."""

import os
import re
import shutil
import subprocess

import pytest

import mx_bit_quantized_amd as mxq

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
WAIT_STATES = 5


def scalar_regs(operand):
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    if m:
        return set(range(int(m.group(1)), int(m.group(2)) + 1))
    m = re.fullmatch(r"s(\d+)", operand)
    return {int(m.group(1))} if m else set()


def short_distances(listing):
    """(function, memory instruction, writer) of every read that comes too early in straight-line code."""
    found, function, recent = [], None, []
    for line in listing.splitlines():
        m = re.match(r"^[0-9a-f]+ <(\S+)>:", line)
        if m:
            function, recent = m.group(1), []
            continue
        text = line.split("//")[0].strip()
        if not line.startswith("\t") or not text:
            continue
        op, _, rest = text.partition(" ")
        args = [a.split()[0] for a in rest.split(",") if a.strip()]
        if op.startswith(("buffer_", "global_", "scratch_", "flat_")):
            need, states = set().union(*(scalar_regs(a) for a in args)), 0
            for width, writer, written in reversed(recent[-2 * WAIT_STATES:]):
                if states >= WAIT_STATES:
                    break
                if written & need:
                    found.append((function, text, writer))
                    break
                states += width
        written = scalar_regs(args[0]) if op.startswith(("v_readlane", "v_readfirstlane", "v_cmp")) and args else set()
        recent.append((int(rest) + 1 if op == "s_nop" else 1, text, written))
    return found


def test_scan_finds_a_short_distance():
    text = "0000 <f>:\n\tv_readlane_b32 s7, v1, 3\n\ts_nop {}\n\tbuffer_store_dword v0, v1, s[4:7], 0 offen\n"
    assert short_distances(text.format(3)) and not short_distances(text.format(4))
    assert not short_distances(text.format(0).replace("s[4:7]", "s[8:11]"))


def test_built_kernels_keep_the_distance(tmp_path):
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump in this image")
    lib = shutil.copy(mxq.LIB_PATH, tmp_path / "libmxq.so")
    subprocess.run([OBJDUMP, "--offloading", lib], cwd=tmp_path, check=True, stdout=subprocess.DEVNULL)
    objects = [f for f in os.listdir(tmp_path) if f.endswith("gfx950")]
    assert objects, "no gfx950 code in the library"
    functions = 0
    for name in objects:
        out = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", name], cwd=tmp_path, check=True, stdout=subprocess.PIPE,
                             text=True).stdout
        functions += out.count(">:")
        assert not short_distances(out), short_distances(out)[:3]
    assert functions > 50
