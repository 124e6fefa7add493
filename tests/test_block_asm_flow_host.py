"""The distance between a scalar register's write by a vector instruction and its read by a vector memory instruction, along every path
through a built kernel: a write in front of a branch or at a loop's end counts for the reads behind it.

Each function's instructions form a graph (branches by their target addresses). A forward pass keeps, for each scalar register,
the smallest number of wait states since such a write on any path that leads here, up to the 5 that are needed."""

import os
import re
import shutil
import subprocess

import pytest

import mx_bit_quantized_amd as mxq
from test_block_asm_host import OBJDUMP, WAIT_STATES, scalar_regs

MEMORY = ("buffer_", "global_", "scratch_", "flat_")


def functions(listing):
    """(name, [(address, text, branch target or None)]) of a disassembly."""
    name, base, body = None, 0, []
    for line in listing.splitlines():
        m = re.match(r"^([0-9a-f]+) <(\S+)>:", line)
        if m:
            if body:
                yield name, body
            base, name, body = int(m.group(1), 16), m.group(2), []
            continue
        text, _, comment = line.partition("//")
        if not line.startswith("\t") or not text.strip() or not comment.strip():
            continue
        target = re.search(r"<[^<>+]+(?:\+0x([0-9a-f]+))?>\s*$", comment)
        body.append((int(comment.split(":")[0], 16), text.strip(), base + int(target.group(1) or "0", 16) if target else None))
    if body:
        yield name, body


def early_reads(body):
    """[(memory instruction, wait states)] of reads that come too early on some path, and the opcodes that no path reaches."""
    index = {address: i for i, (address, _, _) in enumerate(body)}
    steps = []
    for i, (_, text, target) in enumerate(body):
        op, _, rest = text.partition(" ")
        args = [a.split()[0] for a in rest.split(",") if a.strip()]
        needs = set().union(*(scalar_regs(a) for a in args)) if op.startswith(MEMORY) else set()
        writes = scalar_regs(args[0]) if op.startswith(("v_readlane", "v_readfirstlane", "v_cmp")) and args else set()
        assert op not in ("s_setpc_b64", "s_swappc_b64"), "a call: the pass would have to follow it"
        after = [] if op in ("s_endpgm", "s_branch") else [i + 1]
        if op == "s_branch" or op.startswith("s_cbranch"):
            after.append(index[target])
        steps.append((needs, writes, int(rest) + 1 if op == "s_nop" else 1, [j for j in after if j < len(body)]))
    state = [None] * len(body)
    state[0], work, found = {}, [0], {}
    while work:
        i = work.pop()
        needs, writes, states, after = steps[i]
        early = [state[i][r] for r in needs if state[i].get(r, WAIT_STATES) < WAIT_STATES]
        if early:
            found[i] = (body[i][1], min(early))
        out = {r: d + states for r, d in state[i].items() if d + states < WAIT_STATES}
        out.update((r, 0) for r in writes)
        for j in after:
            if state[j] is None:
                state[j] = dict(out)
                work.append(j)
                continue
            nearer = {r: d for r, d in out.items() if d < state[j].get(r, WAIT_STATES)}
            if nearer:
                state[j].update(nearer)
                work.append(j)
    return list(found.values()), {text.split()[0] for s, (_, text, _) in zip(state, body) if s is None}


def listing(*lines):
    """A function at address 0 whose instructions are 4 bytes long; '->n' names the branched-to line."""
    out = ["0000 <f>:"]
    for i, text in enumerate(lines):
        text, _, target = text.partition("->")
        out.append(f"\t{text.strip()} // {4 * i:08X}: 0" + (f" <f+0x{4 * int(target):x}>" if target else ""))
    return "\n".join(out) + "\n"


def found(*lines):
    (_, body), = functions(listing(*lines))
    return early_reads(body)[0]


STORE = "buffer_store_dword v0, v1, s[4:7], 0 offen"


@pytest.mark.parametrize("want, lines", [
    (True, ("v_readlane_b32 s7, v1, 3", "s_nop 3", STORE, "s_endpgm")),
    (False, ("v_readlane_b32 s7, v1, 3", "s_nop 4", STORE, "s_endpgm")),
    (False, ("v_readlane_b32 s8, v1, 3", STORE, "s_endpgm")),
    # a write in front of a taken branch
    (True, ("v_readlane_b32 s7, v1, 3", "s_cbranch_scc1 2 ->4", "s_nop 7", "s_endpgm", STORE, "s_endpgm")),
    # the fall-through has waited, the other path has not
    (True, ("v_readfirstlane_b32 s4, v1", "s_cbranch_scc1 1 ->3", "s_nop 7", STORE, "s_endpgm")),
    (False, ("v_readfirstlane_b32 s4, v1", "s_nop 4", "s_cbranch_scc1 1 ->4", "s_nop 7", STORE, "s_endpgm")),
    # a write at the end of a loop, the read at its head
    (True, ("s_nop 0", STORE, "v_readlane_b32 s6, v1, 3", "s_cbranch_scc1 65532 ->1", "s_endpgm")),
    (False, ("s_nop 0", STORE, "v_readlane_b32 s6, v1, 3", "s_nop 4", "s_cbranch_scc1 65531 ->1", "s_endpgm")),
])
def test_pass_follows_branches(want, lines):
    assert bool(found(*lines)) == want


def test_built_kernels_keep_the_distance_on_every_path(tmp_path):
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump in this image")
    lib = shutil.copy(mxq.LIB_PATH, tmp_path / "libmxq.so")
    subprocess.run([OBJDUMP, "--offloading", lib], cwd=tmp_path, check=True, stdout=subprocess.DEVNULL)
    seen = 0
    for name in sorted(f for f in os.listdir(tmp_path) if f.endswith("gfx950")):
        out = subprocess.run([OBJDUMP, "-d", name], cwd=tmp_path, check=True, stdout=subprocess.PIPE, text=True).stdout
        for function, body in functions(out):
            early, unreached = early_reads(body)
            assert not early, (function, early[:3])
            assert not any(op.startswith(MEMORY) for op in unreached), (function, unreached)  # only padding
            seen += 1
    assert seen > 50
