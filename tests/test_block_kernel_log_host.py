"""What MXQ_LOG says of a block operator's kernel is what the call launches (no GPU needed: the line is written before the launch,
which fails in a process that is given no device)."""

import json
import os
import subprocess
import sys

import pytest

from conftest import ROOT

CALL = """
import ctypes, json, sys
import mx_bit_quantized_amd as mxq
from mx_bit_quantized_amd import block
c = json.loads(sys.argv[1])
P = 0x10000  # never read: there is no device
st = block._lib().mxq_gemm_residual(c["mode"], P, P, P, P, None, 0, P, P if c["gate"] else None, c["type"], c["ld"], c["rpg"], P,
                                    c["m"], c["n"], c["k"], None)
assert st == mxq.ERR_HIP, st
print(mxq.block_kernel_name(c["mode"], c["m"], c["n"], c["k"]))
"""


def logged(**change):
    """(kernel in the log line, kernel of the query) of a residual product's call."""
    c = dict(mode=0, gate=True, type=0, m=4096, n=4096, k=4096, rpg=1000)
    c.update(change)
    c.setdefault("ld", c["n"])
    env = dict(os.environ, MXQ_LOG="1", HIP_VISIBLE_DEVICES="-1", CUDA_VISIBLE_DEVICES="-1", ROCR_VISIBLE_DEVICES="-1", PYTHONPATH=ROOT)
    env.pop("MXQ_BLOCK_KERNEL", None)
    env.pop("MXQ_CHECK_FINITE", None)
    r = subprocess.run([sys.executable, "-c", CALL, json.dumps(c)], env=env, cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
    line = [x for x in r.stderr.splitlines() if x.startswith("[mxq] gemm_residual")]
    assert len(line) == 1, r.stderr[-2000:]
    return line[0].rsplit("kernel=", 1)[1].strip(), r.stdout.strip()


@pytest.mark.parametrize("mode, suffix", [(0, "w4a4"), (1, "w4a8")])
def test_log_names_the_kernel_of_the_call(mode, suffix):
    pipe, tokens = f"pipe_{suffix}", f"tokens_{suffix}"
    assert logged(mode=mode, gate=False) == (pipe, pipe)
    assert logged(mode=mode, ld=4096 + 8) == (pipe, pipe)
    # several groups, rows of the table no multiple of 8 apart: not the pipelined kernel's, whatever the query (which
    # knows of no gate) says of the shape
    assert logged(mode=mode, ld=4096 + 4) == (tokens, pipe)
    assert logged(mode=mode, ld=4096 + 1, type=1) == (tokens, pipe)
    # one vector for all rows: its stride is not read
    assert logged(mode=mode, ld=4096 + 4, rpg=0) == (pipe, pipe)
    assert logged(mode=mode, m=1, rpg=0) == (tokens, tokens)
