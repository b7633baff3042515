"""Calls on a machine without a GPU return an error that names them, in a process that
goes on."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# (the child has no device, and makes sure of it: the pointers are none)
CALLS = r"""
import ctypes, struct, sys
import bit_vq_routed_gb300 as bv
import torch
assert not torch.cuda.is_available()
lib, P = bv.load(), ctypes.c_void_p(4096)
call = {"moe_linear_8bit": lambda T: lib.moe_linear_8bit(P, 64, P, P, 64, P, None, None, 0, P, 32, T, 32, 64, 0, 0, P, 256, None),
        "moe_linear": lambda T: lib.moe_linear(P, 64, P, 64, None, None, 0, P, 32, T, 32, 64, 0, 0, P, 256, None),
        "moe_rms_norm": lambda T: lib.moe_rms_norm(P, 64, 0, None, 0, None, 0, None, 1e-6, P, 64, None, 0, None, T, 64, 0, None),
        "moe_quantize_rows": lambda T: lib.moe_quantize_rows(P, 64, 0, P, 64, P, T, 64, None),
        "moe_route_scored": lambda T: lib.moe_route_scored(P, T, 16, 2, struct.pack("@iifP3i4x", 1, 1, 1.0, 0, 1, 1, 1), P, P, None)
        }[sys.argv[1]]
for T in (1, 16, 40, 300):
    print(call(T), lib.moe_last_error().decode(), flush=True)
"""


@pytest.mark.parametrize("name", ["moe_linear", "moe_linear_8bit", "moe_rms_norm", "moe_quantize_rows", "moe_route_scored"])
def test_error(name):
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="", PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", CALLS, name], capture_output=True, text=True, env=env)
    assert r.returncode == 0, r.stdout + r.stderr[-2000:]
    lines = r.stdout.splitlines()
    assert len(lines) == 4
    for line in lines:
        status, message = line.split(" ", 1)
        assert int(status) < 0 and message.startswith(name + ":"), line
