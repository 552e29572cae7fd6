"""CPU: sizes at the edge of what the training and adapter entry points take.
The host answers all of them; nothing is launched."""
import ctypes
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p(4096)  # aligned, never dereferenced
OK, EINVAL, EWORKSPACE = 0, 1, 3


@pytest.fixture(scope="module")
def lib():
    from routed_expert_ffn_gate_amd import moelb as M
    if not os.path.exists(M.LIB_PATH):
        pytest.fail("libmoelb.so is not built (run python -m routed_expert_ffn_gate_amd.build)")
    return M.lib()


def test_ffn_backward_size_of_refused_shapes_is_zero():
    """A size query answers 0 for shapes that the call refuses, whatever they are (2 * inter past 2^31 made a tile
    count of 0 and divided by it, which ends the process: asked in a process of its own)."""
    code = """
from routed_expert_ffn_gate_amd import moelb as M
f = M.moelb_grouped_ffn_backward_workspace_bytes
top = 2 ** 31 - 1
for rows, groups, E, d, inter in ((8, 1, 1, 8, top), (8, 1, 1, 8, 2 ** 31 - 120), (8, 1, 1, top, 8), (8, 1, 1, top, top),
                                  (8, 1, 1, (1 << 19) + 8, 8), (8, 1, 1, 8, (1 << 19) + 8), (8, 1, 257, 8, 8),
                                  (8, 32769, 1, 8, 8), (8, 1, top, 8, 8)):
    for dtype in (0, 1):
        assert f(rows, groups, E, d, inter, dtype) == 0, (rows, groups, E, d, inter, dtype)
assert f(8, 1, 1, 1 << 19, 8, 1) > 0 and f(8, 1, 1, 8, 1 << 19, 1) > 0 and f(8, 32768, 256, 8, 8, 1) > 0
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])
