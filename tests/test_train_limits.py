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


def test_gate_backward_refuses_rows_whose_offsets_wrap(lib):
    """bf16: w and h are read 64 memory rows at a time by 32-bit byte offsets, the rows past the last one included
    (they have to lie past the operand's end to read as zeros): 64 rows of 2 d bytes are 2^32 at d = 2^25.  No
    workspace: nothing is launched."""
    def call(d, dt):
        return lib.moelb_gate_backward(P, 4, d, 4, 1, dt, P, P, P, P, None, 0, P, P, P, None)
    row = lambda d, k: k * 2 * d + 2 * (d - 8) + 15  # noqa: E731  last byte of a 16-byte load of row k
    assert row(1 << 25, 63) < 1 << 32 <= row((1 << 25) + 8, 63)
    assert call(1 << 25, 1) == EWORKSPACE
    assert call((1 << 25) + 8, 1) == EINVAL and call(1 << 28, 1) == EINVAL
    assert call((1 << 25) + 8, 0) == EWORKSPACE  # fp32 rows are addressed with 64 bits


def ffn(lib, back, rows, E, d, inter, dt, dx=P, d13=P, d2=P, ws=P):
    """The call with `rows` rows in one group an expert."""
    if back:
        return lib.moelb_grouped_ffn_backward(P, P, max(rows, 1), rows, P, E, E, 1, -1, None, 1, d, inter, dt, P, P, P, ws,
                                              1 << 62, dx, d13, d2, None)
    return lib.moelb_grouped_ffn_train(P, max(rows, 1), rows, P, E, E, 1, -1, None, 1, d, inter, dt, P, P, ws, 1 << 62, P,
                                       P, None)


def test_ffn_refuses_launches_of_2_32_threads(lib):
    """fp32, 256 experts, the widest layers: 64 x 16 tiles of the gate and up columns, or 64 x 32 tiles of the three
    gradients together, pass 2^32 threads of 512 a tile; the runtime would run what the lower bits say."""
    wide = 1 << 19
    assert (8 // 64 + 1 + 256) * (wide // 16) * 512 >= 1 << 32
    assert ffn(lib, False, 8, 256, 8, wide, 0) == EINVAL
    # dw13 (16 rows) and dx 2^31 each, dw2 2^30
    assert ffn(lib, True, 8, 256, wide, 8, 0) == EINVAL


def test_gate_backward_refuses_launches_of_2_32_threads(lib):
    """fp32: 64-column tiles of dh and of dw, 512 threads each, in one launch.  T = 1, d = 2^29 is 2^32 of them for dh
    alone, d = 2^28 for both."""
    def call(d, dh=P, dw=P):
        return lib.moelb_gate_backward(P, 1, d, 1, 1, 0, P, P, P, P, P, 1 << 62, dh, dw, P, None)
    assert call(1 << 29) == EINVAL and call((1 << 28) + 64) == EINVAL and call(1 << 28) == EINVAL
    assert call(1 << 29, dw=None) == EINVAL and call(1 << 29, dh=None) == EINVAL
