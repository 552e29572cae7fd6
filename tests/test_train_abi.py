"""CPU: the training and adapter entry points refuse bad arguments on the host
before anything is launched, through the C ABI and through the binding."""
import ctypes
import os

import pytest
import torch

P = ctypes.c_void_p(4096)   # aligned, never dereferenced: the checks fail first, or nothing is launched
ODD = ctypes.c_void_p(4104)
N = None
OK, EINVAL, EWORKSPACE = 0, 1, 3


@pytest.fixture(scope="module")
def lib():
    from routed_expert_ffn_gate_amd import moelb as M
    if not os.path.exists(M.LIB_PATH):
        pytest.fail("libmoelb.so is not built (run python -m routed_expert_ffn_gate_amd.build)")
    return M.lib()


def train(lib, x=P, rows_x=8, rows=8, off=P, groups=8, E=2, G=2, rank=-1, gather=N, gk=1, d=8, i=8, dt=1, w13=P, w2=P,
          ws=P, n=1 << 30, z=P, y=P):
    return lib.moelb_grouped_ffn_train(x, rows_x, rows, off, groups, E, G, rank, gather, gk, d, i, dt, w13, w2, ws, n, z,
                                       y, N)


def back(lib, dy=P, x=P, rows_x=8, rows=8, off=P, groups=8, E=2, G=2, rank=-1, gather=N, gk=1, d=8, i=8, dt=1, w13=P,
         w2=P, z=P, ws=P, n=1 << 30, dx=P, d13=P, d2=P):
    return lib.moelb_grouped_ffn_backward(dy, x, rows_x, rows, off, groups, E, G, rank, gather, gk, d, i, dt, w13, w2, z,
                                          ws, n, dx, d13, d2, N)


BAD_FFN = [dict(rows=-1), dict(rows_x=-1), dict(rows_x=0), dict(groups=0), dict(groups=32769), dict(E=0), dict(E=257),
           dict(d=0), dict(d=12), dict(i=0), dict(i=12), dict(dt=2), dict(rank=0, groups=7), dict(rank=2),
           dict(rank=0, G=0), dict(gather=P, gk=0), dict(off=N), dict(w13=N), dict(w2=N), dict(x=N), dict(x=ODD),
           dict(w13=ODD), dict(w2=ODD), dict(z=N), dict(z=ODD), dict(rows=1 << 28, rows_x=1 << 28),
           dict(rows=1 << 20, d=8, i=2048), dict(d=1 << 15, i=1 << 15)]


@pytest.mark.parametrize("bad", BAD_FFN + [dict(y=N), dict(y=ODD)], ids=str)
def test_ffn_train_refuses(lib, bad):
    assert train(lib, **bad) == EINVAL


@pytest.mark.parametrize("bad", BAD_FFN + [dict(dy=N), dict(dy=ODD), dict(dx=ODD), dict(d13=ODD), dict(d2=ODD)], ids=str)
def test_ffn_backward_refuses(lib, bad):
    assert back(lib, **bad) == EINVAL


def test_ffn_workspaces(lib):
    need = lib.moelb_grouped_ffn_workspace_bytes(8, 8, 2, 8, 8, 1)
    assert train(lib, n=need - 1) == EWORKSPACE and train(lib, ws=N) == EWORKSPACE
    need = lib.moelb_grouped_ffn_backward_workspace_bytes(8, 8, 2, 8, 8, 1)
    assert need > 0
    assert back(lib, n=need - 1) == EWORKSPACE and back(lib, ws=N) == EWORKSPACE and back(lib, ws=ODD) == EWORKSPACE
    # nothing asked for, no rows: nothing is launched
    assert back(lib, dx=N, d13=N, d2=N) == OK
    assert train(lib, rows=0, x=N, y=N, z=N) == OK
    assert lib.moelb_grouped_ffn_backward_workspace_bytes(-1, 8, 2, 8, 8, 1) == 0
    assert lib.moelb_grouped_ffn_backward_workspace_bytes(8, 8, 2, 8, 8, 3) == 0
    big = lib.moelb_grouped_ffn_backward_workspace_bytes(1 << 16, 8, 2, 1024, 1024, 1)
    assert big < lib.moelb_grouped_ffn_backward_workspace_bytes(1 << 17, 8, 2, 1024, 1024, 1)


def test_combine_backward_refuses(lib):
    def call(dout=P, y=P, rows=8, pos=P, wts=P, T=4, k=2, d=8, dt=1, dy=P, dw=P):
        return lib.moelb_combine_backward(dout, y, rows, pos, wts, T, k, d, dt, dy, dw, N)
    for bad in (dict(T=-1), dict(rows=-1), dict(k=0), dict(k=17), dict(d=0), dict(d=12), dict(dt=2), dict(dout=N),
                dict(pos=N), dict(wts=N), dict(dw=N), dict(y=N), dict(dy=N), dict(dout=ODD), dict(y=ODD), dict(dy=ODD)):
        assert call(**bad) == EINVAL, bad
    assert call(T=0) == OK


def test_gate_backward_refuses(lib):
    def call(h=P, T=4, d=8, E=4, k=2, dt=1, w=P, b=P, idx=P, g=P, ws=P, n=1 << 30, dh=P, dw=P, db=P):
        return lib.moelb_gate_backward(h, T, d, E, k, dt, w, b, idx, g, ws, n, dh, dw, db, N)
    for bad in (dict(T=-1), dict(d=0), dict(d=12), dict(E=0), dict(E=257), dict(k=0), dict(k=5), dict(E=32, k=17),
                dict(dt=2), dict(h=N), dict(w=N), dict(b=N), dict(idx=N), dict(g=N), dict(h=ODD), dict(w=ODD),
                dict(dh=ODD), dict(dw=ODD), dict(T=1 << 28)):
        assert call(**bad) == EINVAL, bad
    need = lib.moelb_gate_backward_workspace_bytes(4, 8, 4, 1)
    assert call(n=need - 1) == EWORKSPACE and call(ws=N) == EWORKSPACE and call(ws=ODD) == EWORKSPACE
    assert call(dh=N, dw=N, db=N) == OK
    assert lib.moelb_gate_backward_workspace_bytes(4, 8, 257, 1) == 0


def test_adapter_refuses(lib):
    def call(x=P, T=40, di=8, do=16, dt=1, w=P, ids=P, a=P, b=P, s=P, n=2, r=8, gated=0, ws=P, nb=1 << 30, y=P):
        return lib.moelb_adapter_projection(x, T, di, do, dt, w, ids, a, b, s, n, r, gated, ws, nb, y, N)
    for bad in (dict(T=-1), dict(di=0), dict(di=12), dict(do=0), dict(do=12), dict(do=24, gated=1), dict(dt=2),
                dict(n=-1), dict(r=0), dict(r=12), dict(r=264), dict(w=N), dict(a=N), dict(b=N), dict(s=N), dict(x=N),
                dict(y=N), dict(ids=N), dict(x=ODD), dict(w=ODD), dict(a=ODD), dict(b=ODD), dict(y=ODD),
                dict(T=1 << 29), dict(n=1 << 25)):
        assert call(**bad) == EINVAL, bad
    need = lib.moelb_adapter_projection_workspace_bytes(40, 8, 16, 2, 8, 1)
    assert need > 0
    assert call(nb=need - 1) == EWORKSPACE and call(ws=N) == EWORKSPACE and call(ws=ODD) == EWORKSPACE
    assert call(T=0) == OK and call(T=0, n=0, r=0, ids=N, a=N, b=N, s=N, ws=N, nb=0) == OK
    # one token with few ranks needs none
    assert lib.moelb_adapter_projection_workspace_bytes(1, 8, 16, 2, 8, 1) == 0


def test_gate_backward_refuses_operands_past_the_descriptor(lib):
    """w and dz (E padded to 64) are addressed with 32-bit byte offsets too.  No workspace: nothing is launched."""
    def call(T, d, E, dt):
        return lib.moelb_gate_backward(P, T, d, E, 1, dt, P, P, P, P, N, 0, P, P, P, N)
    assert call(1 << 26, 8, 64, 1) == EINVAL and call(1 << 25, 8, 8, 0) == EINVAL   # dz of 8 GiB
    assert call(4, 1 << 23, 256, 1) == EINVAL                                       # w of 4 GiB
    assert call(1 << 24, 8, 64, 1) == EWORKSPACE and call(4, 1 << 22, 256, 1) == EWORKSPACE


def test_adapter_refuses_an_adapter_past_the_descriptor(lib):
    """r * d_in of 8 GiB: one adapter's A is addressed with 32-bit byte offsets.  T = 0: nothing is launched."""
    def call(di, r):
        return lib.moelb_adapter_projection(P, 0, di, 8, 1, P, P, P, P, P, 1, r, 0, P, 1 << 30, P, N)
    assert call(1 << 24, 256) == EINVAL
    assert call(1 << 24, 64) == OK


def test_binding_refuses():
    """Shapes, types and devices are the binding's to check: the library sees pointers."""
    from routed_expert_ffn_gate_amd import moelb as M
    bf, f = torch.bfloat16, torch.float32
    x, w = torch.zeros((4, 8), dtype=bf), torch.zeros((16, 8), dtype=bf)
    with pytest.raises(M.MoelbError, match="not on the current GPU"):
        M.moelb_adapter_projection(x, w, None, None, None, None, None, torch.zeros((4, 16), dtype=bf))
    with pytest.raises(M.MoelbError, match="not on the current GPU"):
        M.moelb_combine_backward(x, x, torch.zeros(8, dtype=torch.int32), torch.zeros(4, 2), x, torch.zeros(4, 2))
    with pytest.raises(M.MoelbError, match="not on the current GPU"):
        M.moelb_gate_backward(x, w, torch.zeros(16), torch.zeros((4, 2), dtype=torch.int32), torch.zeros(4, 2), None)
    for good, bad in ((torch.zeros(4, 8), dict(shape=(4, 9))), (torch.zeros(4, 8), dict(dtype=bf)),
                      (torch.zeros(8, 4).t(), dict()), (torch.zeros(4, 8), dict(dev=0))):
        kw = dict(dict(shape=(4, 8), dtype=f, dev=-1), **bad)
        with pytest.raises(M.MoelbError):
            M._arg("call", "t", good, kw["shape"], kw["dtype"], kw["dev"])
    assert M._arg("call", "t", None, (1,), f, -1) is None
    t = torch.zeros(4, 8)
    assert M._arg("call", "t", t, (4, 8), f, -1) == t.data_ptr()
    with pytest.raises(M.MoelbError):
        M._ffn_args("call", x, 5, torch.zeros(2, dtype=torch.int32), 1, torch.zeros((16, 8), dtype=bf),
                    torch.zeros((8, 8), dtype=bf), None, -1)
    with pytest.raises(M.MoelbError):
        M._ffn_args("call", x, 4, torch.zeros(2, dtype=torch.int32), 2, torch.zeros((16, 8), dtype=bf),
                    torch.zeros((8, 8), dtype=bf), None, -1)
    with pytest.raises(M.MoelbError):
        M._ffn_args("call", x, 4, torch.zeros(2, dtype=torch.int32), 1, torch.zeros((1, 16, 8), dtype=bf),
                    torch.zeros((1, 8, 8), dtype=bf), torch.zeros(3, dtype=torch.int32), -1)
