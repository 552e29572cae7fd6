"""CPU: the scored router's and the MX 4-bit entry points refuse bad arguments on
the host before anything is launched, through the C ABI and through the binding."""
import ctypes
import math
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


@pytest.mark.parametrize("bad", [dict(T=-1), dict(d=0), dict(d=12), dict(d=(1 << 25) + 8), dict(E=0), dict(E=257),
                                 dict(dt=2), dict(h=N), dict(w=N), dict(z=N), dict(h=ODD), dict(w=ODD), dict(wn=ODD),
                                 dict(wn=N, bn=P), dict(wn=N, bn=N), dict(zn=N), dict(d=1 << 25, E=64)], ids=str)
def test_logits_refuses(lib, bad):
    a = dict(h=P, T=4, d=8, E=4, dt=1, w=P, b=P, wn=P, bn=P, z=P, zn=P)
    a.update(bad)
    assert lib.moelb_gate_logits(*a.values(), N) == EINVAL


def test_logits_of_no_tokens(lib):
    assert lib.moelb_gate_logits(N, 0, 8, 4, 1, P, N, N, N, N, N, N) == OK


@pytest.mark.parametrize("bad", [dict(T=-1), dict(E=0), dict(E=257), dict(k=0), dict(k=9), dict(E=64, k=17),
                                 dict(score=2), dict(score=-1), dict(groups=0), dict(groups=3), dict(groups=16),
                                 dict(topk=0), dict(groups=4, topk=5), dict(groups=4, topk=1, k=3), dict(top=0),
                                 dict(top=3), dict(groups=8, topk=8, top=2), dict(scale=math.inf),
                                 dict(scale=math.nan), dict(z=N), dict(idx=N)], ids=str)
def test_route_refuses(lib, bad):
    a = dict(z=P, T=4, E=8, k=2, score=0, bias=N, groups=1, topk=1, top=1, renorm=1, scale=1.0, idx=P, w=P, gap=P)
    a.update(bad)
    assert lib.moelb_route(*a.values(), N) == EINVAL
    if set(bad) <= {"z", "idx"}:
        assert lib.moelb_route(*{**a, "T": 0}.values(), N) == OK


def route_back(lib, **kw):
    a = dict(h=P, T=4, d=8, E=4, k=2, dt=1, w=P, z=P, idx=P, g=P, score=1, renorm=1, scale=1.0, ws=P, n=1 << 30, dh=P,
             dw=P, db=P)
    a.update(kw)
    return lib.moelb_route_backward(*a.values(), N)


@pytest.mark.parametrize("bad", [dict(T=-1), dict(d=0), dict(d=12), dict(E=0), dict(E=257), dict(k=0), dict(k=5),
                                 dict(E=32, k=17), dict(dt=2), dict(h=N), dict(w=N), dict(z=N), dict(idx=N), dict(g=N),
                                 dict(h=ODD), dict(w=ODD), dict(dh=ODD), dict(dw=ODD), dict(score=2),
                                 dict(scale=math.nan), dict(scale=-math.inf), dict(T=1 << 28, d=64),
                                 dict(d=(1 << 25) + 8)], ids=str)
def test_route_backward_refuses(lib, bad):
    assert route_back(lib, **bad) == EINVAL


def test_route_backward_workspace(lib):
    need = lib.moelb_route_backward_workspace_bytes(4, 8, 4, 1)
    assert need > 0
    assert route_back(lib, n=need - 1) == EWORKSPACE and route_back(lib, ws=N) == EWORKSPACE
    assert route_back(lib, ws=ODD) == EWORKSPACE
    assert route_back(lib, dh=N, dw=N, db=N) == OK
    for bad in ((-1, 8, 4, 1), (4, 0, 4, 1), (4, 8, 257, 1), (4, 8, 4, 2)):
        assert lib.moelb_route_backward_workspace_bytes(*bad) == 0


def test_mx_scale_bytes(lib):
    assert [lib.moelb_mx_scale_bytes(k) for k in (32, 512, 544, 2048, 4096)] == [16, 16, 32, 64, 128]
    assert [lib.moelb_mx_scale_bytes(k) for k in (0, -32, 16, 40)] == [0, 0, 0, 0]


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(K=0), dict(K=48), dict(K=-32), dict(dt=2), dict(x=N), dict(q=N),
                                 dict(s=N), dict(x=ODD), dict(q=ODD), dict(s=ODD), dict(rows=1 << 50),
                                 dict(rows=1 << 40)], ids=str)
def test_mx_quantize_refuses(lib, bad):
    a = dict(x=P, rows=4, K=64, dt=1, q=P, s=P)
    a.update(bad)
    assert lib.moelb_mx_quantize(a["x"], a["rows"], a["K"], a["dt"], a["q"], a["s"], N) == EINVAL
    assert lib.moelb_mx_dequantize(a["q"], a["s"], a["rows"], a["K"], a["dt"], a["x"], N) == EINVAL


def test_mx_quantize_of_no_rows(lib):
    assert lib.moelb_mx_quantize(N, 0, 64, 1, N, N, N) == OK
    assert lib.moelb_mx_dequantize(N, N, 0, 64, 1, N, N) == OK


def mx_ffn(lib, **kw):
    a = dict(x=P, rows_x=8, rows=8, off=P, groups=8, E=2, G=2, rank=-1, gather=N, gk=1, d=64, i=64, dt=1, w13=P, s13=P,
             w2=P, s2=P, ws=P, n=1 << 30, y=P)
    a.update(kw)
    return lib.moelb_mx_grouped_ffn(*a.values(), N)


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(rows_x=-1), dict(rows_x=0), dict(groups=0), dict(groups=32769),
                                 dict(E=0), dict(E=257), dict(d=0), dict(d=48), dict(d=1 << 20), dict(i=0), dict(i=48),
                                 dict(i=1 << 20), dict(dt=2), dict(rank=0, groups=7), dict(rank=2), dict(rank=0, G=0),
                                 dict(gather=P, gk=0), dict(off=N), dict(w13=N), dict(s13=N), dict(w2=N), dict(s2=N),
                                 dict(x=N), dict(y=N), dict(x=ODD), dict(w13=ODD), dict(s13=ODD), dict(w2=ODD),
                                 dict(s2=ODD), dict(y=ODD), dict(rows=1 << 28, rows_x=1 << 28), dict(rows=1 << 27),
                                 dict(rows_x=1 << 28), dict(d=1 << 17, i=1 << 15)], ids=str)
def test_mx_ffn_refuses(lib, bad):
    assert mx_ffn(lib, **bad) == EINVAL


def test_mx_ffn_workspace(lib):
    need = lib.moelb_mx_grouped_ffn_workspace_bytes(8, 8, 8, 2, 64, 64)
    assert need > 0
    assert mx_ffn(lib, n=need - 1) == EWORKSPACE and mx_ffn(lib, ws=N) == EWORKSPACE and mx_ffn(lib, ws=ODD) == EWORKSPACE
    assert mx_ffn(lib, rows=0, x=N, y=N) == OK
    for bad in ((-1, 8, 8, 2, 64, 64), (8, -1, 8, 2, 64, 64), (8, 8, 0, 2, 64, 64), (8, 8, 8, 257, 64, 64),
                (8, 8, 8, 2, 48, 64), (8, 8, 8, 2, 64, 16), (8, 1 << 30, 8, 2, 64, 64)):
        assert lib.moelb_mx_grouped_ffn_workspace_bytes(*bad) == 0


def test_binding_checks_tensors(monkeypatch):
    """Shapes, types and devices, before the library is called."""
    from routed_expert_ffn_gate_amd import moelb as M
    monkeypatch.setattr(M, "_device", lambda name, t: t.get_device())
    monkeypatch.setattr(M, "_queue", lambda stream, dev: None)
    E = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype)  # noqa: E731
    i32, u8, bf = torch.int32, torch.uint8, torch.bfloat16
    calls = [
        lambda: M.moelb_gate_logits(E(4, 8), E(6, 8), E(5), None, None, E(4, 6)),
        lambda: M.moelb_gate_logits(E(4, 8), E(6, 8, dtype=bf), E(6), None, None, E(4, 6)),
        lambda: M.moelb_gate_logits(E(4, 8), E(6, 8), E(6), E(5, 8), None, E(4, 6), E(4, 6)),
        lambda: M.moelb_gate_logits(E(4, 8), E(6, 8), E(6), None, None, E(4, 6, dtype=bf)),
        lambda: M.moelb_route(E(4, 6), E(4, 2), E(4, 2)),
        lambda: M.moelb_route(E(4, 6), E(3, 2, dtype=i32), E(4, 2)),
        lambda: M.moelb_route(E(4, 6), E(4, 2, dtype=i32), E(4, 3)),
        lambda: M.moelb_route(E(4, 6), E(4, 2, dtype=i32), E(4, 2), bias=E(5)),
        lambda: M.moelb_route(E(6, 4).t(), E(4, 2, dtype=i32), E(4, 2)),
        lambda: M.moelb_route_backward(E(4, 8), E(6, 8), E(4, 5), E(4, 2, dtype=i32), E(4, 2), E(1 << 16, dtype=u8)),
        lambda: M.moelb_mx_quantize(E(4, 48), E(4, 24, dtype=u8), E(4, 16, dtype=u8)),
        lambda: M.moelb_mx_quantize(E(4, 64), E(4, 64, dtype=u8), E(4, 16, dtype=u8)),
        lambda: M.moelb_mx_quantize(E(4, 64), E(4, 32, dtype=u8), E(4, 2, dtype=u8)),
        lambda: M.moelb_mx_quantize(E(4, 64, dtype=torch.float16), E(4, 32, dtype=u8), E(4, 16, dtype=u8)),
        lambda: M.moelb_mx_dequantize(E(4, 32), E(4, 16, dtype=u8), E(4, 64)),
        # weights of two experts for three; a row too many without a gather; the gather too short
        lambda: M.moelb_mx_grouped_ffn(E(4, 64), 4, E(4, dtype=i32), 3, E(2, 64, 32, dtype=u8), E(2, 64, 16, dtype=u8),
                                       E(2, 64, 16, dtype=u8), E(2, 64, 16, dtype=u8), None, E(4, 64)),
        lambda: M.moelb_mx_grouped_ffn(E(4, 64), 5, E(3, dtype=i32), 2, E(2, 64, 32, dtype=u8), E(2, 64, 16, dtype=u8),
                                       E(2, 64, 16, dtype=u8), E(2, 64, 16, dtype=u8), None, E(5, 64)),
        lambda: M.moelb_mx_grouped_ffn(E(4, 64), 5, E(3, dtype=i32), 2, E(2, 64, 32, dtype=u8), E(2, 64, 16, dtype=u8),
                                       E(2, 64, 16, dtype=u8), E(2, 64, 16, dtype=u8), None, E(5, 64),
                                       gather=E(4, dtype=i32), gather_k=2),
    ]
    for call in calls:
        with pytest.raises(M.MoelbError):
            call()
