"""GPU: the router's gradient where a workgroup of dh takes several column
tiles one after another, and the norm of every error.

Tolerances: per element as for the smaller cases.  On the norm: bf16 dh and
dw carry two roundings to the type in a row (dz, the result), each at most u =
eps / 2 and independent from element to element: 4 u.  fp32 results and db:
logits and sums of up to a few thousand fp32 terms, 1e-5.
"""
import pytest
import torch

from tests.gpu_layer import log
from tests.test_gpu_combine_gate_backward import half, router_case, router_check, router_run

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def column_tiles(T, d):
    """128-column tiles of dh a bf16 workgroup takes, at least."""
    m, ntn = -(-T // 128), -(-d // 128)
    parts = min(-(-256 // m), ntn)
    return ntn // parts


def values(h, w, b, idx, dwts):
    p = torch.softmax(h.double() @ w.double().t() + b.double(), 1)
    q = torch.zeros_like(p).scatter_add_(1, idx.long(), dwts.double())
    dz = p * (q - (p * q).sum(1, keepdim=True))
    return dict(dh=dz @ w.double(), dw=dz.t() @ h.double(), db=dz.sum(0))


def norms(c, got):
    for n, want in values(*c).items():
        tol = 4 * half(BF) if c[0].dtype == BF and n != "db" else 1e-5
        rel = ((got[n].double() - want).norm() / want.norm()).item()
        log(f"    {n}: rel {rel:.2e} of {tol:.1e}")
        assert rel <= tol, n


@pytest.mark.parametrize("T,d,E,k", [(20000, 1000, 16, 2), (20000, 1000, 100, 8), (20000, 1000, 160, 8),
                                     (20000, 1000, 256, 8), (33000, 520, 16, 2), (33000, 520, 128, 4),
                                     (33000, 520, 256, 16), (4000, 4096, 64, 8)])
def test_several_column_tiles(moelb, T, d, E, k):
    n = column_tiles(T, d)
    assert n >= 3
    log(f"[gate backward] T={T} d={d} E={E} k={k}: {n} column tiles a workgroup")
    c = router_case(T, d, E, k, BF, seed=T + E)
    got = router_run(*c)
    router_check(*c, got)
    norms(c, got)
    again = router_run(*c)
    for name in got:
        assert torch.equal(got[name], again[name]), name


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,d,E,k", [(300, 1000, 128, 8), (1000, 136, 160, 3), (517, 264, 256, 16), (5000, 512, 16, 2),
                                     (40000, 64, 8, 2), (9000, 136, 64, 6)])
def test_norms(moelb, T, d, E, k, dtype):
    log(f"[gate backward] norms T={T} d={d} E={E} k={k} {dtype}")
    c = router_case(T, d, E, k, dtype, seed=T + E)
    norms(c, router_run(*c))
