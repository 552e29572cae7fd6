"""GPU: the gate of the fp32 training form and of the fp32 gated projection, element by element.

x is a unit vector, so that z is a column of W13 exactly, W2 the identity and
dy ones, so that y is a and dw13 is dz exactly.  Tolerance, before any run,
in units of 2^-24 relative: the exponential 2 (one ulp), 1 + e^-g 1, the
quotient 1, g and u 1 each: a and du within 8.  dg = da u s (1 + g (1 - s)) is a
sum of two terms, so the same holds of u s (1 + |g| (1 - s)), with 1 - s off by
at most 4 of itself: 16.  Gates from -80 to 80: results below 1e-33 would
leave the normal range.
"""
import pytest
import torch

from tests.gpu_layer import log

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24


def gates(n, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    g = torch.linspace(-80, 80, n, device="cuda") + torch.rand((n,), generator=gen, device="cuda")
    g[0], g[1] = -1.2784645, 0.0  # silu' = 0, and the middle
    u = torch.randn((n,), generator=gen, device="cuda")
    return g, u.sign() * (0.5 + u.abs())


def test_training_form(moelb):
    from routed_expert_ffn_gate_amd import moelb as M
    i = 512
    g, u = gates(i, 1)
    x = torch.zeros((1, i), device="cuda")
    x[0, 5] = 1.0
    w13 = torch.zeros((1, 2 * i, i), device="cuda")
    w13[0, :i, 5], w13[0, i:, 5] = g, u
    w2 = torch.eye(i, device="cuda").unsqueeze(0).contiguous()
    off = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    z, y, dx = (torch.empty((1, n), device="cuda") for n in (2 * i, i, i))
    dw13, dw2, dy = torch.empty_like(w13), torch.empty_like(w2), torch.ones((1, i), device="cuda")
    F = M.MOELB_F32
    byte = lambda n: torch.empty((n,), dtype=torch.uint8, device="cuda")  # noqa: E731
    M.moelb_grouped_ffn_train(x, 1, off, 1, w13, w2, byte(M.moelb_grouped_ffn_workspace_bytes(1, 1, 1, i, i, F)),
                                  z, y)
    M.moelb_grouped_ffn_backward(dy, x, 1, off, 1, w13, w2, z,
                                     byte(M.moelb_grouped_ffn_backward_workspace_bytes(1, 1, 1, i, i, F)), dx, dw13,
                                     dw2)
    torch.cuda.synchronize()
    assert torch.equal(z[0, :i], g) and torch.equal(z[0, i:], u)
    G, U = g.double(), u.double()
    s, c = 1 / (1 + torch.exp(-G)), 1 / (1 + torch.exp(G))
    a, du, dg = G * s * U, G * s, U * s * (1 + G * c)
    for name, got, want, size, allow in (("a", y[0], a, a, 8), ("a again", dw2[0, 3], a, a, 8),
                                         ("du", dw13[0, i:, 5], du, du, 8),
                                         ("dg", dw13[0, :i, 5], dg, U * s * (1 + G.abs() * c), 16)):
        over = ((got.double() - want).abs() / (EPS * size.abs() + 1e-40)).max().item()
        log(f"[f32 gates] {name}: off by {over:.2f} of {allow} x 2^-24")
        assert over <= allow, name


@pytest.mark.parametrize("T,n", [(1, 0), (3, 0), (64, 0), (64, 1), (200, 1)], ids=str)
def test_gated_projection(moelb, T, n):
    """One launch, the tile, the sum's kernel; tokens with an adapter of zeros or none."""
    from routed_expert_ffn_gate_amd import moelb as M
    o = 512
    g, u = gates(o, 2)
    x = torch.zeros((T, 8), device="cuda")
    x[:, 3] = 1.0
    w = torch.zeros((2 * o, 8), device="cuda")
    w[:o, 3], w[o:, 3] = g, u
    y = torch.empty((T, o), device="cuda")
    r = 8
    ad = (None,) * 4 if n == 0 else (torch.zeros((T,), dtype=torch.int32, device="cuda"),
                                     torch.zeros((n, r, 8), device="cuda"), torch.zeros((n, 2 * o, r), device="cuda"),
                                     torch.ones((n,), device="cuda"))
    ws = torch.empty((max(1, M.moelb_adapter_projection_workspace_bytes(T, 8, 2 * o, n, r if n else 0,
                                                                            M.MOELB_F32)),), dtype=torch.uint8,
                     device="cuda")
    M.moelb_adapter_projection(x, w, *ad, ws, y, gated=True)
    torch.cuda.synchronize()
    G = g.double()
    want = G / (1 + torch.exp(-G)) * u.double()
    over = ((y.double() - want).abs() / (EPS * want.abs() + 1e-40)).max().item()
    log(f"[f32 gates] projection T={T} n={n}: off by {over:.2f} of 8 x 2^-24")
    assert over <= 8
