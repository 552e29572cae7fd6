"""GPU: the shared projection with adapters against its formula in float64.

Tolerances, before any run; u = eps / 2 of the storage type.  y is rounded
once (u), the r values low = scale x A^T once (u of each, so u of the sum of
|low| |B|), and sums of n terms are formed in fp32 (n 2^-24 of their
magnitudes).  Gated: y = silu(g) u', whose error is at most |u'| 1.1 err(g) +
|silu(g)| err(u') (|silu'| <= 1.1) and a few ulp of the exponential.
"""
import pytest
import torch

from tests.gpu_layer import log

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def make(T, d_in, d_out, n, r, dtype, seed, ids=None):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    N = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, w = N(max(T, 1), d_in).to(dtype)[:T], (N(d_out, d_in) / d_in ** 0.5).to(dtype)
    a, b = (N(n, r, d_in) / d_in ** 0.5).to(dtype), (N(n, d_out, r) / r ** 0.5).to(dtype)
    scale = 0.5 + torch.rand((n,), generator=gen, device="cuda")
    if ids == "requests":  # runs of neighbours, some without an adapter
        runs = torch.randint(-1, n, (max(1, T // 37 + 1),), generator=gen, device="cuda")
        ids = runs[torch.arange(T, device="cuda") * len(runs) // max(T, 1)]
    elif ids is None:      # every token its own, ids outside [0, n) among them
        ids = torch.randint(-2, n + 2, (T,), generator=gen, device="cuda")
    return x, w, ids.to(torch.int32), a, b, scale


def run(x, w, ids, a, b, scale, gated):
    from routed_expert_ffn_gate_amd import moelb as M
    T, d_in = x.shape
    d_out = w.shape[0]
    y = torch.full((T, d_out // 2 if gated else d_out), 7.0, dtype=x.dtype, device="cuda")
    n, r = a.shape[:2] if a is not None else (0, 0)
    ws = torch.full((M.moelb_adapter_projection_workspace_bytes(T, d_in, d_out, n, r, M.dtype_code(x)),), 0xff,
                    dtype=torch.uint8, device="cuda")
    M.moelb_adapter_projection(x, w, ids, a, b, scale, ws, y, gated=gated)
    torch.cuda.synchronize()
    return y


def check(x, w, ids, a, b, scale, gated, y):
    u, f = torch.finfo(x.dtype).eps / 2, 2.0 ** -24
    X, W = x.double(), w.double()
    z, m = X @ W.t(), X.abs() @ W.abs().t()
    err = (x.shape[1] + 64) * f * m
    if a is not None:
        n, r = a.shape[:2]
        for v in ids.unique().tolist():
            if not 0 <= v < n:
                continue
            rows = (ids == v).nonzero()[:, 0]
            A, B, s = a[v].double(), b[v].double(), scale[v].double()
            low = s * (X[rows] @ A.t())
            lm = s * (X[rows].abs() @ A.abs().t())
            z[rows] += low @ B.t()
            err[rows] += (u * low.abs() + (x.shape[1] + 2) * f * lm) @ B.abs().t() * 1.01
            err[rows] += (r + 64) * f * (low.abs() @ B.abs().t())
    if gated:
        h = w.shape[0] // 2
        g, up, eg, eu = z[:, :h], z[:, h:], err[:, :h], err[:, h:]
        s = torch.sigmoid(g)
        want = g * s * up
        err = up.abs() * 1.1 * eg + (g * s).abs() * eu + 1.1 * eg * eu + 2.0 ** -20 * want.abs()
    else:
        want = z
    allow = 1.02 * (err + u * want.abs()) + 1e-30
    over = ((y.double() - want).abs() / allow).max().item() if want.numel() else 0.0
    rel = ((y.double() - want).norm() / want.norm().clamp_min(1e-30)).item()
    log(f"    at most {over:.3f} of the allowed error, rel {rel:.2e}")
    assert over <= 1.0


SHAPES = [
    # T, d_in, d_out, n, r
    (1, 8, 16, 1, 8), (1, 2048, 2048, 8, 16), (4, 264, 272, 3, 16), (3, 1000, 528, 2, 8), (1, 136, 48, 2, 64),
    (2, 520, 80, 5, 32), (1, 264, 272, 3, 72), (5, 4096, 144, 2, 16), (2, 72, 80, 3, 24), (16, 264, 48, 5, 16), (17, 200, 208, 40, 8),
    (33, 1000, 528, 64, 32), (64, 4096, 512, 64, 16), (65, 136, 144, 7, 64), (100, 512, 272, 9, 40),
    (129, 328, 272, 3, 72), (255, 2056, 272, 9, 16), (257, 1544, 528, 9, 24), (300, 264, 1040, 50, 256), (400, 4096, 656, 12, 16), (700, 520, 1040, 5, 128), (513, 64, 64, 2048, 8),
]


@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("order", ["requests", "mixed"])
@pytest.mark.parametrize("shape", SHAPES, ids=["x".join(map(str, s)) for s in SHAPES])
def test_against_formula(moelb, shape, order, dtype, gated):
    T, d_in, d_out, n, r = shape
    log(f"[adapter] T={T} d_in={d_in} d_out={d_out} n={n} r={r} {order} {dtype} gated={gated}")
    c = make(T, d_in, d_out, n, r, dtype, seed=T + r, ids="requests" if order == "requests" else None)
    check(*c, gated, run(*c, gated))


@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
def test_large_tiles(moelb, gated):
    # 256-row tiles: 12 requests over 5000 tokens, then every token its own adapter
    for ids in ("requests", None):
        log(f"[adapter] large gated={gated} {ids}")
        c = make(5000, 1032, 2560, 30, 64, BF, seed=9, ids=ids)
        check(*c, gated, run(*c, gated))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 40, 200])
def test_no_adapters_and_all_bare(moelb, T, dtype):
    x, w, ids, a, b, scale = make(T, 264, 272, 4, 16, dtype, seed=3)
    bare = run(x, w, None, None, None, None, True)
    check(x, w, ids, None, None, None, True, bare)
    assert torch.equal(run(x, w, torch.full_like(ids, -1), a, b, scale, True), bare)


def test_other_tokens_do_not_matter(moelb):
    """A token's result does not depend on the others: adapters and tokens full of NaN beside it leave it alone."""
    for T, dt in ((40, BF), (300, BF), (8000, BF), (40, F32), (300, F32)):
        x, w, ids, a, b, scale = make(T, 136, 144 if T < 8000 else 2064, 3, 16, dt, seed=4)
        ids = torch.arange(T, device="cuda").remainder(3).to(torch.int32)
        good = run(x, w, ids, a, b, scale, False)
        a2, b2, x2 = a.clone(), b.clone(), x.clone()
        a2[1], b2[1], x2[2::3] = float("nan"), float("nan"), float("nan")
        got = run(x2, w, ids, a2, b2, scale, False)
        assert torch.equal(got[0::3], good[0::3]), T
        assert bool(torch.isnan(got[1::3]).all()) and bool(torch.isnan(got[2::3]).all())


def test_same_bits_twice_and_captured(moelb):
    from routed_expert_ffn_gate_amd import moelb as M
    for T in (1, 50, 400):
        x, w, ids, a, b, scale = make(T, 264, 272, 6, 32, BF, seed=5, ids="requests")
        eager = run(x, w, ids, a, b, scale, True)
        y = torch.empty_like(eager)
        ws = torch.empty((M.moelb_adapter_projection_workspace_bytes(T, 264, 272, 6, 32, 1),), dtype=torch.uint8,
                         device="cuda")
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            M.moelb_adapter_projection(x, w, ids, a, b, scale, ws, y, gated=True)
        for _ in range(3):
            y.fill_(9.0)
            graph.replay()
            assert torch.equal(run(x, w, ids, a, b, scale, True), eager)
            assert torch.equal(y, eager)


@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("order", ["requests", "mixed"])
@pytest.mark.parametrize("shape", [(40, 2064, 2064, 9, 256), (128, 1288, 144, 5, 16), (129, 1288, 144, 5, 16),
                                   (1100, 4104, 80, 7, 16), (3, 4104, 48, 4, 16)], ids=lambda s: "x".join(map(str, s)))
def test_f32_parts_of_k(moelb, shape, order, gated):
    """fp32 calls with few tiles: k and a tile's adapters in parts, whole and with a short last part; few tokens whose
    rows of B are many; four ranks a wave."""
    t = make(*shape, F32, seed=21, ids="requests" if order == "requests" else None)
    check(*t, gated, run(*t, gated))


def test_f32_parts_keep_tokens_apart(moelb):
    """As test_other_tokens_do_not_matter, with k and the adapters in parts."""
    for T in (3, 40, 300):
        x, w, ids, a, b, scale = make(T, 2056, 144, 3, 16, F32, seed=22)
        ids = torch.arange(T, device="cuda").remainder(3).to(torch.int32)
        good = run(x, w, ids, a, b, scale, False)
        a2, b2, x2 = a.clone(), b.clone(), x.clone()
        a2[1], b2[1], x2[2::3] = float("nan"), float("inf"), float("nan")
        got = run(x2, w, ids, a2, b2, scale, False)
        assert torch.equal(got[0::3], good[0::3]), T
        assert bool(torch.isnan(got[1::3]).all()) and bool(torch.isnan(got[2::3]).all())


def test_f32_same_bits_twice_and_captured(moelb):
    from routed_expert_ffn_gate_amd import moelb as M
    for T in (2, 50, 400):
        x, w, ids, a, b, scale = make(T, 1544, 272, 6, 16, F32, seed=23)
        eager = run(x, w, ids, a, b, scale, True)
        y = torch.empty_like(eager)
        ws = torch.empty((max(1, M.moelb_adapter_projection_workspace_bytes(T, 1544, 272, 6, 16, M.dtype_code(x))),),
                         dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            M.moelb_adapter_projection(x, w, ids, a, b, scale, ws, y, gated=True)
        for _ in range(3):
            y.fill_(9.0)
            graph.replay()
            assert torch.equal(run(x, w, ids, a, b, scale, True), eager)
            assert torch.equal(y, eager)
