"""GPU: the shared projection with adapters at sizes whose launches pass 2^32 threads."""
import pytest
import torch

from tests.gpu_layer import log

pytestmark = pytest.mark.gpu


def test_f32_low_products_of_many_tokens(moelb):
    """fp32, T r = 335 M low products of a wave each (21 M workgroups of 256 threads).  Tolerance as for every fp32
    call: sums of 8 and of 40 terms, (n + 64) 2^-24 of the terms' magnitudes."""
    from routed_expert_ffn_gate_amd import moelb as M
    T, d, n, r = 1 << 23, 8, 3, 40
    log(f"[adapter] f32 T={T} d={d} n={n} r={r}")
    gen = torch.Generator(device="cuda").manual_seed(31)
    N = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, w, a, b = N(T, d), N(d, d), N(n, r, d), N(n, d, r) / r ** 0.5
    scale = torch.tensor([0.5, 1.0, 2.0], device="cuda")
    ids = (torch.arange(T, device="cuda") // 37 % 4 - 1).to(torch.int32)
    ws = torch.empty((M.moelb_adapter_projection_workspace_bytes(T, d, d, n, r, M.MOELB_F32),),
                     dtype=torch.uint8, device="cuda")
    y = torch.full((T, d), 7.0, device="cuda")
    M.moelb_adapter_projection(x, w, ids, a, b, scale, ws, y)
    torch.cuda.synchronize()
    rows = torch.cat([torch.arange(5000, device="cuda"), torch.arange(T - 5000, T, device="cuda"),
                      torch.randint(0, T, (100000,), generator=gen, device="cuda")])
    X, W, own = x[rows].double(), w.double(), ids[rows]
    want, mag = X @ W.t(), X.abs() @ W.abs().t()
    for v in range(n):
        at = (own == v).nonzero()[:, 0]
        A, B, s = a[v].double(), b[v].double(), scale[v].double()
        want[at] += s * (X[at] @ A.t() @ B.t())
        mag[at] += s * (X[at].abs() @ A.abs().t() @ B.abs().t())
    over = ((y[rows].double() - want).abs() / ((8 + 40 + 64) * 2.0 ** -24 * mag)).max().item()
    log(f"    at most {over:.3f} of the allowed error")
    assert over <= 1.0


@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
def test_one_token_many_rows(moelb, gated):
    """One launch of 16 (gated: 8 and 8) rows a workgroup of 1024 threads, 2^22 workgroups and more.  Tolerance: sums
    of 8 terms, (8 + 64) 2^-24 of their magnitudes, silu's slope at most 1.1, one rounding to bf16."""
    from routed_expert_ffn_gate_amd import moelb as M
    bf = torch.bfloat16
    d, o = 8, (1 << 26) + 48
    log(f"[adapter] one token d_out={o} gated={gated}")
    gen = torch.Generator(device="cuda").manual_seed(32)
    x = torch.randn((1, d), generator=gen, device="cuda").to(bf)
    w = torch.randn((o, d), generator=gen, device="cuda").to(bf)
    y = torch.full((1, o // 2 if gated else o), 7.0, dtype=bf, device="cuda")
    M.moelb_adapter_projection(x, w, None, None, None, None, None, y, gated=gated)
    torch.cuda.synchronize()
    v, e = torch.zeros(o, device="cuda"), torch.zeros(o, device="cuda")
    for j in range(d):  # elementwise (a library product of 2^26 rows and a vector came out wrong); fp32 like the call
        p = w[:, j].float() * x[0, j].float()
        v += p
        e += p.abs() * (72 * 2.0 ** -24)
    if gated:
        g, u, eg, eu = v[:o // 2], v[o // 2:], e[:o // 2], e[o // 2:]
        s = g * torch.sigmoid(g)
        v = s * u
        e = 1.1 * u.abs() * eg + s.abs() * eu + 1.1 * eg * eu + 2.0 ** -20 * v.abs()
    over = ((y[0].float() - v).abs() / (1.02 * (e + 2.0 ** -8 * v.abs()) + 1e-30)).max().item()
    log(f"    at most {over:.3f} of the allowed error")
    assert over <= 1.0


def sampled(x, w, y, gated, seed):
    """The largest share of the allowed error over 4 M outputs: random ones and the last rows' last columns."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T, out = y.shape
    n = 1 << 22
    t = torch.randint(0, T, (n,), generator=gen, device="cuda")
    c = torch.randint(0, out, (n,), generator=gen, device="cuda")
    t[:1000], c[:1000] = T - 1, torch.arange(out - 1000, out, device="cuda")
    X = x[t].double()

    def row(i):
        W = w[i].double()
        return (X * W).sum(1), (X.abs() * W.abs()).sum(1) * (72 * 2.0 ** -24)
    v, e = row(c)
    if gated:
        u, eu = row(c + out)
        s = v * torch.sigmoid(v)
        v, e = s * u, 1.1 * u.abs() * e + s.abs() * eu + 1.1 * e * eu + 2.0 ** -20 * (s * u).abs()
    half = torch.finfo(y.dtype).eps / 2
    return ((y[t, c].double() - v).abs() / (1.02 * (e + half * v.abs()) + 1e-30)).max().item()


@pytest.mark.parametrize("T,o,dtype,gated", [(200, (1 << 25) + (1 << 24), torch.bfloat16, False),
                                             ((1 << 20) + 64, 1 << 15, torch.float32, True)], ids=["few", "f32 tile"])
def test_many_outputs(moelb, T, o, dtype, gated):
    """4.8e9 threads of the few tokens' sum (two outputs each), and 4.3e9 of the fp32 tiles: 20 to 70 GB of outputs."""
    from routed_expert_ffn_gate_amd import moelb as M
    torch.cuda.empty_cache()
    d = 8
    log(f"[adapter] T={T} d_out={o} {dtype} gated={gated}")
    gen = torch.Generator(device="cuda").manual_seed(33)
    x = torch.randn((T, d), generator=gen, device="cuda").to(dtype)
    w = torch.randn((o, d), generator=gen, device="cuda").to(dtype)
    code = M.MOELB_BF16 if dtype == torch.bfloat16 else M.MOELB_F32
    ws = torch.empty((max(1, M.moelb_adapter_projection_workspace_bytes(T, d, o, 0, 0, code)),), dtype=torch.uint8,
                     device="cuda")
    y = torch.full((T, o // 2 if gated else o), 7.0, dtype=dtype, device="cuda")
    M.moelb_adapter_projection(x, w, None, None, None, None, ws, y, gated=gated)
    torch.cuda.synchronize()
    over = sampled(x, w, y, gated, 34)
    log(f"    at most {over:.3f} of the allowed error")
    del x, w, ws, y
    torch.cuda.empty_cache()
    assert over <= 1.0
