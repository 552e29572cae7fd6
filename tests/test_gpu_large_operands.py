"""GPU: operands between 2 and 4 GiB (byte offsets past the signed 32 bits) and
weights of more than 4 GiB in all, calls beside each other on two streams, and
values that are not numbers beside ones that are.  Tolerances as in the smaller
cases, on sampled rows: each output within 4 u of the float64 value's norm (u =
eps / 2; at most four roundings in a row), sums in fp32 far below that."""
import pytest
import torch

from tests.gpu_layer import log
from tests.test_gpu_combine_gate_backward import router_case, router_run
from tests.test_gpu_ffn_train import make, run
from tests.test_gpu_adapter import make as adapter_make
from tests.test_gpu_layer_train import build, dense_gradients, step

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -8


def rel(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


def filled(shape, gen, dtype=BF, scale=1.0):
    """Random values without a copy of the whole in fp32."""
    t = torch.empty(shape, dtype=dtype, device="cuda")
    for part in t.view(-1).split(1 << 26):
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda") * scale)
    return t


@pytest.mark.parametrize("gathered", [True, False], ids=["gather", "rows"])
def test_ffn_rows_past_2_gib(moelb, gathered):
    """x, dy, y and dx of 4.09 GB (the limit is 2^32 - 2^21 bytes); two experts, the second's rows behind 2 GiB."""
    torch.cuda.empty_cache()
    d, i, P = 2048, 40, 1_000_000
    gen = torch.Generator(device="cuda").manual_seed(41)
    c = dict(x=filled((P, d), gen), dy=filled((P, d), gen), w13=filled((2, 2 * i, d), gen, scale=d ** -0.5),
             w2=filled((2, d, i), gen, scale=i ** -0.5), E=2, P=P, d=d, inter=i, dtype=BF, k=1,
             off=torch.tensor([0, 400_000, P], dtype=torch.int32, device="cuda"),
             gather=torch.randperm(P, generator=gen, device="cuda").to(torch.int32) if gathered else None)
    log(f"[large operands] ffn rows {P} x {d} gathered={gathered}")
    got = run(c)
    torch.cuda.synchronize()
    rows = torch.cat([torch.arange(0, 3000, device="cuda"), torch.arange(399_000, 401_000, device="cuda"),
                      torch.arange(P - 3000, P, device="cuda")])
    dw13, dw2 = torch.zeros((2, 2 * i, d), dtype=torch.float64, device="cuda"), torch.zeros(
        (2, d, i), dtype=torch.float64, device="cuda")
    for e, (lo, hi) in enumerate(((0, 400_000), (400_000, P))):
        w13, w2 = c["w13"][e].double(), c["w2"][e].double()

        def grads(q):
            x = c["x"][q if c["gather"] is None else c["gather"][q].long()].double()
            dy = c["dy"][q].double()
            g, u = (x @ w13.t()).chunk(2, 1)
            s = torch.sigmoid(g)
            da = dy @ w2
            return x, dy, g * s * u, torch.cat([da * u * s * (1 + g * (1 - s)), da * g * s], 1)
        for q in torch.arange(lo, hi, device="cuda").split(50_000):
            x, dy, a, dz = grads(q)
            dw13[e] += dz.t() @ x
            dw2[e] += dy.t() @ a
        q = rows[(rows >= lo) & (rows < hi)]
        x, dy, a, dz = grads(q)
        for n, want in (("y", a @ w2.t()), ("dx", dz @ w13)):
            assert rel(got[n][q], want) <= 4 * U, (n, e)
    for n, want in (("dw13", dw13), ("dw2", dw2)):
        for e in range(2):
            assert rel(got[n][e], want[e]) <= 4 * U, (n, e)
    del c, got
    torch.cuda.empty_cache()


def test_ffn_weights_past_4_gib(moelb):
    """W13 of 4.7 GB in all, rows for the first and the last experts only; the others' gradients are zeros."""
    torch.cuda.empty_cache()
    d, i, E = 4096, 14336, 20
    gen = torch.Generator(device="cuda").manual_seed(42)
    counts = [9] + [0] * (E - 3) + [70, 33]
    P = sum(counts)
    c = dict(x=filled((P, d), gen), dy=filled((P, d), gen), w13=filled((E, 2 * i, d), gen, scale=d ** -0.5),
             w2=filled((E, d, i), gen, scale=i ** -0.5), E=E, P=P, d=d, inter=i, dtype=BF, k=1, gather=None,
             off=torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32, device="cuda"))
    log(f"[large operands] ffn weights {E} x {2 * i} x {d}")
    got = run(c)
    torch.cuda.synchronize()
    off = c["off"].tolist()
    for e in (0, E - 2, E - 1):
        q = slice(off[e], off[e + 1])
        x, dy, w13, w2 = c["x"][q].double(), c["dy"][q].double(), c["w13"][e].double(), c["w2"][e].double()
        g, u = (x @ w13.t()).chunk(2, 1)
        s = torch.sigmoid(g)
        a, da = g * s * u, dy @ w2
        dz = torch.cat([da * u * s * (1 + g * (1 - s)), da * g * s], 1)
        for n, have, want in (("y", got["y"][q], a @ w2.t()), ("dx", got["dx"][q], dz @ w13),
                              ("dw13", got["dw13"][e], dz.t() @ x), ("dw2", got["dw2"][e], dy.t() @ a)):
            assert rel(have, want) <= 4 * U, (n, e)
    assert not any(bool(got[n][1:E - 2].any()) for n in ("dw13", "dw2"))
    del c, got
    torch.cuda.empty_cache()


@pytest.mark.parametrize("E", [16, 200])
def test_router_rows_past_2_gib(moelb, E):
    torch.cuda.empty_cache()
    T, d, k = 1_000_000, 2048, 4
    gen = torch.Generator(device="cuda").manual_seed(43)
    h, w, b = filled((T, d), gen), filled((E, d), gen, scale=d ** -0.5), torch.randn(E, generator=gen, device="cuda")
    idx = torch.stack([(torch.arange(T, device="cuda") * 7 + j * (E // k)) % E for j in range(k)], 1).to(torch.int32)
    dwts = torch.randn((T, k), generator=gen, device="cuda")
    log(f"[large operands] router {T} x {d} E={E}")
    got = router_run(h, w, b, idx, dwts)
    dw, db = torch.zeros((E, d), dtype=torch.float64, device="cuda"), torch.zeros(E, dtype=torch.float64, device="cuda")
    for q in torch.arange(T, device="cuda").split(50_000):
        p = torch.softmax(h[q].double() @ w.double().t() + b.double(), 1)
        g = torch.zeros_like(p).scatter_add_(1, idx[q].long(), dwts[q].double())
        dz = p * (g - (p * g).sum(1, keepdim=True))
        dw += dz.t() @ h[q].double()
        db += dz.sum(0)
        if int(q[0]) in (0, 500_000, 950_000):
            assert rel(got["dh"][q], dz @ w.double()) <= 4 * U
    assert rel(got["dw"], dw) <= 4 * U and rel(got["db"], db) <= 1e-5
    del h, got
    torch.cuda.empty_cache()


@pytest.mark.parametrize("mixed", [False, True], ids=["requests", "mixed"])
def test_adapter_rows_past_2_gib(moelb, mixed):
    from routed_expert_ffn_gate_amd import moelb as M
    torch.cuda.empty_cache()
    T, d, o, n, r = 1_000_000, 2048, 80, 5, 24
    gen = torch.Generator(device="cuda").manual_seed(44)
    x, w = filled((T, d), gen), filled((o, d), gen, scale=d ** -0.5)
    a, b = filled((n, r, d), gen, scale=d ** -0.5), filled((n, o, r), gen, scale=r ** -0.5)
    scale = 0.5 + torch.rand(n, generator=gen, device="cuda")
    t = torch.arange(T, device="cuda")
    ids = ((t if mixed else t // 4097) % (n + 1) - 1).to(torch.int32)
    ws = torch.empty((M.moelb_adapter_projection_workspace_bytes(T, d, o, n, r, M.MOELB_BF16),), dtype=torch.uint8,
                     device="cuda")
    y = torch.full((T, o), 7.0, dtype=BF, device="cuda")
    log(f"[large operands] adapter {T} x {d} mixed={mixed}")
    M.moelb_adapter_projection(x, w, ids, a, b, scale, ws, y)
    torch.cuda.synchronize()
    for q in t.split(50_000):
        X = x[q].double()
        want = X @ w.double().t()
        for v in range(n):
            at = (ids[q] == v).nonzero()[:, 0]
            want[at] += scale[v].double() * (X[at] @ a[v].double().t() @ b[v].double().t())
        assert rel(y[q], want) <= 4 * U, int(q[0])
    del x, y, ws
    torch.cuda.empty_cache()


def test_calls_beside_each_other(moelb):
    """Two streams at once, each with workspaces of its own: the bits of each call alone."""
    from tests.test_gpu_adapter import run as adapter_run
    from routed_expert_ffn_gate_amd import moelb as M
    cs = [make([700, 0, 1900, 333], 520, 264, BF, seed=51, k=3, T=1000), make([50] * 30, 264, 520, BF, seed=52)]
    alone = [run(c) for c in cs]
    rc = [router_case(3000, 520, 100, 8, BF, seed=53), router_case(900, 264, 200, 8, BF, seed=54)]
    ralone = [router_run(*c) for c in rc]
    ac = [adapter_make(600, 1032, 528, 9, 32, BF, seed=55), adapter_make(70, 520, 272, 9, 16, BF, seed=56)]
    aalone = [adapter_run(*c, False) for c in ac]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]

    def queue(j):
        """All three on the current stream, without a wait."""
        out = [run(cs[j])]
        h, w, b, idx, g = rc[j]
        ws = torch.empty((M.moelb_gate_backward_workspace_bytes(*h.shape, w.shape[0], M.MOELB_BF16),), dtype=torch.uint8,
                         device="cuda")
        o = [torch.empty_like(t) for t in (h, w, b)]
        M.moelb_gate_backward(h, w, b, idx, g, ws, *o)
        x, w, ids, a, b, s = ac[j]
        ws2 = torch.empty((M.moelb_adapter_projection_workspace_bytes(*x.shape, w.shape[0], *a.shape[:2], M.MOELB_BF16),),
                          dtype=torch.uint8, device="cuda")
        y = torch.empty((x.shape[0], w.shape[0]), dtype=BF, device="cuda")
        M.moelb_adapter_projection(x, w, ids, a, b, s, ws2, y)
        return out + [dict(zip(("dh", "dw", "db"), o)), y, ws, ws2]
    for _ in range(4):
        torch.cuda.synchronize()
        got = []
        for j, st in enumerate(streams):
            with torch.cuda.stream(st):
                got.append(queue(j))
        torch.cuda.synchronize()
        for j in range(2):
            assert all(torch.equal(got[j][0][n], alone[j][n]) for n in alone[j])
            assert all(torch.equal(got[j][1][n], ralone[j][n]) for n in ralone[j])
            assert torch.equal(got[j][2], aalone[j])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_an_experts_nan_stays_its_own(moelb, dtype):
    """Rows, gradients and weights of one expert full of NaN: the others keep their bits."""
    c = make([70, 130, 5, 64], 136, 72, dtype, seed=61)
    good = run(c)
    bad = dict(c, x=c["x"].clone(), dy=c["dy"].clone(), w13=c["w13"].clone(), w2=c["w2"].clone())
    for t, at in ((bad["x"], slice(70, 200)), (bad["dy"], slice(70, 200)), (bad["w13"], 1), (bad["w2"], 1)):
        t[at] = float("nan")
    got = run(bad)
    torch.cuda.synchronize()
    for n in ("y", "dx"):
        assert torch.equal(got[n][:70], good[n][:70]) and torch.equal(got[n][200:], good[n][200:]), n
        assert bool(torch.isnan(got[n][70:200]).all()), n
    for n in ("dw13", "dw2"):
        for e in (0, 2, 3):
            assert torch.equal(got[n][e], good[n][e]), (n, e)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("E", [24, 200])
def test_a_tokens_nan_stays_out_of_other_tokens(moelb, E, dtype):
    h, w, b, idx, g = router_case(300, 136, E, 4, dtype, seed=62)
    good = router_run(h, w, b, idx, g)["dh"]
    h2, g2 = h.clone(), g.clone()
    h2[7::10], g2[3::10] = float("nan"), float("inf")
    got = router_run(h2, w, b, idx, g2)["dh"]
    keep = torch.ones(300, dtype=torch.bool, device="cuda")
    keep[7::10] = keep[3::10] = False
    assert torch.equal(got[keep], good[keep])


@pytest.mark.parametrize("gather", [True, False], ids=["gather", "rows"])
def test_layer_with_the_split_beside_the_permutation(moelb, gather):
    """More than 8192 pairs: the split runs on its own stream beside the local half of the permutation."""
    L, t = build("bf16", True, T=1100, d=136, E=32, k=8, inter=72, G=4, N=2, gather=gather)
    assert L.overlap_split
    o = step(L, t, train=True)
    g = L.backward(t["dout"], t["h"], t["wc"], t["bc"], t["w13"], t["w2"], t["s13"], t["s2"])
    torch.cuda.synchronize()
    _, want = dense_gradients(L, t, o.idx)
    for got, ref in ((g.h, want["h"]), (g.w_cur, want["wc"]), (g.b_cur, want["bc"]), (g.w13, want["w13"]),
                     (g.w2, want["w2"]), (g.shared_w13, want["s13"]), (g.shared_w2, want["s2"])):
        assert rel(got, ref) <= 4 * U
    L.step_two_stage(t["h"], t["wc"], t["bc"], t["wn"], t["bn"], t["home"], t["replica"], t["w13"], t["w2"], t["s13"],
                     t["s2"])
    with pytest.raises(RuntimeError):
        L.backward(t["dout"], t["h"], t["wc"], t["bc"], t["w13"], t["w2"], t["s13"], t["s2"])
