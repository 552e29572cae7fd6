"""GPU: the grouped FFN's training form against its formulas in float64.

Tolerances, before any run.  With u = eps / 2 of the storage type (bf16 2^-8,
fp32 2^-24), each output is rounded once (error at most u relative to the
value) and its product reads operands rounded once more (a or dz): every term
of a sum is off by at most u of itself, so the sum by at most u times the sum
of the terms' magnitudes.  Those are compared per element: |got - want| <=
u |want| + c u sum|terms|, c = 1 for bf16 with 2 % for the second order and
the fp32 arithmetic behind.  fp32: nothing is rounded between, but sums of n
terms in fp32 in any order are off by at most n 2^-24 of the magnitudes, and
the inputs of a nonlinearity are themselves such sums; c = 2 (d + inter + n)
covers both products and the hardware exponential and reciprocal (a few ulp).
"""
import pytest
import torch

from tests.gpu_layer import log

pytestmark = pytest.mark.gpu


def make(counts, d, inter, dtype, seed, k=None, T=None, scale=1.0):
    """Rows sorted into groups of the given sizes; with k, gathered from T tokens."""
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    E, P = len(counts), sum(counts)
    n = lambda *s: torch.randn(s, generator=gen, device=dev)  # noqa: E731
    rows_x = P if k is None else T
    x = (n(max(rows_x, 1), d) * scale).to(dtype)[:rows_x]
    gather = None
    if k is not None:
        gather = torch.randint(0, T * k, (P,), generator=gen, device=dev).to(torch.int32)
    off = torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32, device=dev)
    w13 = (n(E, 2 * inter, d) * (1.0 / d ** 0.5)).to(dtype)
    w2 = (n(E, d, inter) * (1.0 / inter ** 0.5)).to(dtype)
    dy = n(max(P, 1), d).to(dtype)[:P]
    return dict(x=x, off=off, w13=w13, w2=w2, dy=dy, gather=gather, k=k or 1, E=E, P=P, d=d, inter=inter, dtype=dtype)


def run(c, G=1, rank=-1, num_groups=None, fill=0.0, want=("dx", "dw13", "dw2"), stream=None):
    from routed_expert_ffn_gate_amd import moelb as M
    code = M.MOELB_BF16 if c["dtype"] == torch.bfloat16 else M.MOELB_F32
    P, d, i, E = c["P"], c["d"], c["inter"], c["E"]
    ng = c["off"].numel() - 1
    dev = "cuda"
    z = torch.empty((P, 2 * i), dtype=torch.float32, device=dev)
    y, dx = (torch.full((P, d), fill, dtype=c["dtype"], device=dev) for _ in range(2))
    dw13, dw2 = torch.full_like(c["w13"], 7.0), torch.full_like(c["w2"], 7.0)
    ws = torch.full((M.moelb_grouped_ffn_workspace_bytes(P, ng, E, d, i, code),), 0xff, dtype=torch.uint8, device=dev)
    wb = torch.full((M.moelb_grouped_ffn_backward_workspace_bytes(P, ng, E, d, i, code),), 0xff, dtype=torch.uint8,
                    device=dev)
    kw = dict(G=G, rank=rank, gather=c["gather"], gather_k=c["k"], stream=stream)
    M.moelb_grouped_ffn_train(c["x"], P, c["off"], E, c["w13"], c["w2"], ws, z, y, **kw)
    M.moelb_grouped_ffn_backward(c["dy"], c["x"], P, c["off"], E, c["w13"], c["w2"], z, wb,
                                 dx if "dx" in want else None, dw13 if "dw13" in want else None,
                                 dw2 if "dw2" in want else None, **kw)
    return dict(y=y, dx=dx, dw13=dw13, dw2=dw2, z=z)


def formulas(c, groups=None):
    """float64 values and the sums of the terms' magnitudes; groups: (lo, hi, expert)."""
    E, i = c["E"], c["inter"]
    off = c["off"].tolist()
    if groups is None:
        groups = [(off[g], off[g + 1], g % E) for g in range(len(off) - 1)]
    D = lambda t: t.double()  # noqa: E731
    val = dict(y=torch.zeros_like(D(c["dy"])), dx=torch.zeros_like(D(c["dy"])), dw13=torch.zeros_like(D(c["w13"])),
               dw2=torch.zeros_like(D(c["w2"])))
    mag = {n: t.clone() for n, t in val.items()}
    for lo, hi, e in groups:
        src = torch.arange(lo, hi, device="cuda") if c["gather"] is None else c["gather"][lo:hi].long() // c["k"]
        x, dy = D(c["x"])[src], D(c["dy"])[lo:hi]
        w13, w2 = D(c["w13"][e]), D(c["w2"][e])
        z = x @ w13.t()
        g, u = z[:, :i], z[:, i:]
        s = torch.sigmoid(g)
        a = g * s * u
        da = dy @ w2
        dz = torch.cat([da * u * s * (1 + g * (1 - s)), da * g * s], 1)
        for n, p, q in (("y", a, w2.t()), ("dx", dz, w13), ("dw13", dz.t(), x), ("dw2", dy.t(), a)):
            at = slice(lo, hi) if n in ("y", "dx") else e
            if n in ("y", "dx"):
                val[n][at], mag[n][at] = p @ q, p.abs() @ q.abs()
            else:
                val[n][at] += p @ q
                mag[n][at] += p.abs() @ q.abs()
        # fp32 errors of the products before the nonlinearity reach dz through
        # every term: their magnitudes, with |da| as a sum
        if c["dtype"] == torch.float32:
            zm = x.abs() @ w13.abs().t()
            dam = dy.abs() @ w2.abs()
            gm, um = zm[:, :i], zm[:, i:]
            am = gm * (1 + um)
            dzm = torch.cat([dam * (1 + um) * 2 * (1 + gm), dam * (1 + gm)], 1)
            for n, p, q in (("y", am, w2.abs().t()), ("dx", dzm, w13.abs()), ("dw13", dzm.t(), x.abs()),
                            ("dw2", dy.abs().t(), am)):
                at = slice(lo, hi) if n in ("y", "dx") else e
                if n in ("y", "dx"):
                    mag[n][at] = p @ q
                else:
                    mag[n][at] += p @ q
    return val, mag


def check(c, got, val, mag, names=("y", "dx", "dw13", "dw2")):
    u = torch.finfo(c["dtype"]).eps / 2
    n = c["d"] + c["inter"] + c["P"]
    for name in names:
        want, m = val[name], mag[name]
        cterm = 1.02 if c["dtype"] == torch.bfloat16 else 2.0 * n
        allow = 1.02 * u * want.abs() + cterm * u * m + 1e-30
        over = ((got[name].double() - want).abs() / allow).max().item() if want.numel() else 0.0
        rel = ((got[name].double() - want).norm() / want.norm().clamp_min(1e-30)).item()
        log(f"    {name}: at most {over:.3f} of the allowed error, rel {rel:.2e}")
        assert over <= 1.0, (name, over)
        assert rel <= (4 * u if c["dtype"] == torch.bfloat16 else 2e-6), (name, rel)


SHAPES = [
    # counts, d, inter, k, T
    ([1], 8, 8, None, None),
    ([1], 64, 64, None, None),
    ([5, 0, 1, 130], 72, 40, None, None),
    ([0, 0, 0], 64, 32, None, None),
    ([63, 64, 65, 127, 128, 129], 128, 96, 2, 97),
    ([300, 1, 0, 257], 200, 136, 3, 111),
    ([700], 264, 328, None, None),
    ([2200, 1900], 264, 264, None, None),      # more than 32 steps of rows: the index registers refill
    ([0, 2300, 40], 136, 264, 4, 500),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=[str(i) for i in range(len(SHAPES))])
def test_against_formulas(moelb, shape, dtype):
    counts, d, inter, k, T = shape
    log(f"[ffn train] counts={counts} d={d} inter={inter} k={k} T={T} {dtype}")
    c = make(counts, d, inter, dtype, seed=1, k=k, T=T)
    got = run(c)
    torch.cuda.synchronize()
    check(c, got, *formulas(c))


@pytest.mark.parametrize("counts,d,inter", [([1500, 1300, 900, 1700], 1024, 768), ([6000], 2048, 1040)])
def test_large_tiles(moelb, counts, d, inter):
    """Sizes that take the 256-row tiles, and one block whose weight gradients are split over its rows."""
    log(f"[ffn train] large counts={counts} d={d} inter={inter}")
    c = make(counts, d, inter, torch.bfloat16, seed=2, k=2, T=sum(counts) // 2)
    got = run(c)
    torch.cuda.synchronize()
    check(c, got, *formulas(c))


def test_rows_of_every_tile_height_256(moelb):
    # 24576 rows of 4 experts, d = inter = 2048: the 256-row tiles on every product
    counts = [9000, 6001, 5555, 4020]
    log(f"[ffn train] counts={counts} d=2048 inter=2048")
    c = make(counts, 2048, 2048, torch.bfloat16, seed=3)
    got = run(c)
    torch.cuda.synchronize()
    check(c, got, *formulas(c))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_rank_share_and_rows_outside(moelb, dtype):
    """Groups of two ranks and two segments; one rank computed: its rows only, the rest as they were."""
    E, G = 3, 2
    counts = [5, 70, 0, 33, 1, 130, 12, 0, 9, 64, 3, 40]  # 2 * G * E groups
    c = make(counts, 64, 48, dtype, seed=4)
    c["E"], c["w13"], c["w2"] = E, c["w13"][:E].contiguous(), c["w2"][:E].contiguous()
    c["off"] = c["off"].clone()
    off = c["off"].tolist()
    log("[ffn train] rank 1 of 2")
    got = run(c, G=G, rank=1, fill=3.0)
    torch.cuda.synchronize()
    groups = [(off[g], off[g + 1], g % E) for g in range(len(counts)) if (g // E) % G == 1]
    val, mag = formulas(c, groups)
    outside = torch.ones(c["P"], dtype=torch.bool, device="cuda")
    for lo, hi, _ in groups:
        outside[lo:hi] = False
    for n in ("y", "dx"):
        assert bool((got[n][outside] == 3.0).all())
        val[n][outside] = 3.0
        mag[n][outside] = 0.0
    check(c, got, val, mag)


def test_rows_behind_the_last_group_and_zero_rows(moelb):
    c = make([40, 30], 64, 64, torch.bfloat16, seed=5)
    c["P"] = 90  # 20 rows behind the last group
    c["x"] = torch.cat([c["x"], torch.full((20, 64), float("nan"), device="cuda", dtype=c["dtype"])])
    c["dy"] = torch.cat([c["dy"], torch.full((20, 64), float("nan"), device="cuda", dtype=c["dtype"])])
    got = run(c, fill=3.0)
    torch.cuda.synchronize()
    assert bool((got["y"][70:] == 3.0).all()) and bool((got["dx"][70:] == 3.0).all())
    val, mag = formulas(c)
    for n in ("y", "dx"):
        got[n], val[n], mag[n] = got[n][:70], val[n][:70], mag[n][:70]
    check(c, got, val, mag)
    c = make([0, 0], 64, 64, torch.bfloat16, seed=5)
    got = run(c)
    assert not bool(got["dw13"].any()) and not bool(got["dw2"].any())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_many_groups(moelb, dtype):
    """More groups than the one-launch schedule takes (4096): 1000 groups of each of 5 experts."""
    gen = torch.Generator().manual_seed(12)
    counts = (torch.randint(0, 12, (5000,), generator=gen) // 9).tolist()
    c = make(counts[:5], 72, 40, dtype, seed=12)
    P = sum(counts)
    more = make([P], 72, 40, dtype, seed=13)
    c.update(x=more["x"], dy=more["dy"], P=P,
             off=torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32, device="cuda"))
    got = run(c)
    torch.cuda.synchronize()
    off, E = c["off"].tolist(), 5
    rows = [[r for g in range(e, 5000, E) for r in range(off[g], off[g + 1])] for e in range(E)]
    # an expert's rows gathered together are one group of it
    order = torch.tensor(sum(rows, []), device="cuda")
    d = dict(c, x=c["x"][order], dy=c["dy"][order],
             off=torch.tensor([0] + list(torch.tensor([len(r) for r in rows]).cumsum(0)), device="cuda"))
    for n in ("y", "dx"):
        got[n] = got[n][order]
    check(c, got, *formulas(d))


def test_offsets_out_of_order_stay_inside(moelb):
    """Offsets that are negative, past the rows or decreasing: every access stays in the buffers (the schedule clamps
    them), and groups with sound offsets before them keep their rows."""
    c = make([40, 30, 20], 64, 64, torch.bfloat16, seed=14)
    good = run(c)
    c["off"] = torch.tensor([0, 40, 35, 1 << 30], dtype=torch.int32, device="cuda")
    run(c)
    c["off"] = torch.tensor([-7, 40, -1, 3], dtype=torch.int32, device="cuda")
    got = run(c)
    torch.cuda.synchronize()
    assert torch.equal(got["y"][3:40], good["y"][3:40])


def test_only_what_is_asked(moelb):
    c = make([100, 60], 64, 64, torch.bfloat16, seed=6)
    full = run(c)
    for want in (("dx",), ("dw13",), ("dw2",)):
        got = run(c, want=want)
        for n in ("dx", "dw13", "dw2"):
            if n in want:
                assert torch.equal(got[n], full[n])
            else:
                assert bool((got[n] == (0.0 if n == "dx" else 7.0)).all())


def test_same_bits_twice_and_on_another_stream(moelb):
    c = make([800, 900], 264, 200, torch.bfloat16, seed=7, k=2, T=600)
    a = run(c)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        b = run(c)
    torch.cuda.synchronize()
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_gradient_against_differences(moelb):
    """fp32: the directional derivative of <y, dy> along random directions, by central differences of the
    library's own forward.  The step h = 1e-2 leaves a third-order term of about h^2 and a rounding of about
    2^-24 |y| / h per product, both under 1e-3 of the derivative's size here."""
    c = make([9, 0, 20], 32, 24, torch.float32, seed=8)
    got = run(c)
    gen = torch.Generator(device="cuda").manual_seed(9)
    h = 1e-2
    for name, grad in (("x", "dx"), ("w13", "dw13"), ("w2", "dw2")):
        v = torch.randn(c[name].shape, generator=gen, device="cuda")
        v /= v.norm() / c[name].norm() * 4
        side = []
        for s in (1, -1):
            m = dict(c)
            m[name] = c[name] + s * h * v
            side.append((run(m)["y"].double() * c["dy"].double()).sum())
        diff = ((side[0] - side[1]) / (2 * h)).item()
        mine = (got[grad].double() * v.double()).sum().item()
        size = (got[grad].double().norm() * v.double().norm()).item()
        log(f"    {name}: differences {diff:.6f}, gradient {mine:.6f}, of at most {size:.3f}")
        assert abs(diff - mine) <= 1e-3 * size


def test_extreme_gates(moelb):
    """Gates far outside the exponential's range: silu and its slope go to 0 and to 1, nothing becomes NaN."""
    c = make([64], 64, 64, torch.float32, seed=10, scale=300.0)
    got = run(c)
    torch.cuda.synchronize()
    for n in ("y", "dx", "dw13", "dw2"):
        assert bool(torch.isfinite(got[n]).all()), n
    val, _ = formulas(c)
    for n in ("y", "dx", "dw13", "dw2"):
        # z in the hundreds is off by about |z| 64 2^-24 and the result follows it in proportion
        assert ((got[n].double() - val[n]).norm() / val[n].norm()).item() < 1e-4, n


def test_captured_and_replayed(moelb):
    c = make([500, 300], 128, 136, torch.bfloat16, seed=11, k=2, T=400)
    from routed_expert_ffn_gate_amd import moelb as M
    eager = run(c)
    P, d, i, E = c["P"], c["d"], c["inter"], c["E"]
    z = torch.empty((P, 2 * i), dtype=torch.float32, device="cuda")
    y, dx = torch.empty_like(c["dy"]), torch.empty_like(c["dy"])
    dw13, dw2 = torch.empty_like(c["w13"]), torch.empty_like(c["w2"])
    ws = torch.empty((M.moelb_grouped_ffn_workspace_bytes(P, E, E, d, i, 1),), dtype=torch.uint8, device="cuda")
    wb = torch.empty((M.moelb_grouped_ffn_backward_workspace_bytes(P, E, E, d, i, 1),), dtype=torch.uint8,
                     device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.moelb_grouped_ffn_train(c["x"], P, c["off"], E, c["w13"], c["w2"], ws, z, y, gather=c["gather"], gather_k=2)
        M.moelb_grouped_ffn_backward(c["dy"], c["x"], P, c["off"], E, c["w13"], c["w2"], z, wb, dx, dw13, dw2,
                                     gather=c["gather"], gather_k=2)
    for _ in range(3):
        for t in (z, y, dx, dw13, dw2):
            t.fill_(9.0)
        graph.replay()
        again = run(c)  # the program's own calls between the replays
        torch.cuda.synchronize()
        for n, t in dict(y=y, dx=dx, dw13=dw13, dw2=dw2).items():
            assert torch.equal(t, eager[n]) and torch.equal(again[n], eager[n]), n
