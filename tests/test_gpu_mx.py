"""GPU: MX 4-bit floating point against its definition in 64 bits.

Quantising and reading back are exact: codes, scales and values are equal.  The
FFN, before any run: products of two numbers of the format are exact in fp32,
their sums off by (terms + 8) 2^-24 of the magnitudes; an activation that lies
within its fp32 error of a border between two codes may take either
(oracle.mx.flip_step: the distance of the two, or of the two scales where the
block's largest crosses a power of two), which moves y by that times |W2|; y is
rounded once, u = eps / 2 of its type.
"""
import math

import pytest
import torch

from oracle import mx
from tests.gpu_layer import log

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def quantize(x):
    from routed_expert_ffn_gate_amd import moelb as M
    q = torch.full((*x.shape[:-1], x.shape[-1] // 2), 0xAA, dtype=torch.uint8, device="cuda")
    s = torch.full((*x.shape[:-1], M.moelb_mx_scale_bytes(x.shape[-1])), 0xAA, dtype=torch.uint8, device="cuda")
    M.moelb_mx_quantize(x, q, s)
    torch.cuda.synchronize()
    return q, s


def check_quantize(x):
    from routed_expert_ffn_gate_amd import moelb as M
    q, s = quantize(x)
    wq, wsc = mx.quantize(x)
    assert torch.equal(s, wsc)
    same = q == wq
    assert same.all(), (same.logical_not().nonzero()[:4], q[~same][:4], wq[~same][:4])
    for dtype in (BF, F32):
        v = torch.full(x.shape, 7.0, dtype=dtype, device="cuda")
        M.moelb_mx_dequantize(q, s, v)
        torch.cuda.synchronize()
        want = mx.dequantize(q, s).to(dtype)  # bf16 and fp32 hold the values exactly, or both end at infinity
        assert torch.equal(v.isnan(), want.isnan()) and torch.equal(v[~v.isnan()], want[~want.isnan()])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 32), (3, 64), (7, 96), (33, 544), (130, 2048), (1, 8192), (5, 7, 160),
                                   (1000, 32), (4097, 288)])
def test_quantize(moelb, shape, dtype):
    gen = torch.Generator(device="cuda").manual_seed(sum(shape))
    x = torch.randn(shape, generator=gen, device="cuda")
    x = x * torch.exp(2 * torch.randn((*shape[:-1], 1), generator=gen, device="cuda"))
    x[..., ::7] *= 30
    check_quantize(x.to(dtype))


def test_every_bf16_value(moelb):
    """All 65536 bit patterns, among random ones, and each beside the same largest value."""
    bits = torch.arange(65536, device="cuda", dtype=torch.int32).to(torch.int16)
    every = bits.view(BF)
    gen = torch.Generator(device="cuda").manual_seed(0)
    check_quantize(every[torch.randperm(65536, generator=gen, device="cuda")].view(512, 128))
    fine = every[torch.isfinite(every.float())]
    for big in (4.0, 7.5, 1e-30, 2.0 ** -126, 2.0 ** -133, 3e38):
        small = fine[fine.float().abs() <= big]
        x = torch.zeros(((small.numel() + 30) // 31, 32), dtype=BF, device="cuda")
        pad = torch.zeros((x.shape[0] * 31,), dtype=BF, device="cuda")
        pad[:small.numel()] = small
        x[:, 1:], x[:, 0] = pad.view(-1, 31), big
        check_quantize(x)


def test_borders(moelb):
    """Halfway values and their neighbours at many scales."""
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 6.5, 7.0, 7.99, 0.5, 1.0, 3.0, 0.0], device="cuda")
    x = torch.stack([mid, -mid, mid * (1 + 2.0 ** -23), mid * (1 - 2.0 ** -24)]).reshape(-1)
    row = torch.zeros((64,), device="cuda")
    row[:x.numel()] = x
    row[32], row[60] = 4.0, 4.0
    rows = torch.stack([torch.ldexp(row, torch.tensor(e, device="cuda")) for e in range(-140, 124, 3)])
    check_quantize(rows)


def test_nan_and_infinity_stay_in_their_block(moelb):
    x = torch.ones((4, 128), device="cuda")
    x[0, 40], x[1, 70], x[2, 0], x[3, 127] = math.nan, math.inf, -math.inf, math.nan
    for dtype in (BF, F32):
        q, s = quantize(x.to(dtype))
        v = mx.dequantize(q, s).view(4, 4, 32)
        bad = torch.zeros((4, 4), dtype=torch.bool, device="cuda")
        bad[0, 1] = bad[1, 2] = bad[2, 0] = bad[3, 3] = True
        assert v[bad].isnan().all() and (v[~bad] == 1).all()


def test_quantize_leaves_other_memory(moelb):
    from routed_expert_ffn_gate_amd import moelb as M
    x = torch.ones((3, 96), dtype=BF, device="cuda")
    q, s = torch.full((3 * 48 + 64,), 9, dtype=torch.uint8, device="cuda"), torch.full((3 * 16 + 64,), 9, dtype=torch.uint8, device="cuda")
    v = torch.full((3 * 96 + 64,), 9.0, device="cuda")
    M.moelb_mx_quantize(x, q[:144].view(3, 48), s[:48].view(3, 16))
    M.moelb_mx_dequantize(q[:144].view(3, 48), s[:48].view(3, 16), v[:288].view(3, 96))
    torch.cuda.synchronize()
    assert (q[144:] == 9).all() and (s[48:] == 9).all() and (v[288:] == 9).all() and (v[:288] == 1).all()


# ---------------------------------------------------------------- FFN


def weights(E, d, i, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    w13 = torch.randn((E, 2 * i, d), generator=gen, device="cuda") / d ** 0.5
    w2 = torch.randn((E, d, i), generator=gen, device="cuda") / i ** 0.5
    return *quantize(w13), *quantize(w2)


def run_ffn(x, rows, off, E, w, gather=None, gather_k=1, G=1, rank=-1, y=None):
    from routed_expert_ffn_gate_amd import moelb as M
    w13, s13, w2, s2 = w
    d, i = x.shape[1], w2.shape[-1] * 2
    n = M.moelb_mx_grouped_ffn_workspace_bytes(x.shape[0], rows, off.numel() - 1, E, d, i)
    assert n > 0
    ws = torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")
    y = torch.full((rows, d), 7.0, dtype=x.dtype, device="cuda") if y is None else y
    M.moelb_mx_grouped_ffn(x, rows, off, E, w13, s13, w2, s2, ws, y, G=G, rank=rank, gather=gather, gather_k=gather_k)
    torch.cuda.synchronize()
    return y


def check_ffn(x, counts, w, y, gather=None, gather_k=1, skip=()):
    """counts: rows of each group, group g of expert g mod E; groups in `skip` were not computed."""
    E, u = w[0].shape[0], torch.finfo(x.dtype).eps / 2
    X, w13, w2 = mx.rounded(x), mx.dequantize(w[0], w[1]), mx.dequantize(w[2], w[3])
    at, worst, num, den = 0, 0.0, 0.0, 0.0
    for g, n in enumerate(counts):
        rows = torch.arange(at, at + n, device="cuda")
        at += n
        if n == 0:
            continue
        if g in skip:
            assert (y[rows] == 7).all(), g
            continue
        src = rows if gather is None else gather[rows].long() // gather_k
        want, bound = mx.ffn_rows(X[src], w13[g % E], w2[g % E])
        allow = 1.01 * bound + u * (want.abs() + bound) + 1e-30
        diff = (y[rows].double() - want).abs()
        assert torch.isfinite(y[rows]).all()
        worst = max(worst, (diff / allow).max().item())
        num, den = num + (diff ** 2).sum().item(), den + (want ** 2).sum().item()
    log(f"    at most {worst:.3f} of the allowed error, rel {math.sqrt(num / max(den, 1e-300)):.2e}")
    assert worst <= 1.0
    # borders are rare: nearly all of the error is y's own rounding and a few of them
    assert math.sqrt(num) <= (u + 2e-3) * math.sqrt(den) + 1e-30


def offsets(counts):
    return torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32, device="cuda")


SHAPES = [
    # counts, d, inter
    ([1], 32, 32), ([1], 2048, 768), ([3, 0, 1, 60], 64, 96), ([64, 65, 1], 96, 64), ([5, 130, 33], 160, 224),
    ([0, 0, 17], 288, 32), ([200], 544, 1056), ([300, 40], 1056, 544), ([31, 1, 0, 64, 7, 2, 90, 128], 512, 256),
    ([700, 513], 320, 352), ([2] * 24, 1024, 128), ([257], 2048, 64), ([1] * 8, 256, 2080), ([1300, 20, 600], 256, 512),
]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("counts,d,inter", SHAPES, ids=lambda v: str(v)[:24])
def test_ffn(moelb, counts, d, inter, dtype):
    E, rows = len(counts), sum(counts)
    gen = torch.Generator(device="cuda").manual_seed(rows + d)
    x = torch.randn((rows, d), generator=gen, device="cuda").to(dtype)
    w = weights(E, d, inter, d + inter)
    log(f"[mx ffn] {counts} d={d} inter={inter} {dtype}")
    y = run_ffn(x, rows, offsets(counts), E, w)
    check_ffn(x, counts, w, y)
    assert torch.equal(y, run_ffn(x, rows, offsets(counts), E, w))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_ffn_of_few_rows_and_more_weights_than_the_caches_hold(moelb, dtype):
    """20 experts of 17 MB: their loads are marked non-temporal; K and the columns end inside a tile."""
    counts, d, inter = [2, 0, 3, 1, 9, 1, 0, 2, 4, 1, 5, 2, 1, 0, 6, 3, 1, 66, 2, 1], 2080, 5152
    x = torch.randn((sum(counts), d), generator=torch.Generator(device="cuda").manual_seed(6), device="cuda").to(dtype)
    w = weights(len(counts), d, inter, 7)
    log(f"[mx ffn] 20 experts d={d} inter={inter} {dtype}")
    y = run_ffn(x, sum(counts), offsets(counts), len(counts), w)
    check_ffn(x, counts, w, y)
    assert torch.equal(y, run_ffn(x, sum(counts), offsets(counts), len(counts), w))


def test_ffn_gathers_replicas_and_ranks(moelb):
    """Groups of several ranks share experts, rows come through a gather, one rank's share alone."""
    E, G, d, inter, k, T = 6, 4, 192, 160, 3, 90
    gen = torch.Generator(device="cuda").manual_seed(4)
    counts = torch.randint(0, 14, (2 * G * E,), generator=torch.Generator().manual_seed(5)).tolist()
    rows = sum(counts)
    x = torch.randn((T, d), generator=gen, device="cuda").to(BF)
    gather = torch.randint(0, T * k, (rows + 3,), generator=gen, device="cuda").to(torch.int32)
    w = weights(E, d, inter, 1)
    y = run_ffn(x, rows, offsets(counts), E, w, gather, k, G)
    check_ffn(x, counts, w, y, gather, k)
    for rank in (0, 3):
        part = run_ffn(x, rows, offsets(counts), E, w, gather, k, G, rank)
        check_ffn(x, counts, w, part, gather, k, skip=[g for g in range(2 * G * E) if (g // E) % G != rank])


def test_ffn_of_more_groups_than_one_launch_schedules(moelb):
    """6400 groups: the schedule has its own launches."""
    E, G, d, inter, k, T = 100, 32, 96, 64, 2, 700
    gen = torch.Generator(device="cuda").manual_seed(8)
    counts = torch.randint(0, 3, (2 * G * E,), generator=torch.Generator().manual_seed(9))
    counts[torch.rand((2 * G * E,), generator=torch.Generator().manual_seed(10)) < 0.7] = 0
    rows = int(counts.sum())
    x = torch.randn((T, d), generator=gen, device="cuda").to(BF)
    gather = torch.randint(0, T * k, (rows,), generator=gen, device="cuda").to(torch.int32)
    w = weights(E, d, inter, 11)
    y = run_ffn(x, rows, offsets(counts.tolist()), E, w, gather, k, G)
    check_ffn(x, counts.tolist(), w, y, gather, k)


@pytest.mark.parametrize("d,inter", [(1 << 17, 32), (32, 1 << 17)])
def test_ffn_of_wide_rows(moelb, d, inter):
    x = torch.randn((70, d), generator=torch.Generator(device="cuda").manual_seed(0), device="cuda").to(BF)
    w = weights(1, d, inter, 12)
    log(f"[mx ffn] wide d={d} inter={inter}")
    check_ffn(x, [70], w, run_ffn(x, 70, offsets([70]), 1, w))


def test_ffn_rows_outside_groups_and_offsets_out_of_range(moelb):
    E, d, inter, rows = 3, 64, 64, 100
    x = torch.randn((rows, d), generator=torch.Generator(device="cuda").manual_seed(0), device="cuda").to(BF)
    w = weights(E, d, inter, 2)
    y = run_ffn(x, rows, torch.tensor([10, 30, 30, 70], dtype=torch.int32, device="cuda"), E, w)
    assert (y[:10] == 7).all() and (y[70:] == 7).all()
    check_ffn(x[10:70], [20, 0, 40], w, y[10:70])
    # clamped to [0, rows]: rows 0..29 of expert 0, none of expert 1 (its end lies before its start), 20..99 of
    # expert 2, of which 70 are left of the call's 100 rows; 20..29 get one of the two results
    y = run_ffn(x, rows, torch.tensor([-5, 30, 20, 4000], dtype=torch.int32, device="cuda"), E, w)
    check_ffn(x[:20], [20, 0, 0], w, y[:20])
    check_ffn(x[30:90], [0, 0, 60], w, y[30:90])
    assert (y[90:] == 7).all()
    # gather entries outside the rows read row 0
    gather = torch.full((rows,), -3, dtype=torch.int32, device="cuda")
    gather[50:] = 1 << 30
    y = run_ffn(x, rows, offsets([rows, 0, 0]), E, w, gather, 1)
    check_ffn(x, [rows, 0, 0], w, y, torch.zeros_like(gather), 1)


def test_ffn_of_one_expert_without_leading_dimension(moelb):
    from routed_expert_ffn_gate_amd import moelb as M
    w = weights(1, 96, 64, 3)
    x = torch.randn((40, 96), generator=torch.Generator(device="cuda").manual_seed(0), device="cuda").to(BF)
    y = run_ffn(x, 40, offsets([40]), 1, w)
    ws = torch.empty((M.moelb_mx_grouped_ffn_workspace_bytes(40, 40, 1, 1, 96, 64),), dtype=torch.uint8, device="cuda")
    y2 = torch.empty_like(y)
    M.moelb_mx_grouped_ffn(x, 40, offsets([40]), 1, w[0][0], w[1][0], w[2][0], w[3][0], ws, y2)
    assert torch.equal(y, y2)


@pytest.mark.parametrize("d,inter,n", [(96, 64, 40), (512, 288, 300)])
def test_ffn_nan_of_one_row_or_expert(moelb, d, inter, n):
    """A NaN in a token's row reaches that row only; one in an expert's weights that expert's rows only."""
    E = 3
    x = torch.randn((n, d), generator=torch.Generator(device="cuda").manual_seed(0), device="cuda").to(BF)
    w = weights(E, d, inter, 3)
    counts = [n // 2, n - n // 2 - 3, 3]
    clean = run_ffn(x, n, offsets(counts), E, w)
    bad = x.clone()
    bad[7, 5] = math.nan
    y = run_ffn(bad, n, offsets(counts), E, w)
    assert y[7].isnan().all()
    keep = torch.arange(n, device="cuda") != 7
    assert torch.equal(y[keep], clean[keep])
    s13 = w[1].clone()
    s13[1, 3, 0] = 255
    y = run_ffn(x, n, offsets(counts), E, (w[0], s13, w[2], w[3]))
    own = slice(counts[0], counts[0] + counts[1])
    assert y[own].isnan().all()
    assert torch.equal(y[:own.start], clean[:own.start]) and torch.equal(y[own.stop:], clean[own.stop:])


def test_ffn_two_streams_and_a_graph(moelb):
    from routed_expert_ffn_gate_amd import moelb as M
    E, d, inter, counts = 4, 256, 192, [100, 3, 0, 70]
    rows = sum(counts)
    gen = torch.Generator(device="cuda").manual_seed(0)
    xs = [torch.randn((rows, d), generator=gen, device="cuda").to(BF) for _ in range(2)]
    w, off = weights(E, d, inter, 3), offsets(counts)
    want = [run_ffn(x, rows, off, E, w) for x in xs]
    n = M.moelb_mx_grouped_ffn_workspace_bytes(rows, rows, E, E, d, inter)
    ws = [torch.empty((n,), dtype=torch.uint8, device="cuda") for _ in range(2)]
    ys = [torch.empty_like(want[0]) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for j in range(2):
            M.moelb_mx_grouped_ffn(xs[j], rows, off, E, *w, ws[j], ys[j], stream=streams[j])
    torch.cuda.synchronize()
    assert torch.equal(ys[0], want[0]) and torch.equal(ys[1], want[1])
    x = torch.empty_like(xs[0])
    graph = torch.cuda.CUDAGraph()
    x.copy_(xs[0])
    with torch.cuda.graph(graph):
        M.moelb_mx_grouped_ffn(x, rows, off, E, *w, ws[0], ys[0])
    for j in (1, 0, 1):
        x.copy_(xs[j])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ys[0], want[j])
        assert torch.equal(run_ffn(xs[j], rows, off, E, w), want[j])
