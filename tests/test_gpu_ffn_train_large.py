"""GPU: the grouped FFN's training form with many experts, and on 256-row tiles
at ragged sizes, against its formulas in float64 (the tolerances of the smaller
cases: per element, and on the norm of the difference over the norm)."""
import pytest
import torch

from tests.gpu_layer import log
from tests.test_gpu_ffn_train import check, formulas, make, run
from tests.test_gpu_layer_train import build, dense_gradients, step

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def tile_height(rows, E, d, inter):
    """The bf16 form's row tiles: 256 for 192 rows an expert on average and 192 tiles of the narrower width."""
    return 256 if rows >= 192 * E and -(-rows // 256) * -(-min(d, inter) // 256) >= 192 else 128


def splits(rows, E, M, N, tile):
    """Parts of an expert's rows in a weight gradient."""
    slots = 256 if tile == 256 else 512
    return max(1, min(slots // (E * -(-M // tile) * -(-N // tile)), rows // E // 512, 16))


def routed(T, E, k, seed, spread=0.5):
    """k distinct experts a token over uneven popularities: (rows of every expert, pairs sorted by expert)."""
    gen = torch.Generator().manual_seed(seed)
    score = spread * torch.randn((E,), generator=gen) - torch.log(-torch.log(torch.rand((T, E), generator=gen).clamp(
        1e-20, 1 - 1e-7)))
    assert bool(torch.isfinite(score).all())
    flat = score.topk(k, dim=1).indices.reshape(-1)
    return torch.bincount(flat, minlength=E).tolist(), torch.argsort(flat, stable=True).to(torch.int32).cuda()


def routed_case(T, E, k, d, inter, dtype, seed):
    counts, gather = routed(T, E, k, seed)
    c = make(counts, d, inter, dtype, seed=seed, k=k, T=T)
    c["gather"] = gather
    return c, counts


@pytest.mark.parametrize("T,E,k,d,inter,dtype", [
    (512, 128, 8, 256, 136, BF), (512, 128, 8, 200, 64, F32),     # about 32 rows an expert
    (60, 256, 4, 136, 72, BF), (60, 256, 4, 72, 136, F32),        # experts without rows among them
    (1111, 24, 3, 1000, 520, BF), (1000, 16, 3, 264, 264, BF), (1000, 16, 3, 264, 264, F32),  # 139 and 188 an expert
    (3000, 64, 8, 264, 328, BF)])
def test_many_experts(moelb, T, E, k, d, inter, dtype):
    c, counts = routed_case(T, E, k, d, inter, dtype, seed=T + E)
    log(f"[ffn train] routed T={T} E={E} k={k} d={d} inter={inter} {dtype}: {min(counts)} to {max(counts)} rows")
    got = run(c)
    torch.cuda.synchronize()
    check(c, got, *formulas(c))


@pytest.mark.parametrize("counts,d,inter,k", [
    ([7001, 0, 3333, 2666], 1032, 1032, 2),       # K tails and ragged widths; the training form's own down product
    ([50000], 1032, 520, 3),                      # weight gradients of an expert in parts, gathered
    ([5000, 1, 0, 3333, 2100, 300, 4096], 1024, 1088, 4),  # whole K steps: the forward's down product
    ([130, 0, 9000, 2999, 255, 257, 1, 700], 1288, 1096, None)])
def test_256_row_tiles(moelb, counts, d, inter, k):
    rows, E = sum(counts), len(counts)
    tile = tile_height(rows, E, d, inter)
    assert tile == 256
    if E == 1:
        assert splits(rows, E, 2 * inter, d, tile) > 1 and splits(rows, E, d, inter, tile) > 1
    log(f"[ffn train] 256-row tiles counts={counts} d={d} inter={inter} k={k}")
    c = make(counts, d, inter, BF, seed=rows, k=k, T=rows // k if k else None)
    got = run(c)
    torch.cuda.synchronize()
    check(c, got, *formulas(c))
    again = run(c)
    torch.cuda.synchronize()
    for n in got:
        assert torch.equal(got[n], again[n]), n


def test_256_row_tiles_routed(moelb):
    """Uneven experts of a real routing, 64 of them: T 4096, top 4."""
    c, counts = routed_case(4096, 64, 4, 520, 776, BF, seed=5)
    assert tile_height(c["P"], 64, 520, 776) == 256
    log(f"[ffn train] 256-row tiles routed: {min(counts)} to {max(counts)} rows")
    got = run(c)
    torch.cuda.synchronize()
    check(c, got, *formulas(c))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_gradients_128_experts(moelb, dtype):
    """The layer's step and backward with 128 experts, every gradient by value; tolerance as for the smaller layers:
    four roundings to the type in a row, 1e-5 in fp32."""
    L, t = build(dtype, True, T=512, d=136, E=128, k=8, inter=72, G=8, N=4)
    o = step(L, t, train=True)
    g = L.backward(t["dout"], t["h"], t["wc"], t["bc"], t["w13"], t["w2"], t["s13"], t["s2"])
    torch.cuda.synchronize()
    _, want = dense_gradients(L, t, o.idx)
    tol = 4 * torch.finfo(BF).eps / 2 if dtype == "bf16" else 1e-5
    for name, got, ref in (("h", g.h, want["h"]), ("wc", g.w_cur, want["wc"]), ("bc", g.b_cur, want["bc"]),
                           ("w13", g.w13, want["w13"]), ("w2", g.w2, want["w2"]), ("s13", g.shared_w13, want["s13"]),
                           ("s2", g.shared_w2, want["s2"])):
        rel = ((got.double() - ref).norm() / ref.norm()).item()
        log(f"[layer train] 128 experts {dtype} {name}: rel {rel:.2e} of {tol:.1e}")
        assert rel <= tol, name
