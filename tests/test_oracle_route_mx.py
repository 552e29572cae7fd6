"""CPU: the references of the scored router and of MX 4-bit, pinned to values worked out by hand."""
import math

import pytest
import torch

from oracle import mx, scored_router as R


def test_softmax_renormalised():
    z = torch.log(torch.tensor([[1.0, 2.0, 4.0, 1.0]]))
    idx, w, gap = R.route(z, 2, renorm=True)
    assert idx.tolist() == [[2, 1]]
    assert w[0].tolist() == pytest.approx([4 / 6, 2 / 6], rel=1e-6)
    assert gap[0] == pytest.approx(2 / 8 - 1 / 8, rel=1e-6)
    idx, w, _ = R.route(z, 4)
    assert idx.tolist() == [[2, 1, 0, 3]] and w.sum() == pytest.approx(1.0)


def test_bias_moves_picks_not_weights():
    z = torch.zeros((1, 4))
    idx, w, _ = R.route(z, 2, score="sigmoid", bias=torch.tensor([0.0, 0.2, 0.1, -1.0]), scale=3.0)
    assert idx.tolist() == [[1, 2]] and w[0].tolist() == [1.5, 1.5]


def test_groups():
    s = torch.tensor([[0.9, 0.1, 0.6, 0.6, 0.8, 0.3]])
    z = torch.log(s / (1 - s))
    kw = dict(score="sigmoid", groups=3, topk_groups=1)
    assert R.route(z, 2, group_top=1, **kw)[0].tolist() == [[0, 1]]
    assert R.route(z, 2, group_top=2, **kw)[0].tolist() == [[2, 3]]


def test_masks():
    z = torch.tensor([[-math.inf, 1.0, math.nan, 0.0], [-math.inf] * 4])
    for score in ("softmax", "sigmoid"):
        idx, w, gap = R.route(z, 3, score=score, renorm=True)
        assert idx.tolist() == [[1, 3, -1], [-1, -1, -1]]
        assert w[0].sum() == pytest.approx(1.0) and w[0, 2] == 0 and w[1].sum() == 0
        assert torch.isinf(gap).all()


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_against_differences(score, renorm):
    gen = torch.Generator().manual_seed(3)
    z = torch.randn((5, 9), generator=gen, dtype=torch.float64).float()
    g = torch.randn((5, 3), generator=gen, dtype=torch.float64)
    kw = dict(score=score, renorm=renorm, scale=1.7)
    idx = R.route(z, 3, **kw)[0]
    dz, mag = R.route_dz(z, idx, g, **kw)

    def value(x):
        s = torch.softmax(x, 1) if score == "softmax" else torch.sigmoid(x)
        w = s.gather(1, idx.long())
        return (1.7 * g * (w / (w.sum(1, keepdim=True) + 1e-20) if renorm else w)).sum()
    for t in range(5):
        for e in range(9):
            h = torch.zeros((5, 9), dtype=torch.float64)
            h[t, e] = 1e-5
            diff = (value(z.double() + h) - value(z.double() - h)) / 2e-5
            assert abs(diff - dz[t, e]) < 1e-8
    assert (mag >= dz.abs() - 1e-12).all()


def test_mx_codes():
    x = torch.zeros((1, 32))
    x[0, :10] = torch.tensor([4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, -0.3, 7.9, 5.0])
    q, s = mx.quantize(x)
    assert s.shape == (1, 16) and s[0, 0] == 127 and s[0, 1:].sum() == 0
    v = mx.dequantize(q, s)
    # ties go to the even code; beyond 6 to 6
    assert v[0, :10].tolist() == [4.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, -0.5, 6.0, 4.0]
    assert (q[0, 0] & 15) == 6 and (q[0, 0] >> 4) == 0


def test_mx_scales():
    x = torch.zeros((1, 32 * 18))
    x[0, 0], x[0, 32], x[0, 64], x[0, 96], x[0, 128] = 8.0, 7.999, math.inf, math.nan, 2.0 ** -126
    q, s = mx.quantize(x)
    assert s.shape == (1, 32) and s[0, :5].tolist() == [128, 127, 255, 255, 0]
    v = mx.dequantize(q, s)
    assert v[0, 0] == 8 and v[0, 32] == 6 and torch.isnan(v[0, 64:128]).all() and v[0, 128] == 2.0 ** -126
    assert (v[0, 160:] == 0).all()


def test_flip_step_is_zero_away_from_borders():
    a = torch.full((1, 32), 4.0, dtype=torch.float64)
    a[0, 1], a[0, 2] = 1.25 + 1e-9, 1.3
    step = mx.flip_step(a + 0.3, torch.full_like(a, 1e-7))
    assert step.sum() == 0
    a[0, 0] = 5.5
    step = mx.flip_step(a, torch.full_like(a, 1e-7))
    assert step[0, 1] == 0.5 and step[0, 2] == 0


def test_mx_ffn_by_hand():
    """One activation of 100 in its block: 2^4 times 6.25, which rounds to 6, so 96; times 2."""
    x, w13, w2 = torch.zeros(1, 32).double(), torch.zeros(64, 32).double(), torch.zeros(32, 32).double()
    x[0, 0], w13[0, 0], w13[32, 0], w2[0, 0] = 2.0, 50.0, 0.5, 2.0
    y, bound = mx.ffn_rows(x, w13, w2)
    want = torch.zeros(1, 32).double()
    want[0, 0] = 192.0
    assert torch.equal(y, want)
    assert (bound[0, 1:] == 0).all() and 0 < bound[0, 0] < 1e-2
