"""GPU: uses of the layer's training and adapter steps that are refused."""
import pytest
import torch

from tests.gpu_layer import log
from tests.test_gpu_layer_train import BF, build, make_adapters, step

pytestmark = pytest.mark.gpu


def test_adapters_refuse_weights_of_another_shape(moelb):
    """The shared expert's weights come as one expert's, with or without a leading dimension.  Any other shape of as
    many elements (a weight kept as [d, 2 inter]) was read in the wrong order without a word."""
    L, t = build("bf16", True)
    ad = make_adapters(L, 3, 8, 8, BF)
    want = step(L, t, shared_adapters=ad).out.clone()
    lead = step(L, dict(t, s13=t["s13"].unsqueeze(0), s2=t["s2"].unsqueeze(0)), shared_adapters=ad).out.clone()
    torch.cuda.synchronize()
    assert torch.equal(lead, want)
    strided = torch.stack([t["s13"], t["s13"]], 2)[..., 0]
    for bad in (dict(s13=t["s13"].t().contiguous()), dict(s2=t["s2"].t().contiguous()),
                dict(s13=t["s13"].reshape(2, -1, L.d)), dict(s2=t["s2"].reshape(-1)), dict(s13=strided)):
        log(f"[layer adapters] {[(n, tuple(v.shape)) for n, v in bad.items()]}")
        with pytest.raises(moelb.MoelbError):
            step(L, dict(t, **bad), shared_adapters=ad)
    torch.cuda.synchronize()
    assert torch.equal(step(L, t, shared_adapters=ad).out, want)


def test_backward_outside_of_the_steps_capture(moelb):
    """A captured step has not run when its capture ends: backward called eagerly after it would read what an earlier
    step left."""
    L, t = build("bf16", True)
    args = (t["dout"], t["h"], t["wc"], t["bc"], t["w13"], t["w2"], t["s13"], t["s2"])
    step(L, t, train=True)
    want = L.backward(*args).h.clone()
    step(L, dict(t, h=-t["h"]), train=True)  # what the buffers hold from here on
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(L, t, train=True)
    with pytest.raises(RuntimeError, match="captured"):
        L.backward(*args)
    # in the same graph, or a step that has run, it is answered
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(L, t, train=True)
        got = L.backward(*args)
    for _ in range(3):
        got.h.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got.h, want)
    step(L, t, train=True)
    assert torch.equal(L.backward(*args).h, want)


def test_missing_shared_weights_are_refused_first(moelb):
    """A layer with a shared expert, called without its weights: refused before anything is queued (it ended in an
    AttributeError half-way, with the layer's buffers overwritten)."""
    L, t = build("bf16", True)
    ad = make_adapters(L, 3, 8, 8, BF)
    args = (t["dout"], t["h"], t["wc"], t["bc"], t["w13"], t["w2"])
    step(L, t, train=True)
    want = L.backward(*args, t["s13"], t["s2"])
    torch.cuda.synchronize()
    held = {n: getattr(want, n).clone() for n in ("h", "w_cur", "w13", "w2")}
    with pytest.raises(ValueError, match="shared"):
        L.backward(-t["dout"], *args[1:])
    with pytest.raises(ValueError, match="shared"):
        L.backward(-t["dout"], *args[1:], t["s13"])
    torch.cuda.synchronize()
    assert all(torch.equal(getattr(want, n), v) for n, v in held.items())
    idx = L.idx.clone()
    for kw in (dict(train=True), dict(shared_adapters=ad)):
        for miss in (dict(s13=None), dict(s2=None)):
            with pytest.raises(ValueError, match="shared"):
                step(L, dict(t, h=-t["h"], **miss), **kw)
    torch.cuda.synchronize()
    assert torch.equal(L.idx, idx)
    # nothing was queued, so the training step is still the layer's last one
    assert torch.equal(L.backward(*args, t["s13"], t["s2"]).h, held["h"])
