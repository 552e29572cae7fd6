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
