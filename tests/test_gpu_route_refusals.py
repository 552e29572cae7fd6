"""GPU: a step that MoELayer refuses over its router's bias or its weights' format leaves every buffer as it was."""
import pytest
import torch

from tests.test_gpu_layer_router_mx import build, step

pytestmark = pytest.mark.gpu
BUFFERS = ("idx", "wts", "gap", "idx_next", "counts", "counts_next", "host_count", "load", "group_off", "perm", "pos", "y",
           "shared", "out")


def test_refused_steps_write_nothing(moelb):
    from routed_expert_ffn_gate_amd.layer import SharedAdapters
    L, t = build(use_mx=True)
    plain, tp = build()
    torch.cuda.synchronize()
    for layer in (L, plain):
        for n in BUFFERS:
            getattr(layer, n).fill_(113)
    bias = torch.zeros(12, device="cuda")
    calls = [lambda: step(L, t, train=True), lambda: step(L, t, shared_adapters=SharedAdapters(*[None] * 7)),
             lambda: step(L, {**t, "w2": tp["w2"]}), lambda: step(L, {**t, "bias": bias}),
             lambda: plain.predict_plan(tp["h_prev"], tp["wc"], tp["bc"], tp["home"], tp["replica"], route_bias=bias)]
    for call in ("step", "step_two_stage"):
        calls += [lambda call=call: step(plain, {**tp, "s13": t["s13"]}, call),
                  lambda call=call: step(plain, {**tp, "bias": bias}, call),
                  lambda call=call: step(plain, {**tp, "bias_next": bias}, call),
                  lambda call=call: step(L, {**t, "w13": tp["w13"]}, call)]
    for call in calls:
        with pytest.raises(ValueError):
            call()
    torch.cuda.synchronize()
    for layer in (L, plain):
        for n in BUFFERS:
            assert (getattr(layer, n) == 113).all(), n
