"""GPU: a MoE layer's training step and its gradients through MoELayer, and the
shared expert with adapters, on small configurations.

The gradients are compared with float64 autograd over the layer's dense
definition, built from the step's own picks (the top-k choice has no
gradient).  Tolerance, before any run, on the norm of the difference over the
norm: each gradient is a chain of at most four roundings to the storage type
in a row (y or dx, dy, dz or a, the sum), each at most u = eps / 2 relative
and independent: 4 u for bf16; fp32 sums of up to a few thousand terms:
1e-5.  The forward's out is compared with the inference step's bit for bit
where both run the same products, else within 4 u.
"""
import pytest
import torch

from synth import workloads as W
from tests.gpu_layer import log

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def build(dtype, shared, T=192, d=136, E=12, k=3, inter=72, G=4, N=2, gather=True, seed=0, packed=False):
    from routed_expert_ffn_gate_amd.layer import MoELayer
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = BF if dtype == "bf16" else torch.float32
    n = lambda *s: torch.randn(s, generator=gen, device=dev)  # noqa: E731
    si = 88 if shared else 0
    L = MoELayer(T, d, E, k, inter, G, N, 1, dtype, shared_inter=si, gather_rows=gather, packed_weights=packed)
    t = dict(h_prev=n(T, d).to(dt), h=n(T, d).to(dt), wc=(n(E, d) / d ** 0.5).to(dt), wn=(n(E, d) / d ** 0.5).to(dt),
             bc=n(E) * 0.3, bn=n(E) * 0.3, w13=(n(E, 2 * inter, d) / d ** 0.5).to(dt),
             w2=(n(E, d, inter) / inter ** 0.5).to(dt), dout=n(T, d).to(dt),
             home=torch.arange(E, dtype=torch.int32, device=dev) // (E // G))
    t["s13"] = (n(2 * si, d) / d ** 0.5).to(dt) if shared else None
    t["s2"] = (n(d, si) / si ** 0.5).to(dt) if shared else None
    t["replica"] = torch.empty((G, N), dtype=torch.int32, device=dev)
    L.predict_plan(t["h_prev"], t["wc"], t["bc"], t["home"], t["replica"])
    return L, t


def step(L, t, **kw):
    return L.step(t["h"], t["wc"], t["bc"], t["wn"], t["bn"], t["home"], t["replica"], t["w13"], t["w2"], t["s13"],
                  t["s2"], **kw)


def dense_gradients(L, t, idx):
    """float64 autograd over out[t] = sum_j softmax(z)[idx] expert_idx(h) + shared(h)."""
    p = {n: t[n].double().requires_grad_() for n in ("h", "wc", "bc", "w13", "w2", "s13", "s2") if t[n] is not None}

    def block(x, w13, w2):
        g, u = (x @ w13.t()).chunk(2, dim=1)
        return (g * torch.sigmoid(g) * u) @ w2.t()
    probs = torch.softmax(p["h"] @ p["wc"].t() + p["bc"], 1)
    out = torch.zeros_like(p["h"])
    for e in range(L.E):
        weight = (probs[:, e] * (idx == e).sum(1)).unsqueeze(1)
        out = out + weight * block(p["h"], p["w13"][e], p["w2"][e])
    if "s13" in p:
        out = out + block(p["h"], p["s13"], p["s2"])
    (out * t["dout"].double()).sum().backward()
    return out.detach(), {n: v.grad for n, v in p.items()}


@pytest.mark.parametrize("gather", [True, False], ids=["gather", "rows"])
@pytest.mark.parametrize("shared", [False, True], ids=["routed", "shared"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_gradients(moelb, dtype, shared, gather):
    L, t = build(dtype, shared, gather=gather)
    log(f"[layer train] {dtype} shared={shared} gather={gather}")
    o = step(L, t, train=True)
    if not gather:
        # the copied rows: train reads x_perm, which the permutation wrote
        assert o.x_perm is not None
    out = o.out.clone()
    g = L.backward(t["dout"], t["h"], t["wc"], t["bc"], t["w13"], t["w2"], t["s13"], t["s2"])
    torch.cuda.synchronize()
    want_out, want = dense_gradients(L, t, o.idx)
    tol = 4 * torch.finfo(BF).eps / 2 if dtype == "bf16" else 1e-5
    pairs = [("out", out, want_out), ("h", g.h, want["h"]), ("wc", g.w_cur, want["wc"]), ("bc", g.b_cur, want["bc"]),
             ("w13", g.w13, want["w13"]), ("w2", g.w2, want["w2"])]
    if shared:
        pairs += [("s13", g.shared_w13, want["s13"]), ("s2", g.shared_w2, want["s2"])]
    for name, got, ref in pairs:
        rel = ((got.double() - ref).norm() / ref.norm()).item()
        log(f"    {name}: rel {rel:.2e} of {tol:.1e}")
        assert rel <= tol, name


def test_training_step_equals_inference(moelb):
    L, t = build("bf16", True)
    a = step(L, t).out.clone()
    b = step(L, t, train=True).out.clone()
    torch.cuda.synchronize()
    assert ((a.double() - b.double()).norm() / a.double().norm()).item() <= 4 * torch.finfo(BF).eps / 2


def test_steps_on_another_stream_and_twice(moelb):
    L, t = build("bf16", True)
    step(L, t, train=True)
    names = ("h", "w_cur", "b_cur", "w13", "w2", "shared_w13", "shared_w2")
    args = (t["dout"], t["h"], t["wc"], t["bc"], t["w13"], t["w2"], t["s13"], t["s2"])
    first = {n: getattr(L.backward(*args), n).clone() for n in names}
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    step(L, t, train=True, stream=st)
    again = L.backward(*args, stream=st)
    torch.cuda.synchronize()
    for n in names:
        assert torch.equal(getattr(again, n), first[n]), n


def make_adapters(L, n, r13, r2, dt, seed=1):
    from routed_expert_ffn_gate_amd.layer import SharedAdapters
    gen = torch.Generator(device="cuda").manual_seed(seed)
    N = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    si, d, T = L.shared_inter, L.d, L.T
    return SharedAdapters(torch.randint(-1, n, (T,), generator=gen, device="cuda").to(torch.int32),
                          (N(n, r13, d) / d ** 0.5).to(dt), (N(n, 2 * si, r13) / r13 ** 0.5).to(dt), 0.5 + N(n).abs(),
                          (N(n, r2, si) / si ** 0.5).to(dt), (N(n, d, r2) / r2 ** 0.5).to(dt), 0.5 + N(n).abs())


@pytest.mark.parametrize("dtype,T", [("bf16", 4), ("bf16", 48), ("bf16", 192), ("f32", 48)])
def test_shared_expert_with_adapters(moelb, dtype, T):
    L, t = build(dtype, True, T=T)
    dt = BF if dtype == "bf16" else torch.float32
    ad = make_adapters(L, 5, 16, 8, dt)
    bare = step(L, t)
    y = bare.shared.clone()
    got = step(L, t, shared_adapters=ad)
    torch.cuda.synchronize()
    D = lambda v: v.double()  # noqa: E731
    x = D(t["h"])

    def proj(x, w, a, b, s):
        y = x @ D(w).t()
        for v in range(5):
            rows = (ad.ids == v).nonzero()[:, 0]
            y[rows] += D(s)[v] * (x[rows] @ D(a[v]).t() @ D(b[v]).t())
        return y
    g, u = proj(x, t["s13"], ad.a13, ad.b13, ad.scale13).chunk(2, dim=1)
    want = proj(g * torch.sigmoid(g) * u, t["s2"], ad.a2, ad.b2, ad.scale2)
    rel = ((D(got.shared) - want).norm() / want.norm()).item()
    log(f"[layer adapters] {dtype} T={T}: rel {rel:.2e}")
    assert rel <= (4 * torch.finfo(BF).eps / 2 if dtype == "bf16" else 1e-5)
    # tokens without an adapter: the bare shared expert's rows, within its own rounding
    none = ad.ids < 0
    if bool(none.any()):
        d = ((D(got.shared[none]) - D(y[none])).norm() / D(y[none]).norm()).item()
        assert d <= (4 * torch.finfo(BF).eps / 2 if dtype == "bf16" else 1e-5)


def test_refusals(moelb):
    L, t = build("bf16", False)
    with pytest.raises(RuntimeError):
        L.backward(t["dout"], t["h"], t["wc"], t["bc"], t["w13"], t["w2"])
    with pytest.raises(ValueError):
        step(L, t, shared_adapters=object())   # no shared expert
    L, t = build("bf16", True)
    with pytest.raises(ValueError):
        step(L, t, shared_adapters=make_adapters(L, 2, 8, 8, BF), train=True)
    # the layer's buffers are another step's by now
    args = (t["dout"], t["h"], t["wc"], t["bc"], t["w13"], t["w2"], t["s13"], t["s2"])
    step(L, t, train=True)
    L.backward(*args)
    step(L, t)
    with pytest.raises(RuntimeError):
        L.backward(*args)
    step(L, t, train=True)
    L.predict_plan(t["h_prev"], t["wc"], t["bc"], t["home"], t["replica"])
    with pytest.raises(RuntimeError):
        L.backward(*args)
    L, t = build("bf16", True, d=128, inter=64, packed=True)
    with pytest.raises(ValueError):
        step(L, t, train=True)


def test_a_step_that_fails_keeps_nothing(moelb):
    L, t = build("bf16", True)
    args = (t["dout"], t["h"], t["wc"], t["bc"], t["w13"], t["w2"], t["s13"], t["s2"])
    step(L, t, train=True)
    L.backward(*args)
    with pytest.raises(moelb.MoelbError):  # after the gate wrote this step's picks
        step(L, dict(t, w13=t["w13"][:, 1:]), train=True)
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError):
        L.backward(*args)
    step(L, t, train=True)
    L.backward(*args)


def test_captured_adapters_keep_their_workspace(moelb):
    """A larger rank makes a larger workspace; the one a captured graph writes to stays the layer's."""
    L, t = build("bf16", True)
    small, large = make_adapters(L, 3, 8, 8, BF), make_adapters(L, 3, 256, 256, BF)
    want = step(L, t, shared_adapters=small).out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(L, t, shared_adapters=small)
    held = L._adapter_ws[-1].numel()
    large_out = step(L, t, shared_adapters=large).out.clone()
    assert L._adapter_ws[-1].numel() > held
    canaries = [torch.full((held,), 7, dtype=torch.uint8, device="cuda") for _ in range(8)]
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(L.out, want)
        assert all(bool((c == 7).all()) for c in canaries)
        assert torch.equal(step(L, t, shared_adapters=large).out, large_out)


def test_first_steps_buffers(moelb):
    """The buffers that the first step of a kind makes: refused under capture (nothing is queued), and usable at once
    on a stream that does not wait for the one they were made on."""
    L, t = build("bf16", True)
    ad = make_adapters(L, 3, 8, 8, BF)
    args = (t["dout"], t["h"], t["wc"], t["bc"], t["w13"], t["w2"], t["s13"], t["s2"])
    torch.cuda.synchronize()
    for kw in (dict(train=True), dict(shared_adapters=ad)):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            with pytest.raises(RuntimeError, match="before capturing"):
                step(L, t, **kw)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    busy = torch.randn((4096, 4096), device="cuda")
    for _ in range(4):
        busy = busy @ busy * 1e-2  # the current stream has work queued
    step(L, t, train=True, stream=st)
    got = L.backward(*args, stream=st)
    st.synchronize()
    first = [getattr(got, n).clone() for n in ("h", "w_cur", "b_cur", "w13", "w2", "shared_w13", "shared_w2")]
    torch.cuda.synchronize()
    step(L, t, train=True)
    again = L.backward(*args)
    torch.cuda.synchronize()
    for a, n in zip(first, ("h", "w_cur", "b_cur", "w13", "w2", "shared_w13", "shared_w2")):
        assert torch.equal(a, getattr(again, n)), n


def test_captured_training_step(moelb):
    """step and backward in one graph, replayed between eager steps of other inputs."""
    L, t = build("bf16", True)
    names = ("h", "w_cur", "b_cur", "w13", "w2", "shared_w13", "shared_w2")
    args = (t["dout"], t["h"], t["wc"], t["bc"], t["w13"], t["w2"], t["s13"], t["s2"])
    step(L, t, train=True)
    want = {n: getattr(L.backward(*args), n).clone() for n in names}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(L, t, train=True)
        got = L.backward(*args)
    other = dict(t, h=-t["h"], dout=t["dout"] * 2)
    for _ in range(3):
        step(L, other, train=True)
        L.backward(other["dout"], other["h"], *args[2:])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in names:
            assert torch.equal(getattr(got, n), want[n]), n


def test_full_shape_step(moelb):
    """Qwen3-30B's decode shape (T = 512, d = 2048, E = 128, k = 8, inter = 768) as one training step: random
    routing, every gradient finite and the router's bias gradient summing to zero (a softmax has no gradient along
    a shift of all its logits: the sum of dz over the experts is 0 up to E T 2^-24 of the magnitudes)."""
    cfg = W.config("c2_qwen3_30b_decode")
    L, t = build("bf16", False, T=cfg.T, d=cfg.d, E=cfg.E, k=cfg.k, inter=cfg.inter, G=cfg.G, N=cfg.N)
    step(L, t, train=True)
    g = L.backward(t["dout"], t["h"], t["wc"], t["bc"], t["w13"], t["w2"])
    torch.cuda.synchronize()
    for n in ("h", "w_cur", "b_cur", "w13", "w2"):
        assert bool(torch.isfinite(getattr(g, n)).all()), n
    assert abs(g.b_cur.double().sum().item()) <= 1e-4 * g.b_cur.double().abs().sum().item()
