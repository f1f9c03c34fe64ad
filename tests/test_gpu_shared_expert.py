"""The operators together, as a model's layer uses them: routed MXFP4 experts, the 16-bit shared expert beside
them, and adapters of many requests on top, against the float64 oracles."""
import numpy as np
import pytest
import torch

from oracle import dense as od
from tests import dense_util as du
from tests.gpu_util import device_weights, device_x, oracle_layer, rel_err, x_as_f64
from workloads import gen

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("mxfp4_weight_mixture_amd")
BF, F = torch.bfloat16, torch.float32


def _layer(T, act, seed, H=256, I=128, Is=192):
    s = gen.LayerShape(T=T, H=H, I=I, E=8, k=2, act=act, layout="split", cfg_id=seed)
    li = gen.layer_inputs(s)
    w1, w2 = du.normal((2 * Is, H), H ** -0.5, BF, seed), du.normal((H, Is), Is ** -0.5, BF, seed + 1)
    ffn = mx.GatedFFN(w1, w2, layout="interleaved")
    return s, li, ffn, mx.Layer(*device_weights(s), k=2, layout="split", shared=ffn)


@pytest.mark.parametrize("T,act", [(1, "bf16"), (24, "mxfp8"), (90, "bf16"), (300, "mxfp8")])
def test_layer_with_a_shared_expert(T, act):
    s, li, ffn, layer = _layer(T, act, 230 + T)
    logits = torch.from_numpy(li.logits).to("cuda")
    x, xs = device_x(li)
    xv = x if xs is None else torch.from_numpy(x_as_f64(li)).to(BF).to("cuda")
    out = layer.forward(logits, x, xs, x_shared=None if xs is None else xv)
    routed = mx.Layer(layer.w1p, layer.w1s, layer.w2p, layer.w2s, k=2, layout="split").forward(logits, x, xs)
    # the routed part is the layer's without a shared expert; the shared part is within its bounds of the oracle
    ref, bound, *_ = du.ffn_bounds(du.f64(xv), du.f64(ffn.w1), du.f64(ffn.w2), "interleaved", "silu", BF, F,
                                   add=du.f64(routed))
    du.assert_within(out, ref, bound, "out")
    whole, _ = oracle_layer(s, li)
    shared = od.gated_ffn(du.f64(xv), du.f64(ffn.w1), du.f64(ffn.w2), "interleaved")[0]
    # the layer's own acceptance bounds
    assert rel_err(out.cpu().numpy(), whole + shared) <= (2e-2 if act == "bf16" else 5e-2)


def test_captured_layer_with_a_shared_expert():
    s, li, ffn, layer = _layer(16, "bf16", 250)
    logits, x = torch.from_numpy(li.logits).to("cuda"), li.x_bf16.to("cuda")
    g = layer.capture(logits, x)
    for k in range(3):
        x.copy_(du.normal(tuple(x.shape), 1.0, BF, 900 + k))
        got = g.replay().clone()
        eager = layer.forward(logits, x)
        torch.cuda.synchronize()
        assert torch.equal(got, eager)
    g.close()


def test_shared_expert_refusals():
    s, li, ffn, layer = _layer(8, "mxfp8", 260)
    logits = torch.from_numpy(li.logits).to("cuda")
    x, xs = device_x(li)
    with pytest.raises(ValueError, match="x_shared"):
        layer.forward(logits, x, xs)
    bf = torch.zeros(8, s.H, dtype=BF, device="cuda")
    with pytest.raises(ValueError, match="x_next"):
        layer.forward(logits, x, xs, x_shared=bf, x_next=torch.empty_like(bf))
    with pytest.raises(ValueError, match="shape"):
        layer.forward(logits, x, xs, x_shared=bf[:4])
    plain = mx.Layer(layer.w1p, layer.w1s, layer.w2p, layer.w2s, k=2, layout="split")
    with pytest.raises(ValueError, match="without a shared expert"):
        plain.forward(logits, x, xs, x_shared=bf)
    with pytest.raises(ValueError, match="width"):
        mx.Layer(layer.w1p, layer.w1s, layer.w2p, layer.w2s, k=2, layout="split",
                 shared=mx.GatedFFN(torch.zeros(64, 128, dtype=BF, device="cuda"),
                                    torch.zeros(128, 32, dtype=BF, device="cuda")))


@pytest.mark.parametrize("T", [1, 40, 260])
def test_shared_expert_with_adapters_beside_routed_experts(T):
    """Both projections of the shared expert with each request's adapters, added to the routed experts' sum."""
    s, li, ffn, layer = _layer(T, "bf16", 270 + T)
    n, R, H, Is = 5, 16, s.H, ffn.I
    logits, x = torch.from_numpy(li.logits).to("cuda"), li.x_bf16.to("cuda")
    ids = torch.randint(-1, n, (T,), generator=torch.Generator().manual_seed(T)).int().to("cuda")
    mk = lambda *sh, sd: du.normal(sh, sh[-1] ** -0.5, BF, sd)
    up = mx.AdapterLinear(ffn.w1, mk(n, R, H, sd=1), mk(n, 2 * Is, R, sd=2), epilogue="interleaved")
    down = mx.AdapterLinear(ffn.w2, mk(n, R, Is, sd=3), mk(n, H, R, sd=4))
    routed = mx.Layer(layer.w1p, layer.w1s, layer.w2p, layer.w2s, k=2, layout="split").forward(logits, x)
    base = routed.clone()
    h = up.forward(x, ids)
    out = down.forward(h, ids, add=routed, out=routed)
    host = ids.cpu().numpy()
    ref_h, bound_h = du.adapter_bounds(du.f64(x), du.f64(ffn.w1), host, du.f64(up.lora_a), du.f64(up.lora_b), BF, BF,
                                       epilogue="interleaved")
    du.assert_within(h, ref_h, bound_h, "h")
    ref, bound = du.adapter_bounds(du.f64(h), du.f64(ffn.w2), host, du.f64(down.lora_a), du.f64(down.lora_b), BF, F,
                                   add=du.f64(base))
    du.assert_within(out, ref, bound, "out")


def test_adapters_on_a_quantised_projection():
    """The adapters' part added to what the MXFP4 grouped GEMM gave (one expert: a plain projection)."""
    T, K, N, n, R = 70, 256, 192, 4, 8
    s = gen.LayerShape(T=T, H=K, I=96, E=1, k=1, act="bf16", layout="split", cfg_id=290)
    w1p, w1s, _, _ = device_weights(s)
    x = gen.layer_inputs(s).x_bf16.to("cuda")
    y = mx.grouped_gemm(x, w1p, w1s, torch.tensor([0, T], dtype=torch.int32, device="cuda"))
    ids = (torch.arange(T, device="cuda") % (n + 1) - 1).int()
    f = mx.AdapterLinear(None, du.normal((n, R, K), K ** -0.5, BF, 5), du.normal((n, N, R), R ** -0.5, BF, 6))
    out = f.forward(x, ids, add=y)
    ref, bound = du.adapter_bounds(du.f64(x), None, ids.cpu().numpy(), du.f64(f.lora_a), du.f64(f.lora_b), BF, BF,
                                   add=du.f64(y))
    du.assert_within(out, ref, bound)


def test_two_streams_at_once():
    """Calls in flight on two streams share nothing: forward, backward and adapters of several sizes."""
    H, I, n = 520, 264, 4
    work = []
    for k, T in enumerate((3, 50, 130, 700)):
        f = mx.GatedFFN(du.normal((2 * I, H), H ** -0.5, BF, k), du.normal((H, I), I ** -0.5, BF, k + 9))
        lin = mx.AdapterLinear(f.w1, du.normal((n, 16, H), H ** -0.5, BF, k), du.normal((n, 2 * I, 16), 0.25, BF, k))
        x, dout = du.normal((T, H), 1.0, BF, k), du.normal((T, H), 1.0, BF, k + 5)
        ids = (torch.arange(T, device="cuda") * n // T).int()
        work.append((f, lin, x, dout, ids))

    def step(item, stream=None):
        f, lin, x, dout, ids = item
        out, gu = f.forward(x, save=True, stream=stream)
        return (out,) + tuple(f.backward(dout, x, gu, stream=stream)) + (lin.forward(x, ids, stream=stream),)

    want = [step(w) for w in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [step(w, streams[(i + j) % 2]) for j in range(2) for i, w in enumerate(work)]
        torch.cuda.synchronize()
        for i, g in enumerate(got):
            assert all(torch.equal(a, b) for a, b in zip(g, want[i % len(work)])), i
