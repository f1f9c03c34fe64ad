"""The new calls together, as a user has them.

Serving: the norm takes a layer's fp32 sum and the residual, gives the router and the shared expert 16-bit values and
the MXFP4 experts their MXFP8 activations.  Training: norm, route, permute, experts with 16-bit weights, combine, and
the whole way back, against automatic differentiation in float64 on the CPU."""
import numpy as np
import pytest
import torch

from oracle import moe as omoe
from tests import dense_util as du
from workloads import gen

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("mxfp4_weight_mixture_amd")
BF, HF, F = torch.bfloat16, torch.float16, torch.float32


def test_serving_norm_into_an_mxfp4_layer_with_a_shared_expert():
    s = gen.preset("tiny", act="mxfp8", layout="interleaved")
    li = gen.layer_inputs(s)
    H = s.H
    w = gen.all_expert_weights(s, 0, "cuda:0")
    shared = mx.GatedFFN(du.normal((2 * 64, H), H ** -0.5, BF, 1), du.normal((H, 64), 0.125, BF, 2))
    layer = mx.Layer(*w, k=s.k, layout="interleaved", shared=shared)
    plain = mx.Layer(*w, k=s.k, layout="interleaved")
    norm = mx.RMSNorm((1 + 0.1 * du.normal((H,), 1.0, F, 3)).to(BF))
    logits = torch.from_numpy(li.logits).to("cuda:0")
    total, residual = du.normal((s.T, H), 2.0, F, 4), du.normal((s.T, H), 1.0, BF, 5)
    for _ in range(2):                     # two layers: the second one's norm takes the first one's sum
        kept = (total + residual.float()).to(BF)
        n = norm.forward(total, residual, mxfp8=True)
        assert torch.equal(n.residual, kept)
        out = layer.forward(logits, n.codes, n.scales, x_shared=n.out)
        # the routed experts against the oracle on the very codes, the shared expert's part against its own call
        routed = plain.forward(logits, n.codes, n.scales)
        xa = omoe.activations(x_codes=n.codes.cpu().numpy(), x_scales=n.scales.cpu().numpy())
        ref = omoe.moe_layer(xa, li.logits, s.k, lambda e: [t.numpy() for t in gen.expert_weights(s, e)], "interleaved")
        assert np.abs(routed.cpu().numpy() - ref).max() <= 5e-2 * np.abs(ref).max()   # the layer's bound for MXFP8
        assert torch.equal(out, shared.forward(n.out, add=routed.clone()))
        total, residual = out, n.residual


def _weights(E, H, I, dtype, seed):
    return (du.normal((E, 2 * I, H), H ** -0.5, dtype, seed), du.normal((E, H, I), I ** -0.5, dtype, seed + 1),
            du.normal((E, H), H ** -0.5, dtype, seed + 2), (1 + 0.1 * du.normal((H,), 1.0, F, seed + 3)).to(dtype))


def _step(x, residual, dout, dres, w1, w2, wr, wn, k, layout, act, stream=None):
    """One layer forward and backward by the library's calls (the router's own matrix is the user's)."""
    E, dt = w1.shape[0], w1.dtype
    norm, experts = mx.RMSNorm(wn, eps=1e-5), mx.ExpertFFN(w1, w2, layout=layout, act=act)
    n = norm.forward(x, residual, stream=stream)
    logits = (n.out.float() @ wr.float().t()).contiguous()
    ids, w = mx.route(logits, k, stream=stream)
    off, src, dest = mx.permute(ids, E, stream=stream)
    rows = dict(gather=src, gather_div=k, stream=stream)
    y, gu = experts.forward(n.out, off, save=True, out_dtype=F if dt == HF else None, **rows)
    out = mx.combine(y, dest, w, stream=stream)
    dy, dw = mx.combine_backward(dout, y, dest, w, dy_dtype=dt, stream=stream)
    dlogits = mx.route_backward(dw, ids, w, E, stream=stream)
    dn, dw1, dw2 = experts.backward(dy, n.out, off, gu, dest_row=dest, dx=torch.empty(x.shape, device="cuda"), **rows)
    dn += dlogits @ wr.float()
    dwr = dlogits.t().contiguous() @ n.out.float()
    dx, dwn = norm.backward(dn, n.residual, dresidual=dres, dw_dtype=F, stream=stream)
    return dict(out=out, dx=dx, dwn=dwn, dwr=dwr, dw1=dw1, dw2=dw2), (ids, n.residual)


def _autograd(r, ids, dout, dres, w1, w2, wr, wn, layout, act):
    r, w1, w2, wr, wn = (t.detach().double().cpu().requires_grad_() for t in (r, w1, w2, wr, wn))
    ids, dout, dres = ids.long().cpu(), dout.double().cpu(), dres.double().cpu()
    n = wn * r / torch.sqrt(r.square().mean(1, keepdim=True) + 1e-5)
    w = torch.softmax(torch.gather(n @ wr.t(), 1, ids), 1)
    out = 0
    I = w2.shape[2]
    for j in range(ids.shape[1]):
        gu = torch.einsum("th,tih->ti", n, w1[ids[:, j]])
        g, u = (gu[:, :I], gu[:, I:]) if layout == "split" else (gu[:, 0::2], gu[:, 1::2])
        a = torch.nn.functional.silu(g) if act == "silu" else torch.nn.functional.gelu(g, approximate="tanh")
        out = out + w[:, j: j + 1] * torch.einsum("ti,thi->th", a * u, w2[ids[:, j]])
    ((out * dout).sum() + (r * dres).sum()).backward()
    return dict(out=out.detach(), dx=r.grad, dwn=wn.grad, dwr=wr.grad, dw1=w1.grad, dw2=w2.grad)


@pytest.mark.parametrize("T,E,k,H,I,dtype,layout,act", [(70, 9, 2, 136, 72, BF, "split", "silu"),
                                                        (33, 16, 4, 264, 40, HF, "interleaved", "gelu"),
                                                        (1, 8, 3, 64, 32, BF, "interleaved", "silu")])
def test_training_step_against_autograd(T, E, k, H, I, dtype, layout, act):
    w = _weights(E, H, I, dtype, 11)
    x, residual = du.normal((T, H), 1.0, F, 21), du.normal((T, H), 1.0, dtype, 22)
    dout, dres = du.normal((T, H), 1.0, F, 23), du.normal((T, H), 1.0, dtype, 24)
    got, (ids, r) = _step(x, residual, dout, dres, *w, k, layout, act)
    want = _autograd(r, ids, dout, dres, *w, layout, act)
    # 2-norms: at most eight roundings to 16 bits stand between the inputs and any result (the normed row, h, y, dy,
    # the gates' gradients, the result; the others in fp32), each off by at most u of its own size, and what they
    # feed grows an error by no more than the values it multiplies: 8 u, doubled for the sums of gradients that
    # partly cancel (the softmax's, the norm's)
    for name, ref in want.items():
        err = (got[name].double().cpu() - ref).norm() / ref.norm()
        assert err <= 16 * du.u(dtype), (name, float(err))


def test_training_step_captured_and_replayed_beside_another():
    """Two steps of different sizes, captured; replays in turn with eager steps, on inputs that change."""
    runs = []
    for T in (20, 150):
        w = _weights(6, 136, 72, BF, T)
        x, residual = du.normal((T, 136), 1.0, F, 31), du.normal((T, 136), 1.0, BF, 32)
        dout, dres = du.normal((T, 136), 1.0, F, 33), du.normal((T, 136), 1.0, BF, 34)
        step = lambda a=(x, residual, dout, dres, *w): _step(*a, 2, "split", "silu")[0]
        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = step()
        runs.append((x, step, g, outs))
    for i in range(3):
        for x, step, g, outs in runs:
            x.copy_(du.normal(tuple(x.shape), 1.0, F, 100 * i + x.shape[0]))
            g.replay()
            eager = step()
            torch.cuda.synchronize()
            assert all(torch.equal(outs[n], eager[n]) for n in eager), i
