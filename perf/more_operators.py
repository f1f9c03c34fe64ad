"""What stands around the routed experts of a layer, and experts with 16-bit weights: cases, plain forms and calls.

Three operators:
  * "norm"     the root-mean-square norm that feeds a layer, with the residual's addition:
               r = x + residual (in the residual's type), out = r / rms(r) * weight, in 16 bits
               and, for a layer that takes MXFP8 activations, as E4M3 codes with an E8M0 scale
               for every 32 values; "train" cases also take the gradients of r and of the weight;
  * "experts"  the routed experts with 16-bit weights, as products grouped by expert: row r of
               expert e gets (act(x Wg[e]^T) * (x Wu[e]^T)) W2[e]^T with x the row's token; "train"
               cases also take the gradients of x, W1 and W2;
  * "router"   the way back from the layer's sum through the weighted combine and the top-k
               softmax: gradients of the experts' rows, of the k weights and of the logits.

`own` chooses between elementary torch operations in 32 bits and the library's kernels.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------ cases

def _norm(name, T, H, dtype="bf16", x="bf16", residual="bf16", mxfp8=False, train=False):
    return dict(name=name, op="norm", T=T, H=H, dtype=dtype, x=x, residual=residual, mxfp8=mxfp8, train=train)


def _experts(name, T, H, I, E, k, dtype="bf16", layout="split", act="silu", skew=False, train=False):
    return dict(name=name, op="experts", T=T, H=H, I=I, E=E, k=k, dtype=dtype, layout=layout, act=act, skew=skew,
                train=train)


def _router(name, T, H, E, k, y="bf16", dy="bf16"):
    return dict(name=name, op="router", T=T, H=H, E=E, k=k, y=y, dy=dy)


def listed():
    return [
        # one sequence generating: the norm before the 256-expert layer
        _norm("norm_decode_1", 1, 4096),
        # a chunk of a prompt, rows that no tile divides
        _norm("norm_chunk_odd", 1357, 2216, dtype="fp16", x="fp16", residual="fp32"),
        # a long prompt into the 896-expert layer: takes the sum of the layer before it (fp32), gives
        # the router and the shared expert their 16-bit values and the experts their MXFP8 ones
        _norm("norm_prefill_mxfp8", 8192, 7168, x="fp32", mxfp8=True),
        # a training step: forward and backward before the 256-expert layer
        _norm("norm_train", 8192, 4096, train=True),
        # one sequence generating with the 256-expert layer's widths
        _experts("experts_decode_1", 1, 4096, 2048, 256, 6),
        # a decode batch: a bit more than half of the experts have tokens, one or two each
        _experts("experts_decode_32", 32, 4096, 2048, 256, 6, layout="interleaved"),
        # a chunk of a prompt through a small layer, sizes that no tile divides
        _experts("experts_chunk_odd", 333, 1096, 776, 24, 3, dtype="fp16", layout="interleaved", act="gelu"),
        # a prompt through the 256-expert layer: about a hundred tokens an expert
        _experts("experts_prefill", 4096, 4096, 2048, 256, 6),
        # a training step on a ragged batch of a small model, a few experts taking most of it
        _experts("experts_train_odd", 517, 1096, 776, 9, 2, dtype="fp16", layout="interleaved", act="gelu", skew=True,
                 train=True),
        # a training step: one GPU's 32 of the 256 experts, with the tokens that reach them
        _experts("experts_train", 8192, 4096, 2048, 32, 6, train=True),
        # the same small model's and the same large step's way back to the router
        _router("router_train_odd", 517, 1096, 9, 2, y="fp32", dy="fp16"),
        _router("router_train", 8192, 4096, 256, 6),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi, of=8):
    return max(of, _log(rng, lo, hi) // of * of)


def draw(rng):
    most = [work(c) for c in listed()]
    flops, size = max(w["flops"] for w in most), max(w["bytes"] for w in most)
    while True:
        dtype, op = rng.choice(["bf16", "fp16"]), rng.choice(["norm", "experts", "experts", "router"])
        T = _log(rng, 1, 8192)
        if op == "norm":
            train, mxfp8 = rng.random() < 0.4, rng.random() < 0.4
            c = _norm("", T, _width(rng, 512, 7168, 32 if mxfp8 else 8), dtype=dtype, x=rng.choice([dtype, "fp32"]),
                      residual=rng.choice(["none", dtype, "fp32"]), mxfp8=mxfp8 and not train, train=train)
        elif op == "experts":
            E = _log(rng, 4, 256)
            # few experts may take most of the tokens where there are few of them
            c = _experts("", T, _width(rng, 512, 7168), _width(rng, 256, 3584), E, rng.randint(1, min(8, E)),
                         dtype=dtype, layout=rng.choice(["split", "interleaved"]), act=rng.choice(["silu", "gelu"]),
                         skew=E <= 16 and rng.random() < 0.5, train=rng.random() < 0.4)
        else:
            E = _log(rng, 4, 896)
            c = _router("", T, _width(rng, 512, 7168), E, rng.randint(1, min(16, E)), y=rng.choice([dtype, "fp32"]),
                        dy=dtype)
        del c["name"]
        w = work(c)
        if w["flops"] <= flops and w["bytes"] <= size:
            return c


# ----------------------------------------------------------------- inputs

def _normal(shape, scale, dtype, gen):
    return torch.randn(shape, generator=gen, device=DEV, dtype=dtype).mul_(scale)


def _routing(case, gen):
    """ids [T][k], weights [T][k], and the stable permutation by expert: offsets [E+1], src [T*k] (the flat
    (token, slot) index behind each row), dest [T*k] (the row of each flat index)."""
    T, E, k = case["T"], case["E"], case["k"]
    logits = torch.randn((T, E), generator=gen, device=DEV) * 1.5
    if case.get("skew"):
        logits -= 1.1 * torch.log(torch.arange(1, E + 1, device=DEV, dtype=torch.float32)) * 1.5
    top, ids = torch.topk(logits, k, dim=1)
    flat = ids.reshape(-1)
    src = torch.argsort(flat, stable=True)
    dest = torch.empty_like(src)
    dest[src] = torch.arange(T * k, device=DEV)
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = torch.cumsum(counts, 0)
    i32 = torch.int32
    return dict(ids=ids.to(i32), w=torch.softmax(top, 1), src=src.to(i32), dest=dest.to(i32), offsets=offsets.to(i32))


def _inputs(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    T, H = case["T"], case["H"]
    if case["op"] == "norm":
        dt, f32 = DTYPES[case["dtype"]], torch.float32
        d = dict(x=_normal((T, H), 1.0, DTYPES[case["x"]], gen), residual=None,
                 weight=(1.0 + 0.2 * _normal((H,), 1.0, f32, gen)).to(dt))
        if case["residual"] != "none":
            # the residual's rows differ in size, as they do from layer to layer and token to token
            size = torch.exp2(2.0 * torch.rand((T, 1), generator=gen, device=DEV))
            d["residual"] = (_normal((T, H), 1.0, f32, gen) * size).to(DTYPES[case["residual"]])
        if case["train"]:
            d["dout"] = _normal((T, H), 1.0, dt, gen)
            d["dres"] = _normal((T, H), 1.0, dt, gen)
        return d
    d = _routing(case, gen)
    k, E = case["k"], case["E"]
    if case["op"] == "router":
        return dict(d, dout=_normal((T, H), 1.0, torch.float32, gen), y=_normal((T * k, H), 1.0, DTYPES[case["y"]], gen))
    dt, I = DTYPES[case["dtype"]], case["I"]
    d["x"] = _normal((T, H), 1.0, dt, gen)
    d["w1"], d["w2"] = _normal((E, 2 * I, H), H ** -0.5, dt, gen), _normal((E, H, I), I ** -0.5, dt, gen)
    if case["train"]:
        d["dout"] = _normal((T * k, H), 1.0, dt, gen)
    return d


def prepare(case, seed):
    d = _inputs(case, seed)
    d["case"] = case
    if case["op"] == "experts" and not own:
        # the plain form's batch: the experts that have rows, each with `most` places for them
        n = (d["offsets"][1:] - d["offsets"][:-1]).long()
        d["used"], d["most"] = torch.nonzero(n)[:, 0], int(n.max())
        owner = torch.repeat_interleave(torch.arange(len(d["used"]), device=DEV), n[d["used"]])
        first = d["offsets"][:-1].long()[d["used"]]
        d["place"] = owner * d["most"] + torch.arange(case["T"] * case["k"], device=DEV) - first[owner]
        d["owner"] = owner
    if own:
        import mxfp4_weight_mixture_amd as mx
        if case["op"] == "norm":
            d["call"] = mx.RMSNorm(d["weight"], eps=EPS)
        elif case["op"] == "experts":
            d["call"] = mx.ExpertFFN(d["w1"], d["w2"], layout=case["layout"], act=case["act"])
        else:
            d["call"] = mx
    return d


# -------------------------------------------------------------------- run

def run(d):
    c = d["case"]
    if not own:
        return {"norm": _plain_norm, "experts": _plain_experts, "router": _plain_router}[c["op"]](d, c)
    f = d["call"]
    if c["op"] == "norm":
        n = f.forward(d["x"], d["residual"], mxfp8=c["mxfp8"])
        r = {"out": n.out}
        if d["residual"] is not None:
            r["residual"] = n.residual
        if c["mxfp8"]:
            r["codes"], r["scales"] = n.codes.view(torch.float8_e4m3fn), n.scales.view(torch.float8_e8m0fnu)
        if c["train"]:
            r["dx"], r["dweight"] = f.backward(d["dout"], n.residual if d["residual"] is not None else d["x"],
                                               dresidual=d["dres"])
        return r
    if c["op"] == "experts":
        rows = dict(gather=d["src"], gather_div=c["k"])
        if not c["train"]:
            return f.forward(d["x"], d["offsets"], **rows)
        out, gate_up = f.forward(d["x"], d["offsets"], save=True, **rows)
        dx, dw1, dw2 = f.backward(d["dout"], d["x"], d["offsets"], gate_up, dest_row=d["dest"], **rows)
        return {"out": out, "dx": dx, "dw1": dw1, "dw2": dw2}
    dy, dw = f.combine_backward(d["dout"], d["y"], d["dest"], d["w"], dy_dtype=DTYPES[c["dy"]])
    return {"dy": dy, "dw": dw, "dlogits": f.route_backward(dw, d["ids"], d["w"], c["E"])}


def _plain_norm(d, c):
    dt = DTYPES[c["dtype"]]
    x, w = d["x"].float(), d["weight"].float()
    r = {}
    if d["residual"] is not None:
        r["residual"] = (x + d["residual"].float()).to(d["residual"].dtype)
        x = r["residual"].float()
    inv = 1.0 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
    unit = x * inv
    y = unit * w
    r["out"] = y.to(dt)
    if c["mxfp8"]:
        # the smallest power of two that brings a block to 448 or below, then the nearest E4M3 number
        b = y.view(c["T"], c["H"] // 32, 32)
        top = b.abs().amax(2, keepdim=True)
        e = torch.ceil(torch.log2(top.double() / 448.0)).clamp(-127, 127)
        e = torch.where(top > 0, e, torch.full_like(e, -127.0))
        r["codes"] = (b * torch.exp2(-e).float()).view(c["T"], c["H"]).to(torch.float8_e4m3fn)
        r["scales"] = (e[:, :, 0] + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    if c["train"]:
        dout = d["dout"].float()
        g = dout * w
        r["dx"] = (inv * (g - unit * (g * unit).mean(1, keepdim=True)) + d["dres"].float()).to(dt)
        r["dweight"] = (dout * unit).sum(0).to(dt)
    return r


_C = math.sqrt(2.0 / math.pi)


def _act(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    t = torch.tanh(_C * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * _C * (1.0 + 3 * 0.044715 * g * g)


def _plain_experts(d, c):
    """Batched products over the experts that have rows; an expert's rows are columns here."""
    dt, I = d["x"].dtype, c["I"]
    n, most = len(d["used"]), d["most"]
    w1, w2 = d["w1"][d["used"]].float(), d["w2"][d["used"]].float()

    def batch(rows):
        b = torch.zeros((n * most, rows.shape[1]), device=DEV)
        b[d["place"]] = rows
        return b.view(n, most, -1)

    def turned(b):
        return b.transpose(1, 2).contiguous()

    def rows(b):
        return turned(b).view(n * most, -1)[d["place"]]

    x = batch(d["x"][d["src"].long() // c["k"]].float())
    gu = torch.bmm(w1, turned(x))
    g, u = (gu[:, :I], gu[:, I:]) if c["layout"] == "split" else (gu[:, 0::2], gu[:, 1::2])
    a, da = _act(g, c["act"])
    h = a * u
    out = rows(torch.bmm(w2, h)).to(dt)
    if not c["train"]:
        return out
    dout = batch(d["dout"].float())
    dh = torch.bmm(w2.transpose(1, 2), turned(dout))
    dg, du = dh * u * da, dh * a
    dgu = torch.cat([dg, du], 1) if c["layout"] == "split" else torch.stack([dg, du], 2).flatten(1, 2)
    dx = rows(torch.bmm(w1.transpose(1, 2), dgu))[d["dest"].long()].view(c["T"], c["k"], -1).sum(1)
    dw1, dw2 = torch.zeros_like(d["w1"]), torch.zeros_like(d["w2"])
    dw1[d["used"]] = torch.bmm(dgu, x).to(dt)
    dw2[d["used"]] = torch.bmm(turned(dout), turned(h)).to(dt)
    return {"out": out, "dx": dx.to(dt), "dw1": dw1, "dw2": dw2}


def _plain_router(d, c):
    T, k = c["T"], c["k"]
    dest, w = d["dest"].long().view(T, k), d["w"]
    dout = d["dout"].view(T, 1, -1)
    dy = torch.empty_like(d["y"], dtype=DTYPES[c["dy"]])
    dy[dest] = (w.view(T, k, 1) * dout).to(dy.dtype)
    dw = (d["y"][dest].float() * dout).sum(2)
    dl = torch.zeros((T, c["E"]), device=DEV)
    dl.scatter_(1, d["ids"].long(), w * (dw - (w * dw).sum(1, keepdim=True)))
    return {"dy": dy, "dw": dw, "dlogits": dl}


# ------------------------------------------------------------------- work

_BYTES = {"none": 0, "bf16": 2, "fp16": 2, "fp32": 4}


def work(case):
    T, H = case["T"], case["H"]
    if case["op"] == "norm":
        per = _BYTES[case["x"]] + 2 * _BYTES[case["residual"]] + 2 + (1 + 1 / 32 if case["mxfp8"] else 0)
        if case["train"]:
            per += 2 + 2 + 2
        return {"bytes": T * H * per + 2 * H * (2 if case["train"] else 1), "flops": T * H * (16 if case["train"] else 6)}
    E, k = case["E"], case["k"]
    if case["op"] == "router":
        return {"bytes": T * H * (4 + k * (_BYTES[case["y"]] + _BYTES[case["dy"]])) + 4 * T * (E + 4 * k),
                "flops": 3 * T * k * H}
    I = case["I"]
    hit = E * (1.0 - (1.0 - k / E) ** T)   # experts with at least one row, as expected
    size, flops = T * H + T * k * H + 3 * hit * H * I, 6 * T * k * H * I
    if case["train"]:
        size, flops = size + T * k * H + T * H + 3 * E * H * I, 3 * flops
    return {"bytes": 2 * size + 4 * (E + 1 + 2 * T * k), "flops": flops}


# ------------------------------------------------------------------ exact

def _gate64(g, u, act):
    if act == "silu":
        return g * torch.sigmoid(g) * u
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))) * u


def _exact_norm(case, d):
    r = {}
    s = d["x"].double()
    if d["residual"] is not None:
        s = s + d["residual"].double()
        r["residual"] = s
        s = s.to(d["residual"].dtype).double()     # the sum is kept, and normed, in the residual's type
    s = s.requires_grad_(case["train"])
    w = d["weight"].double().requires_grad_(case["train"])
    y = w * s / torch.sqrt(s.square().sum(1, keepdim=True) / case["H"] + EPS)
    r["out"] = y.detach()
    if case["mxfp8"]:
        blocks = y.view(case["T"], -1, 32)
        _, e = torch.frexp(blocks.abs().amax(2) / 448.0)          # m 2^e with m in [1/2, 1)
        scale = torch.ldexp(torch.ones((), dtype=torch.float64, device=DEV), e)
        scale = torch.where(blocks.abs().amax(2) <= 224.0 * scale, scale / 2, scale)
        r["codes"], r["scales"] = (blocks / scale.unsqueeze(2)).view(case["T"], -1), scale
    if case["train"]:
        ds, r["dweight"] = torch.autograd.grad(y, (s, w), d["dout"].double())
        r["dx"] = ds + d["dres"].double()
    return r


def _exact_experts(case, d):
    """Expert after expert, differentiated automatically."""
    k, train = case["k"], case["train"]
    x = d["x"].double()
    out = torch.zeros((case["T"] * k, case["H"]), dtype=torch.float64, device=DEV)
    if train:
        dx = torch.zeros_like(x)
        dw1, dw2 = (torch.zeros(d[n].shape, dtype=torch.float64, device=DEV) for n in ("w1", "w2"))
    at, order = d["offsets"].tolist(), torch.arange(2 * case["I"], device=DEV)
    gate, up = (order[: case["I"]], order[case["I"]:]) if case["layout"] == "split" else (order[0::2], order[1::2])
    for e in range(case["E"]):
        if at[e] == at[e + 1]:
            continue
        rows = slice(at[e], at[e + 1])
        token = torch.div(d["src"][rows].long(), k, rounding_mode="floor")
        xe, w1, w2 = (t.clone().requires_grad_(train) for t in (x[token], d["w1"][e].double(), d["w2"][e].double()))
        y = torch.mm(_gate64(torch.mm(xe, w1[gate].t()), torch.mm(xe, w1[up].t()), case["act"]), w2.t())
        out[rows] = y.detach()
        if train:
            dxe, dw1[e], dw2[e] = torch.autograd.grad(y, (xe, w1, w2), d["dout"][rows].double())
            dx[token] += dxe      # an expert sees a token once
    return {"out": out, "dx": dx, "dw1": dw1, "dw2": dw2} if train else out


def _exact_router(case, d):
    """Slot after slot, the softmax's Jacobian written out."""
    T, k, y = case["T"], case["k"], d["y"]
    dout, w = d["dout"].double(), d["w"].double()
    dy = torch.zeros((T * k, case["H"]), dtype=torch.float64, device=DEV)
    dw = torch.zeros((T, k), dtype=torch.float64, device=DEV)
    for j in range(k):
        row = d["dest"].view(T, k)[:, j].long()
        dy[row] = w[:, j:j + 1] * dout
        dw[:, j] = torch.linalg.vecdot(y[row].double(), dout)
    jacobian = torch.diag_embed(w) - w.unsqueeze(2) * w.unsqueeze(1)
    kept = (jacobian * dw.unsqueeze(1)).sum(2)
    dl = torch.zeros((T, case["E"]), dtype=torch.float64, device=DEV)
    dl[torch.arange(T, device=DEV).unsqueeze(1), d["ids"].long()] = kept
    return {"dy": dy, "dw": dw, "dlogits": dl}


def exact(case, seed):
    d = _inputs(case, seed)
    return {"norm": _exact_norm, "experts": _exact_experts, "router": _exact_router}[case["op"]](case, d)
