"""The dense operators beside the routed experts: cases, plain forms and calls.

Two operators:
  * "ffn"      the gated feed-forward block with 16-bit weights (the shared expert of a MoE
               layer): out = (act(x Wg^T) * (x Wu^T)) W2^T; "train" cases also take the
               gradients of x, W1 and W2;
  * "adapter"  a projection shared by all tokens plus each token's own low-rank adapter:
               out[t] = x[t] W^T + scale[a] (x[t] A[a]^T) B[a]^T with a = ids[t] (none if
               negative), optionally with the gated epilogue on the sum, or without W and added
               to given values.

`own` chooses between elementary torch operations in 32 bits and the library's kernels.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
DEV = "cuda"


# ------------------------------------------------------------------ cases

def _ffn(name, T, H, I, dtype="bf16", layout="split", act="silu", train=False):
    return dict(name=name, op="ffn", T=T, H=H, I=I, dtype=dtype, layout=layout, act=act, train=train)


def _adapter(name, T, K, N, n, R, ids, dtype="bf16", epilogue="none", act="silu", base=True, ranks=False):
    return dict(name=name, op="adapter", T=T, K=K, N=N, n=n, R=R, ids=ids, dtype=dtype, epilogue=epilogue,
                act=act, base=base, ranks=ranks)


def listed():
    return [
        # one sequence generating: a shared expert of the 256-expert layer's widths
        _ffn("ffn_decode_1", 1, 4096, 2048),
        # a decode batch: a shared expert of the 896-expert layer's widths
        _ffn("ffn_decode_32", 32, 7168, 3584, layout="interleaved"),
        # a chunk of a prompt, sizes that no tile divides
        _ffn("ffn_chunk_odd", 333, 2216, 1000, dtype="fp16", act="gelu"),
        # a long prompt through the 896-expert layer's shared expert
        _ffn("ffn_prefill", 8192, 7168, 3584),
        # a training step on a ragged batch of a small model
        _ffn("ffn_train_odd", 517, 1096, 776, dtype="fp16", layout="interleaved", act="gelu", train=True),
        # a training step: one micro-batch through the 256-expert layer's shared expert
        _ffn("ffn_train", 8192, 4096, 2048, train=True),
        # one sequence generating with its adapter
        _adapter("adapter_decode_1", 1, 4096, 4096, n=8, R=16, ids="each"),
        # a decode batch, each request with an adapter of its own choice, some with none
        _adapter("adapter_decode_32", 32, 7168, 7168, n=16, R=32, ids="each"),
        # a wide decode batch of many tenants through gate and up; adapters of several ranks
        _adapter("adapter_decode_192", 192, 4096, 4096, n=48, R=16, ids="each", epilogue="split", ranks=True),
        # prompts of several requests in one ragged batch
        _adapter("adapter_chunk_odd", 1357, 2216, 1544, n=7, R=64, ids="runs", dtype="fp16", ranks=True),
        # long prompts through gate and up of the 896-expert layer's shared expert
        _adapter("adapter_prefill", 8192, 7168, 7168, n=12, R=16, ids="runs", epilogue="interleaved"),
        # the adapters' part alone, added to what a projection with quantised weights gave
        _adapter("adapter_add", 4096, 2048, 4096, n=9, R=32, ids="runs", base=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    return max(8, _log(rng, lo, hi) // 8 * 8)


def draw(rng):
    most = work(_ffn("", 8192, 7168, 3584))["flops"]
    while True:
        dtype, act = rng.choice(["bf16", "fp16"]), rng.choice(["silu", "gelu"])
        T = _log(rng, 1, 8192)
        if rng.random() < 0.5:
            c = _ffn("", T, _width(rng, 512, 7168), _width(rng, 256, 3584), dtype=dtype,
                     layout=rng.choice(["split", "interleaved"]), act=act, train=rng.random() < 0.4)
        else:
            base = rng.random() < 0.8
            K, N = _width(rng, 512, 7168), _width(rng, 512, 7168)
            c = _adapter("", T, K, N, n=_log(rng, 1, 64), R=8 * rng.randint(1, 8), dtype=dtype, act=act,
                         ids="each" if T <= 256 else "runs", base=base, ranks=rng.random() < 0.5,
                         epilogue=rng.choice(["none", "split", "interleaved"]) if base else "none")
        del c["name"]
        if work(c)["flops"] <= most:
            return c


# ----------------------------------------------------------------- inputs

def _normal(shape, scale, dtype, gen):
    return (torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32) * scale).to(dtype)


def _inputs(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt, T = DTYPES[case["dtype"]], case["T"]
    if case["op"] == "ffn":
        H, I = case["H"], case["I"]
        d = dict(x=_normal((T, H), 1.0, dt, gen), w1=_normal((2 * I, H), H ** -0.5, dt, gen),
                 w2=_normal((H, I), I ** -0.5, dt, gen))
        if case["train"]:
            d["dout"] = _normal((T, H), 1.0, dt, gen)
        return d
    K, N, n, R = case["K"], case["N"], case["n"], case["R"]
    cpu = torch.Generator().manual_seed(seed)
    # every adapter has a request where there are enough; about one request in eight has none
    if case["ids"] == "each":
        ids = torch.randperm(max(T, n), generator=cpu)[:T] % n
        if T > 8:
            ids[torch.randperm(T, generator=cpu)[: T // 8]] = -1
    else:
        requests = n + max(1, n // 8)
        cuts = torch.sort(torch.randperm(max(T - 1, 1), generator=cpu)[: requests - 1] + 1).values
        owner = torch.randperm(requests, generator=cpu)
        ids = owner[torch.bucketize(torch.arange(T), cuts, right=True)]
        ids[ids >= n] = -1
    d = dict(x=_normal((T, K), 1.0, dt, gen), ids=ids.to(torch.int32).to(DEV),
             a=_normal((n, R, K), K ** -0.5, dt, gen), b=_normal((n, N, R), R ** -0.5, dt, gen),
             scales=torch.rand(n, generator=gen, device=DEV) + 0.5)
    d["w"] = _normal((N, K), K ** -0.5, dt, gen) if case["base"] else None
    d["add"] = None if case["base"] else _normal((T, N), 1.0, dt, gen)
    d["ranks"] = None
    if case["ranks"]:
        d["ranks"] = torch.randint(1, R + 1, (n,), generator=cpu).to(torch.int32).to(DEV)
    return d


def prepare(case, seed):
    d = _inputs(case, seed)
    d["case"] = case
    if own:
        import mxfp4_weight_mixture_amd as mx
        if case["op"] == "ffn":
            d["call"] = mx.GatedFFN(d["w1"], d["w2"], layout=case["layout"], act=case["act"])
        else:
            d["call"] = mx.AdapterLinear(d["w"], d["a"], d["b"], scales=d["scales"], ranks=d["ranks"],
                                         epilogue=case["epilogue"], act=case["act"])
    return d


# -------------------------------------------------------------------- run

def run(d):
    c = d["case"]
    if own:
        f = d["call"]
        if c["op"] == "adapter":
            return f.forward(d["x"], d["ids"], add=d["add"])
        if not c["train"]:
            return f.forward(d["x"])
        out, gate_up = f.forward(d["x"], save=True)
        dx, dw1, dw2 = f.backward(d["dout"], d["x"], gate_up)
        return {"out": out, "dx": dx, "dw1": dw1, "dw2": dw2}
    return _plain_ffn(d, c) if c["op"] == "ffn" else _plain_adapter(d, c)


_C = math.sqrt(2.0 / math.pi)


def _act(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    t = torch.tanh(_C * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * _C * (1.0 + 3 * 0.044715 * g * g)


def _halves(gu, layout):
    n = gu.shape[1] // 2
    return (gu[:, :n], gu[:, n:]) if layout == "split" else (gu[:, 0::2], gu[:, 1::2])


def _plain_ffn(d, c):
    dt = d["x"].dtype
    x, w1, w2 = d["x"].float(), d["w1"].float(), d["w2"].float()
    g, u = _halves(x @ w1.T, c["layout"])
    a, da = _act(g, c["act"])
    h = a * u
    out = (h @ w2.T).to(dt)
    if not c["train"]:
        return out
    dout = d["dout"].float()
    dh = dout @ w2
    dg, du = dh * u * da, dh * a
    dgu = torch.cat([dg, du], 1) if c["layout"] == "split" else torch.stack([dg, du], 2).flatten(1)
    return {"out": out, "dx": (dgu @ w1).to(dt), "dw1": (dgu.T @ x).to(dt), "dw2": (dout.T @ h).to(dt)}


def _plain_adapter(d, c):
    dt, T, n, R = d["x"].dtype, c["T"], c["n"], c["R"]
    x = d["x"].float()
    # every adapter's first product in one matrix, then each token keeps its own adapter's block
    s = (x @ d["a"].float().reshape(n * R, -1).T).view(T, n, R) * d["scales"].view(1, n, 1)
    keep = (d["ids"].view(T, 1, 1) == torch.arange(n, device=x.device).view(1, n, 1))
    if d["ranks"] is not None:
        keep = keep & (torch.arange(R, device=x.device).view(1, 1, R) < d["ranks"].view(1, n, 1))
    s = torch.where(keep, s, torch.zeros((), device=x.device))
    y = s.reshape(T, n * R) @ d["b"].float().transpose(1, 2).reshape(n * R, -1)
    if d["w"] is not None:
        y = y + x @ d["w"].float().T
    if d["add"] is not None:
        y = y + d["add"].float()
    if c["epilogue"] != "none":
        g, u = _halves(y, c["epilogue"])
        y = _act(g, c["act"])[0] * u
    return y.to(dt)


# ------------------------------------------------------------------- work

def work(case):
    T = case["T"]
    if case["op"] == "ffn":
        H, I = case["H"], case["I"]
        size, flops = 2 * T * H + 3 * H * I, 6 * T * H * I
        if case["train"]:
            size, flops = size + 2 * T * H + 3 * H * I, 3 * flops
        return {"bytes": 2 * size, "flops": flops}
    K, N, n, R = case["K"], case["N"], case["n"], case["R"]
    n_out = N if case["epilogue"] == "none" else N // 2
    size = T * K + T * n_out + min(n, T) * R * (K + N) + (N * K if case["base"] else T * N)
    return {"bytes": 2 * size + 4 * T, "flops": 2 * T * R * (K + N) + (2 * T * N * K if case["base"] else 0)}


# ------------------------------------------------------------------ exact

def _gate64(g, u, act):
    if act == "silu":
        return g * torch.sigmoid(g) * u
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))) * u


def exact(case, seed):
    d = _inputs(case, seed)
    wide = {k: v.double() if v is not None and v.is_floating_point() else v for k, v in d.items()}
    if case["op"] == "ffn":
        # the definition, differentiated automatically
        x, w1, w2 = (wide[k].requires_grad_(case["train"]) for k in ("x", "w1", "w2"))
        I = case["I"]
        rows = torch.arange(2 * I, device=DEV)
        gate, up = (rows[:I], rows[I:]) if case["layout"] == "split" else (rows[0::2], rows[1::2])
        out = torch.mm(_gate64(torch.mm(x, w1[gate].t()), torch.mm(x, w1[up].t()), case["act"]), w2.t())
        if not case["train"]:
            return out
        dx, dw1, dw2 = torch.autograd.grad(out, (x, w1, w2), wide["dout"])
        return {"out": out.detach(), "dx": dx, "dw1": dw1, "dw2": dw2}
    x, T, N = wide["x"], case["T"], case["N"]
    y = torch.zeros((T, N), dtype=torch.float64, device=DEV)
    if wide["add"] is not None:
        y += wide["add"]
    if wide["w"] is not None:
        y += torch.mm(x, wide["w"].t())
    ids = d["ids"].cpu()
    for i in sorted(set(ids.tolist()) - {-1}):
        rows = (ids == i).nonzero()[:, 0].to(DEV)
        r = case["R"] if d["ranks"] is None else int(d["ranks"][i])
        low = torch.mm(x[rows], wide["a"][i, :r].t())
        y[rows] += wide["scales"][i] * torch.mm(low, wide["b"][i, :, :r].t().contiguous())
    if case["epilogue"] == "split":
        y = _gate64(y[:, : N // 2], y[:, N // 2:], case["act"])
    elif case["epilogue"] == "interleaved":
        y = _gate64(y[:, 0::2], y[:, 1::2], case["act"])
    return y
