"""The projection with per-token low-rank adapters against the float64 oracle (tolerances: dense_util)."""
import numpy as np
import pytest
import torch

from tests import dense_util as du

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("mxfp4_weight_mixture_amd")
BF, HF, F = torch.bfloat16, torch.float16, torch.float32


def _ids(kind, T, n, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "one":
        ids = torch.full((T,), n - 1)
    elif kind == "none":
        ids = torch.full((T,), -1)
    elif kind == "each":
        ids = torch.randint(-1, n, (T,), generator=g)
    elif kind == "outside":
        ids = torch.randint(-3, n + 3, (T,), generator=g)
        ids[0] = 2 ** 31 - 1
        ids[-1] = -2 ** 31
    else:   # runs
        ids = torch.sort(torch.randint(0, n, (T,), generator=g)).values
        ids = torch.randperm(n, generator=g)[ids]
    return ids.to(torch.int32).to("cuda")


def _problem(T, K, N, n, R, dtype, kind, seed, base=True, ranks=None, scales=True, **kw):
    x, ids = du.normal((T, K), 1.0, dtype, seed), _ids(kind, T, n, seed)
    w = du.normal((N, K), K ** -0.5, dtype, seed + 1) if base else None
    a, b = du.normal((n, R, K), K ** -0.5, dtype, seed + 2), du.normal((n, N, R), R ** -0.5, dtype, seed + 3)
    sc = torch.linspace(-1.5, 2.0, n, device="cuda") if scales else None
    rk = torch.tensor(ranks, dtype=torch.int32, device="cuda") if ranks is not None else None
    return x, ids, mx.AdapterLinear(w, a, b, scales=sc, ranks=rk, **kw)


def _check(f, x, ids, out, out_dtype, add=None, epilogue="none", act="silu", what=""):
    host = lambda t: None if t is None else du.f64(t)
    ref, bound = du.adapter_bounds(du.f64(x), host(f.w), ids.cpu().numpy(), du.f64(f.lora_a), du.f64(f.lora_b),
                                   f.dtype, out_dtype, host(f.scales),
                                   None if f.ranks is None else f.ranks.cpu().numpy(), host(add), epilogue, act)
    du.assert_within(out, ref, bound, what)


CASES = [  # T, K, N, n, R, ids
    (1, 8, 8, 1, 8, "one"), (1, 512, 264, 3, 16, "each"), (2, 264, 1032, 2, 64, "none"), (7, 2048, 136, 5, 8, "each"),
    (16, 136, 256, 20, 24, "each"), (17, 520, 128, 4, 128, "outside"), (32, 1000, 520, 40, 16, "each"),
    (33, 392, 96, 2, 256, "runs"), (64, 256, 512, 64, 32, "each"), (65, 72, 200, 70, 16, "each"),
    (130, 328, 392, 9, 40, "outside"), (200, 512, 264, 3, 64, "runs"), (300, 136, 72, 300, 8, "each"),
    (513, 264, 392, 5, 16, "runs"), (257, 1000, 136, 2, 104, "one")]


@pytest.mark.parametrize("T,K,N,n,R,kind", CASES)
@pytest.mark.parametrize("dtype,epilogue,act", [(BF, "none", "silu"), (HF, "split", "gelu"),
                                                (BF, "interleaved", "silu")])
def test_against_oracle(T, K, N, n, R, kind, dtype, epilogue, act):
    N = N if epilogue == "none" else (N + 15) // 16 * 16
    x, ids, f = _problem(T, K, N, n, R, dtype, kind, 10 * T + n, epilogue=epilogue, act=act)
    _check(f, x, ids, f.forward(x, ids), dtype, epilogue=epilogue, act=act)


@pytest.mark.parametrize("T", [1, 3, 17, 40, 64, 100, 257, 300])
@pytest.mark.parametrize("N", [8, 24, 72, 264, 1032, 4504])
@pytest.mark.parametrize("epilogue", ["split", "interleaved"])
def test_gated_widths_of_odd_fours(T, N, epilogue):
    """N / 2 is an odd multiple of four: rows of out are 8-byte aligned, the last group of columns is half one.
    Nothing is read or written past an adapter's rows or the output's."""
    x, ids, f = _problem(T, 136, N, 5, 24, HF, "each", 12, epilogue=epilogue, ranks=[24, 7, 0, 16, 24])
    wide = torch.full((T + 2, N // 2 + 4), 3.0, dtype=HF, device="cuda")
    out = wide[:, : N // 2][1: T + 1] if (N // 2 + 4) * 2 % 16 == 0 else torch.empty((T, N // 2), dtype=HF, device="cuda")
    add = du.normal((T, N), 1.0, HF, 13)
    _check(f, x, ids, f.forward(x, ids, add=add, out=out), HF, add=add, epilogue=epilogue)
    if out.stride(0) != N // 2 or T == 1:
        wide[1: T + 1, : N // 2] = 3.0
        assert (wide == 3.0).all()
    _check(f, x, ids, f.forward(x, ids), HF, epilogue=epilogue)
    _check(f, x, ids, f.forward(x, ids, out_dtype=F), F, epilogue=epilogue)


@pytest.mark.parametrize("T", [1, 13, 40, 150])
@pytest.mark.parametrize("out_dtype", [F, HF])
@pytest.mark.parametrize("base", [True, False])
def test_add_strides_and_no_base(T, out_dtype, base):
    K, N = 264, 136
    x, ids, f = _problem(T, K, N, 6, 24, HF, "each", 5, base=base)
    x = du.strided(x, 16)
    add = du.strided(du.normal((T, N), 2.0, out_dtype, 6), 8)
    wide = torch.full((T + 2, N + 16), 3.0, dtype=out_dtype, device="cuda")
    out = f.forward(x, ids, add=add, out=wide[1: T + 1, 8: N + 8])
    _check(f, x, ids, out, out_dtype, add=add)
    wide[1: T + 1, 8: N + 8] = 3.0
    assert (wide == 3.0).all()
    res = add.clone()
    f.forward(x, ids, add=res, out=res)
    _check(f, x, ids, res, out_dtype, add=add, what="in place")
    _check(f, x, ids, f.forward(x, ids), HF, what="without add")


@pytest.mark.parametrize("T", [9, 150])
@pytest.mark.parametrize("epilogue", ["split", "interleaved"])
def test_add_before_the_gate(T, epilogue):
    x, ids, f = _problem(T, 136, 144, 4, 16, BF, "each", 8, epilogue=epilogue)
    add = du.normal((T, 144), 1.0, F, 9)
    _check(f, x, ids, f.forward(x, ids, add=add), F, add=add, epilogue=epilogue)


@pytest.mark.parametrize("T", [5, 30, 140])
def test_ranks(T):
    ranks = [0, 1, 7, 8, 9, 31, 32, 1000, -4]
    x, ids, f = _problem(T, 200, 264, len(ranks), 32, HF, "each", 21, ranks=ranks)
    # what lies behind an adapter's rank is not used
    for i, r in enumerate(ranks):
        r = min(max(r, 0), 32)
        f.lora_a[i, r:], f.lora_b[i, :, r:] = 0.0, 0.0
    out = f.forward(x, ids)
    _check(f, x, ids, out, HF)
    for i, r in enumerate(ranks):
        r = min(max(r, 0), 32)
        f.lora_a[i, r:], f.lora_b[i, :, r:] = float("nan"), float("inf")
    assert torch.equal(f.forward(x, ids), out)


@pytest.mark.parametrize("T", [1, 30, 64, 200])
def test_no_adapter_gives_the_shared_projection(T):
    x, ids, f = _problem(T, 520, 136, 3, 16, BF, "none", 31)
    f.lora_a.fill_(float("nan")), f.lora_b.fill_(float("nan"))
    ref = f.forward(x, ids)
    none = mx.AdapterLinear(f.w, f.lora_a[:0], f.lora_b[:0])
    assert torch.equal(none.forward(x, ids), ref)
    refv, bound = du.adapter_bounds(du.f64(x), du.f64(f.w), ids.cpu().numpy(), np.zeros((0, 16, 520)),
                                    np.zeros((0, 136, 16)), BF, BF)
    du.assert_within(ref, refv, bound)


@pytest.mark.parametrize("T", [12, 60, 150, 600])
@pytest.mark.parametrize("epilogue", ["none", "split"])
def test_rows_do_not_reach_each_other(T, epilogue):
    """Infinities and NaN in one adapter or token stay with its rows, which share tiles with all others."""
    x, ids, f = _problem(T, 264, 144, 5, 16, BF, "each", 41, epilogue=epilogue)
    clean = f.forward(x, ids)
    f.lora_a[1, 3, 7], f.lora_b[2, :, 5] = float("inf"), float("nan")
    f.scales[3] = float("inf")
    x[T // 2, 3] = float("nan")
    out = f.forward(x, ids)
    hit = (ids == 1) | (ids == 2) | (ids == 3)
    hit[T // 2] = True
    assert torch.equal(out[~hit], clean[~hit])
    assert out[ids == 2].isnan().all() and out[T // 2].isnan().all()


@pytest.mark.parametrize("T", [1, 24, 90, 400])
def test_token_order_side_stream_and_repeat(T):
    x, ids, f = _problem(T, 392, 264, 7, 16, BF, "each", 51)
    ref = f.forward(x, ids)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = f.forward(x, ids, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, ref)
    p = torch.randperm(T, generator=torch.Generator().manual_seed(1)).to("cuda")
    assert torch.equal(f.forward(x[p].contiguous(), ids[p].contiguous()), ref[p])


def test_no_tokens_and_replaced_adapter():
    x, ids, f = _problem(0, 64, 32, 2, 8, BF, "none", 3)
    assert f.forward(x, ids).shape == (0, 32)
    x, ids, f = _problem(20, 64, 32, 2, 8, BF, "one", 4)
    f.forward(x, ids)
    f.lora_b[1] = du.normal((32, 8), 1.0, BF, 77)
    _check(f, x, ids, f.forward(x, ids), BF)


def test_two_graphs_replayed_in_turn():
    """Replays read the current tokens, ids and adapters."""
    runs = []
    for T in (4, 30, 180):
        x, ids, f = _problem(T, 264, 144, 6, 16, HF, "each", 60 + T, epilogue="split", act="gelu")
        f.forward(x, ids)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = f.forward(x, ids)
        runs.append((x, ids, f, g, out))
    for k in range(3):
        for x, ids, f, g, out in runs:
            T = x.shape[0]
            x.copy_(du.normal(tuple(x.shape), 1.0, HF, 100 * k + T))
            ids.copy_(_ids("each", T, 6, 200 * k + T))
            f.lora_a.mul_(-1)
            g.replay()
            eager = f.forward(x, ids)
            torch.cuda.synchronize()
            assert torch.equal(out, eager), (k, T)


def test_binding_refusals():
    x, ids, f = _problem(4, 64, 32, 2, 8, BF, "each", 5)
    for bad, needle in ((dict(ids=ids.long()), "ids"), (dict(ids=ids[:3]), "ids"), (dict(ids=ids.cpu()), "ids"),
                        (dict(x=x.float()), "float32"), (dict(x=x[:, :56]), "shape"),
                        (dict(out=torch.zeros(4, 32, dtype=HF, device="cuda")), "out is"),
                        (dict(add=torch.zeros(4, 24, dtype=BF, device="cuda")), "add has")):
        with pytest.raises(ValueError, match=needle):
            f.forward(**{"x": x, "ids": ids, **bad})
    a, b = f.lora_a, f.lora_b
    for kw, needle in ((dict(w=f.w[:16]), "w must"), (dict(w=f.w, scales=torch.ones(3, device="cuda")), "scales"),
                       (dict(w=f.w, ranks=torch.ones(2, device="cuda")), "ranks"),
                       (dict(w=None, epilogue="split"), "needs w"), (dict(w=f.w, act="relu"), "act")):
        with pytest.raises(ValueError, match=needle):
            mx.AdapterLinear(kw.pop("w"), a, b, **kw)
    with pytest.raises(ValueError, match="lora_a"):
        mx.AdapterLinear(f.w, a, b.transpose(1, 2).contiguous())
    with pytest.raises(mx.MoeError, match="overlaps"):
        sq = mx.AdapterLinear(du.normal((64, 64), 1.0, BF, 1), a, du.normal((2, 64, 8), 1.0, BF, 2))
        sq.forward(x, ids, out=x)
