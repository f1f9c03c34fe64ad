"""The dense operators at sizes that fill the chip: whole rounds of 256 x 256 tiles, a last round whole, in
halves and in quarters, ragged edges, many adapter runs.

The reference is plain float64 on the GPU (torch.mm), the bounds those of dense_util."""
import pytest
import torch

from tests import dense_util as du

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("mxfp4_weight_mixture_amd")
BF, HF, F = torch.bfloat16, torch.float16, torch.float32
mm = torch.mm


def _act(g, act):
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * (1 - s)
    c = (2 / torch.pi) ** 0.5
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g ** 2)


def _halves(gu, layout):
    n = gu.shape[1] // 2
    return (gu[:, :n], gu[:, n:]) if layout == "split" else (gu[:, 0::2], gu[:, 1::2])


def _join(g, u, layout):
    return torch.cat([g, u], 1) if layout == "split" else torch.stack([g, u], 2).flatten(1)


def _within(got, ref, err, what):
    u = du.u(got.dtype)
    bound = err + u * (ref.abs() + err) + du.floor(got.dtype)
    over = (got.double() - ref).abs() - bound
    assert got.isfinite().all(), what
    assert over.max() <= 0, (what, got.dtype, over.max().item(), divmod(int(over.argmax()), ref.shape[1]))


def _hoeff(q2, dtype):
    return 7 * du.u(dtype) * q2.sqrt()


# T x 1544 x 1544: FC1 has ceil(T / 256) * 13 tiles of 256 x 256, FC2 and dx ceil(T / 256) * 7: fewer than a
# quarter, a half, and all of the CUs, and more than the CUs
@pytest.mark.parametrize("T,dtype,layout,act,save", [
    (700, BF, "split", "silu", True), (1288, HF, "interleaved", "gelu", "half"), (2601, BF, "interleaved", "silu", True),
    (5001, HF, "split", "gelu", True)])
def test_ffn(T, dtype, layout, act, save):
    _check_ffn(T, 1544, 1544, dtype, layout, act, save)


# few tiles and a long reduction: K is split over blocks (forward, dh, dx or the weights' gradients)
@pytest.mark.parametrize("T,H,I,dtype,layout,act,save", [
    (87, 1312, 3480, BF, "split", "silu", True), (70, 8200, 136, HF, "interleaved", "gelu", True),
    (300, 136, 9000, BF, "interleaved", "gelu", "half"), (20000, 72, 200, HF, "split", "silu", True),
    (1281, 4560, 264, BF, "split", "gelu", True)])
def test_ffn_with_long_reductions(T, H, I, dtype, layout, act, save):
    _check_ffn(T, H, I, dtype, layout, act, save)


def _check_ffn(T, H, I, dtype, layout, act, save):
    x, dout = du.normal((T, H), 1.0, dtype, T), du.normal((T, H), 1.0, dtype, T + 1)
    w1, w2 = du.normal((2 * I, H), H ** -0.5, dtype, T + 2), du.normal((H, I), I ** -0.5, dtype, T + 3)
    f = mx.GatedFFN(w1, w2, layout=layout, act=act)
    out, gu = f.forward(x, save=save)
    assert torch.equal(f.forward(x), out)
    dx, dw1, dw2 = f.backward(dout, x, gu)

    X, W1, W2, DO = x.double(), w1.double(), w2.double(), dout.double()
    GU = mm(X, W1.t())
    e_gu = H * du.F32 * mm(X.abs(), W1.abs().t())
    _within(gu, GU, e_gu, "gate_up")
    (g, up), (eg, eu) = _halves(GU, layout), _halves(e_gu, layout)
    a, da = _act(g, act)
    h = a * up
    e_h = up.abs() * (da.abs() * eg + 1.2 * eg ** 2) + (a.abs() + 1.2 * eg) * eu + du.GATE * h.abs() + du.floor(dtype)
    err = mm(e_h, W2.abs().t()) + I * du.F32 * mm(h.abs(), W2.abs().t()) + _hoeff(mm(h ** 2, (W2 ** 2).t()), dtype)
    _within(out, mm(h, W2.t()), err, "out")

    # the backward pass, with gate_up's rounding when kept
    e_gu = e_gu + (du.u(gu.dtype) if gu.dtype != F else du.F32) * GU.abs() + du.floor(gu.dtype)
    eg, eu = _halves(e_gu, layout)
    dh = mm(DO, W2)
    e_dh = H * du.F32 * mm(DO.abs(), W2.abs())
    e_g = (up.abs() + eu) * (da.abs() + 1.2 * eg) * e_dh \
        + dh.abs() * (eu * da.abs() + (up.abs() + eu) * 1.2 * eg) + du.GATE * (dh * up).abs() * (da.abs() + 1)
    e_u = (a.abs() + 1.2 * eg) * e_dh + dh.abs() * 1.2 * eg + du.GATE * (dh * a).abs()
    e_h = up.abs() * (da.abs() * eg + 1.2 * eg ** 2) + (a.abs() + 1.2 * eg) * eu + du.GATE * h.abs() + du.floor(dtype)
    dgu, e_dgu = _join(dh * up * da, dh * a, layout), _join(e_g, e_u, layout) + du.floor(dtype)
    _within(dx, mm(dgu, W1), mm(e_dgu, W1.abs()) + 2 * I * du.F32 * mm(dgu.abs(), W1.abs())
            + _hoeff(mm(dgu ** 2, W1 ** 2), dtype), "dx")
    _within(dw1, mm(dgu.t(), X), mm(e_dgu.t(), X.abs()) + T * du.F32 * mm(dgu.abs().t(), X.abs())
            + _hoeff(mm((dgu ** 2).t(), X ** 2), dtype), "dw1")
    _within(dw2, mm(DO.t(), h), mm(DO.abs().t(), e_h) + T * du.F32 * mm(DO.abs().t(), h.abs())
            + _hoeff(mm((DO ** 2).t(), h ** 2), dtype), "dw2")


@pytest.mark.parametrize("T,n,R,kind,dtype,epilogue,act", [
    (700, 5, 16, "runs", BF, "none", "silu"), (1288, 9, 40, "runs", HF, "split", "gelu"),
    (2601, 40, 8, "each", BF, "none", "silu"), (5001, 12, 64, "runs", BF, "interleaved", "silu"),
    (2601, 3, 200, "runs", HF, "split", "silu")])
@pytest.mark.parametrize("base", [True, False])
def test_adapters(T, n, R, kind, dtype, epilogue, act, base):
    if not base and epilogue != "none":
        epilogue = "none"
    _check_adapters(T, 1000, 3088, n, R, kind, dtype, epilogue, act, base)


# few tiles and long rows: K is split over blocks, the adapters' part goes with one of them
@pytest.mark.parametrize("T,K,N,n,R,kind,dtype,epilogue", [
    (100, 9000, 136, 6, 16, "each", BF, "none"), (256, 7168, 528, 40, 24, "each", HF, "split"),
    (400, 8008, 272, 3, 64, "runs", BF, "interleaved"), (2407, 4888, 960, 2, 16, "runs", HF, "none"),
    (1100, 12000, 528, 5, 40, "runs", BF, "split"), (90, 6000, 136, 4, 8, "each", HF, "split"),
    (300, 8000, 520, 3, 16, "runs", HF, "interleaved"), (2050, 512, 4504, 5, 16, "runs", BF, "interleaved"),
    (2050, 512, 4504, 5, 16, "runs", BF, "split")])
def test_adapters_with_long_rows(T, K, N, n, R, kind, dtype, epilogue):
    _check_adapters(T, K, N, n, R, kind, dtype, epilogue, "gelu", True)


def _check_adapters(T, K, N, n, R, kind, dtype, epilogue, act, base):
    x = du.normal((T, K), 1.0, dtype, T)
    w = du.normal((N, K), K ** -0.5, dtype, T + 1) if base else None
    a, b = du.normal((n, R, K), K ** -0.5, dtype, T + 2), du.normal((n, N, R), R ** -0.5, dtype, T + 3)
    scales = torch.linspace(-1.5, 2.0, n, device="cuda")
    g = torch.Generator().manual_seed(T)
    ranks = torch.randint(0, R + 1, (n,), generator=g)
    ids = torch.randint(-1, n, (T,), generator=g)
    if kind == "runs":
        ids = torch.sort(ids).values
    f = mx.AdapterLinear(w, a, b, scales=scales, ranks=ranks.int().to("cuda"), epilogue=epilogue, act=act)
    add = None if base else du.normal((T, N), 1.0, dtype, T + 4)
    out = f.forward(x, ids.int().to("cuda"), add=add)

    X = x.double()
    y = torch.zeros((T, N), dtype=torch.float64, device="cuda")
    err = torch.zeros_like(y)
    if base:
        y += mm(X, w.double().t())
        err += K * du.F32 * mm(X.abs(), w.double().abs().t())
    for i in range(n):
        rows, r = (ids == i).nonzero()[:, 0].to("cuda"), int(ranks[i])
        if r == 0 or rows.numel() == 0:
            continue
        A, B, sc = a[i, :r].double(), b[i, :, :r].double().contiguous(), scales[i].double()
        s = sc * mm(X[rows], A.t())
        e_s = sc.abs() * (K + 2) * du.F32 * mm(X[rows].abs(), A.abs().t()) + du.floor(dtype)
        y[rows] += mm(s, B.t())
        # s enters as two 16-bit numbers: off by u^2 of it at most
        err[rows] += mm(e_s + ((R + 2) * du.F32 + du.u(dtype) ** 2) * s.abs(), B.abs().t())
    if add is not None:
        y += add.double()
    err += 8 * du.F32 * (y.abs() + err + 4)
    if epilogue != "none":
        (gt, up), (eg, eu) = _halves(y, epilogue), _halves(err, epilogue)
        av, da = _act(gt, act)
        err = (up.abs() + eu) * (da.abs() * eg + 1.2 * eg ** 2) + (av.abs() + 1.2 * eg) * eu \
            + du.GATE * (av * up).abs()
        y = av * up
    _within(out, y, err, "out")


def test_rows_do_not_reach_each_other_in_large_batches():
    """Infinities and NaN in one adapter or token stay with its rows, whatever tiles they share."""
    T, K, N, n, R = 3000, 264, 3088, 6, 16
    x, ids = du.normal((T, K), 1.0, BF, 1), (torch.arange(T, device="cuda") * 7 // 500 % (n + 1) - 1).int()
    w = du.normal((N, K), K ** -0.5, BF, 2)
    a, b = du.normal((n, R, K), K ** -0.5, BF, 3), du.normal((n, N, R), R ** -0.5, BF, 4)
    for base, epilogue in ((w, "none"), (w, "split"), (None, "none")):
        f = mx.AdapterLinear(base, a.clone(), b.clone(), epilogue=epilogue)
        clean = f.forward(x, ids)
        f.lora_a[1, 3, 7], f.lora_b[2, :, 5] = float("inf"), float("nan")
        y = x.clone()
        y[1500, 3] = float("nan")
        out = f.forward(y, ids)
        hit = (ids == 1) | (ids == 2)
        hit[1500] = True
        assert torch.equal(out[~hit], clean[~hit])
        assert out[ids == 2].isnan().all()
        # token 1500 has no adapter: its NaN shows through the shared projection only
        assert ids[1500] == -1 and (out[1500].isnan().all() if base is not None else not out[1500].any())


@pytest.mark.parametrize("T", [300, 2000])
def test_adapters_do_not_depend_on_the_order_of_tokens(T):
    K, N, n, R = 264, 3088, 9, 24
    x, w = du.normal((T, K), 1.0, HF, 1), du.normal((N, K), K ** -0.5, HF, 2)
    a, b = du.normal((n, R, K), K ** -0.5, HF, 3), du.normal((n, N, R), R ** -0.5, HF, 4)
    f = mx.AdapterLinear(w, a, b)
    g = torch.Generator().manual_seed(5)
    ids = torch.sort(torch.randint(-1, n, (T,), generator=g)).values.int().to("cuda")
    ref = f.forward(x, ids)
    p = torch.randperm(T, generator=g).to("cuda")
    assert torch.equal(f.forward(x[p].contiguous(), ids[p].contiguous()), ref[p])


def test_offsets_past_32_bits():
    """Rows of x and out that start past 4 GiB, and a gate_up of 5 GB."""
    T, H, I = 270000, 64, 2312
    stride = 8192
    x = torch.empty((T, stride), dtype=BF, device="cuda")[:, :H]
    x.copy_(du.normal((1000, H), 1.0, BF, 1).repeat(270, 1))
    f = mx.GatedFFN(du.normal((2 * I, H), H ** -0.5, BF, 2), du.normal((H, I), I ** -0.5, BF, 3))
    out = torch.empty((T, stride), dtype=BF, device="cuda")[:, :H]
    _, gu = f.forward(x, out=out, save=True)
    ref, gref = f.forward(x[:1000].contiguous(), save=True)
    for i in (0, 131, 200, 269):   # the same rows, far down: the same kernel, so the same numbers
        assert torch.equal(gu[i * 1000: i * 1000 + 1000], gu[:1000])
        assert torch.equal(out[i * 1000: i * 1000 + 1000], out[:1000])
    # against the smaller call, which may take other kernels: both are within a rounding of h and of out
    assert (out[:1000].double() - ref.double()).abs().max() <= 16 * du.u(BF) * ref.double().abs().max()
    assert (gu[:1000] - gref).abs().max() <= 2 * H * du.F32 * 64


@pytest.mark.parametrize("T", [3, 20, 300])
def test_up_rows_far_behind_the_gate_rows(T):
    """w1 of 2 GiB: in the split order a gate row's up row lies 1 GiB behind it; the interleaved order of the
    same weights keeps them together.  Both against float64 on some columns."""
    H, I = 8192, 65536
    w1 = torch.empty((2 * I, H), dtype=BF, device="cuda").normal_(0, H ** -0.5, generator=torch.Generator("cuda")
                                                                  .manual_seed(1))
    x = du.normal((T, H), 1.0, BF, 2)
    cols = torch.tensor([0, 1, 31, 32, 33000, 65527, 65535], device="cuda")
    pick = torch.zeros((H, I), dtype=BF, device="cuda")   # out[:, j] = h[:, cols[j]]
    pick[torch.arange(len(cols)), cols] = 1.0
    inter = torch.stack([w1[:I], w1[I:]], 1).reshape(2 * I, H)
    g, up = mm(x.double(), w1[cols].double().t()), mm(x.double(), w1[I + cols].double().t())
    h = g * torch.sigmoid(g) * up
    e = H * du.F32 * (H ** 0.5) * 4   # sum |x w| of these spreads is below 0.64 sqrt(H) + 7 sigma < sqrt(H)
    err = e * (1.1 * up.abs() + g.abs() + 4 * e) + du.u(BF) * h.abs()
    for w, layout in ((w1, "split"), (inter, "interleaved")):
        out = mx.GatedFFN(w, pick, layout=layout).forward(x)
        _within(out[:, : len(cols)], h, err, layout)
        assert not out[:, len(cols):].any()


def test_16_bit_subnormals_count():
    """Operands below the smallest normal number are not flushed to zero."""
    K, N = 64, 16
    for dtype, tiny in ((HF, 2.0 ** -20), (BF, 2.0 ** -130)):
        for T in (1, 20, 300):
            x = torch.full((T, K), tiny, dtype=dtype, device="cuda")
            w = torch.full((N, K), 2.0, dtype=dtype, device="cuda")
            none = mx.AdapterLinear(w, w.new_zeros((0, 8, K)), w.new_zeros((0, N, 8)))
            assert (none.forward(x, torch.zeros(T, dtype=torch.int32, device="cuda"), out_dtype=F)
                    == 2 * K * tiny).all(), (dtype, T)


@pytest.mark.parametrize("T", [1, 40, 100, 700])
def test_no_projection_and_no_adapter(T):
    N, K = 136, 64
    x, add = du.normal((T, K), 1.0, BF, 1), du.normal((T, N), 1.0, BF, 2)
    ids = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    for n in (0, 2):
        f = mx.AdapterLinear(None, x.new_full((n, 8, K), float("nan")), x.new_full((n, N, 8), float("nan")))
        assert torch.equal(f.forward(x, ids, add=add), add)
        assert not f.forward(x, ids).any()
