"""What is added, where rows lie and what stands behind a rank, through every kernel of the dense operators: the
few-row kernel, 64 x 64 tiles alone and in groups, 256 x 256 tiles in quarters, halves and whole, K in parts.

No tolerances: the sums before an addition do not depend on what is added or on strides, so each result equals
the same call's fp32 sums with the addition and the rounding done by torch."""
import pytest
import torch

from tests import dense_util as du

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("mxfp4_weight_mixture_amd")
BF, HF, F = torch.bfloat16, torch.float16, torch.float32

SIZES = [(3, 264, 136), (50, 264, 136), (300, 264, 136), (700, 1544, 1544), (2601, 1544, 1544), (5001, 1544, 1544),
         (87, 1312, 3480), (70, 8200, 136), (300, 136, 9000), (20000, 72, 200), (1281, 4560, 264)]


def _block(T, H, I, dtype):
    f = mx.GatedFFN(du.normal((2 * I, H), H ** -0.5, dtype, T), du.normal((H, I), I ** -0.5, dtype, T + 1))
    return f, du.normal((T, H), 1.0, dtype, T + 2)


@pytest.mark.parametrize("T,H,I", SIZES)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_accumulated_weight_gradients(T, H, I, dtype):
    f, x = _block(T, H, I, dtype)
    dout = du.normal((T, H), 1.0, dtype, T + 3)
    _, gu = f.forward(x, save=True)
    _, g1, g2 = f.backward(dout, x, gu, dw_dtype=F)
    for t in (F, dtype):
        b1, b2 = du.normal((2 * I, H), 3.0, t, 5), du.normal((H, I), 3.0, t, 6)
        a1, a2 = b1.clone(), b2.clone()
        f.backward(dout, x, gu, dw1=a1, dw2=a2, accumulate=True)
        assert torch.equal(a1, (g1 + b1.float()).to(t)) and torch.equal(a2, (g2 + b2.float()).to(t)), t


@pytest.mark.parametrize("T,H,I", SIZES)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_added_rows_and_strides(T, H, I, dtype):
    f, x = _block(T, H, I, dtype)
    sums, gu = f.forward(x, out_dtype=F, save=True)
    far = du.strided(x, 24)
    for t in (F, dtype):
        add = du.strided(du.normal((T, H), 2.0, t, 7), 40)
        wide = torch.full((T + 2, H + 16), 3.0, dtype=t, device="cuda")
        out = wide[1: T + 1, 8: H + 8]
        _, kept = f.forward(far, add=add, out=out, save=True)
        assert torch.equal(out, (sums + add.float()).to(t)) and torch.equal(kept, gu)
        wide[1: T + 1, 8: H + 8] = 3.0
        assert (wide == 3.0).all()
        res = add.clone()
        f.forward(x, add=res, out=res)
        assert torch.equal(res, (sums + add.float()).to(t))
    dout = du.normal((T, H), 1.0, dtype, T + 3)
    want = f.backward(dout, x, gu)
    wide = torch.full((T + 2, H + 16), 3.0, dtype=dtype, device="cuda")
    got = f.backward(du.strided(dout, 8), far, gu, dx=wide[1: T + 1, 8: H + 8])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    wide[1: T + 1, 8: H + 8] = 3.0
    assert (wide == 3.0).all()


# N of adapters whose tokens are taken by the few-row kernel, 64 x 64 tiles, their own kernel (no projection) or
# 256 x 256 tiles in quarters, halves and whole, and K in parts (the last two)
@pytest.mark.parametrize("T,K,N", [(3, 136, 136), (40, 136, 264), (200, 136, 264), (300, 136, 264), (700, 136, 3088),
                                   (1100, 136, 3088), (3000, 136, 3088), (2407, 4888, 960), (90, 6000, 136)])
@pytest.mark.parametrize("base,dtype,epilogue", [
    (True, BF, "none"), (True, HF, "none"), (True, BF, "split"), (True, HF, "interleaved"), (False, BF, "none"),
    (False, HF, "none")])
def test_what_lies_behind_a_rank_does_not_count(T, K, N, base, dtype, epilogue):
    ranks = [0, 1, 7, 8, 9, 23, 24, 31, 32, 40, 99, -3]
    n, R = len(ranks), 40
    x = du.normal((T, K), 1.0, dtype, T)
    ids = (torch.arange(T, device="cuda") * 13 // 50 % (n + 1) - 1).int()
    a, b = du.normal((n, R, K), K ** -0.5, dtype, T + 1), du.normal((n, N, R), R ** -0.5, dtype, T + 2)
    w = du.normal((N, K), K ** -0.5, dtype, T + 3) if base else None
    f = mx.AdapterLinear(w, a, b, ranks=torch.tensor(ranks, dtype=torch.int32, device="cuda"), epilogue=epilogue)
    outs = []
    for behind in (0.0, 1.0, float("nan"), float("inf")):
        for i, r in enumerate(ranks):
            r = min(max(r, 0), R)
            a[i, r:], b[i, :, r:] = behind, behind
        outs.append(f.forward(x, ids, out_dtype=F))
    assert outs[0].isfinite().all() and all(torch.equal(o, outs[0]) for o in outs[1:])
