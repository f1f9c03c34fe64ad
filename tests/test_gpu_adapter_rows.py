"""The adapters' low-rank rows keep their fp32 precision and range in every kernel, and what is not finite in an
adapter reaches exactly what the definition says.

Every token has one nonzero value, so its products with A and W are exact in fp32 and its low-rank row is
off by its scale's rounding alone: 2^-24.  What is left of the error (rank r): the split of the row for the matrix
cores, none in bf16 (three parts of 8 bits) and 2^-22 of each value in fp16 (two of 11), with 2^-39 of the row's
largest (subnormal parts, 2^-25 beside 2^14); the sum of r terms in fp32, 2^-24 each, counted twice for sums that
the matrix cores cut instead of rounding; and what is added to the projection: the kernels of up to 256 tokens add
the r terms to its sum one by one, so r additions round a partial sum that is |projection| + sum|terms| at most:
r 2^-24 of each of the two."""
import pytest
import torch

from tests import dense_util as du

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("mxfp4_weight_mixture_amd")
BF, HF, F = torch.bfloat16, torch.float16, torch.float32
F32 = 2.0 ** -24

# tokens and columns of the few-row kernel (with and without DMA), the 64 x 64 tiles, 256 x 256 tiles in quarters,
# halves and whole; without a projection the adapters' own kernel from 257 tokens on
SIZES = [(3, 136), (40, 264), (200, 264), (300, 264), (700, 3088), (1100, 3088), (3000, 3088)]
K = 136


def _one_hot(T, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.zeros(T, K)
    x[torch.arange(T), torch.randint(0, K, (T,), generator=g)] = torch.randn(T, generator=g)
    return x.to(dtype).to("cuda")


def _rows(x, a, scales, ids, ranks):
    """The low-rank rows [T][R] in 64 bits, 0 behind the rank, and where a token has an adapter."""
    s = torch.zeros((x.shape[0], a.shape[1]), dtype=torch.float64, device="cuda")
    for i in range(a.shape[0]):
        rows = (ids == i).nonzero()[:, 0]
        s[rows, : ranks[i]] = scales[i].double() * torch.mm(x[rows].double(), a[i, : ranks[i]].double().t())
    return s


def _applied(s, b, ids, ranks):
    y = torch.zeros((s.shape[0], b.shape[1]), dtype=torch.float64, device="cuda")
    for i in range(b.shape[0]):
        rows, r = (ids == i).nonzero()[:, 0], ranks[i]
        y[rows] = torch.mm(s[rows, :r], b[i, :, :r].double().t().contiguous())
    return y


@pytest.mark.parametrize("T,N", SIZES)
@pytest.mark.parametrize("base", ["random", "zero", None])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_precision_and_range(T, N, base, dtype):
    """Scales from 1e-6 to 1e6, ranks from one: fp32 results to a few fp32 roundings."""
    R, scales = 24, torch.tensor([1.1, 1.3e-6, -1.7e6, 1e-3, 0.7, 1.9e4], device="cuda")
    ranks, n = [24, 1, 2, 7, 1, 16], 6
    x = _one_hot(T, dtype, T)
    ids = (torch.arange(T, device="cuda") * 7 // 40 % (n + 1) - 1).int()
    a, b = du.normal((n, R, K), 1.0, dtype, T + 1), du.normal((n, N, R), 1.0, dtype, T + 2)
    w = du.normal((N, K), float(base == "random"), dtype, T + 3) if base else None
    f = mx.AdapterLinear(w, a, b, scales=scales, ranks=torch.tensor(ranks, dtype=torch.int32, device="cuda"))
    got = f.forward(x, ids, out_dtype=F).double()
    s = _rows(x, a, scales, ids, ranks)
    ref, low = _applied(s, b, ids, ranks), _applied(s.abs(), b.abs(), ids, ranks)
    top = _applied(s.abs().amax(1, keepdim=True).expand_as(s), b.abs(), ids, ranks)
    r = torch.tensor([0] + ranks, device="cuda")[(ids + 1).long()].double()[:, None]
    split = (2.0 ** -22 * low + 2.0 ** -39 * top) if dtype == HF else 0.0
    main = torch.mm(x.double(), w.double().t()) if base else torch.zeros_like(ref)
    bound = F32 * low + split + 2 * (r + 2) * F32 * low + (r + 4) * F32 * (main.abs() + ref.abs())
    over = (got - ref - main).abs() - bound
    assert got.isfinite().all() and over.max() <= 0, (over.max().item(), ids[over.amax(1).argmax()].item())


@pytest.mark.parametrize("T,N", SIZES)
@pytest.mark.parametrize("base", ["random", None])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_infinities_in_an_adapter(T, N, base, dtype):
    """An infinity in B gives infinities of the right sign (NaN where it meets a zero or one of the other sign),
    whatever the number of tokens; an infinite scale gives infinities of the signs of x A^T and B."""
    R, n = 24, 4
    x = du.normal((T, K), 1.0, dtype, T)
    ids = (torch.arange(T, device="cuda") * 5 // 30 % (n + 1) - 1).int()
    a, b = du.normal((n, R, K), K ** -0.5, dtype, T + 1), du.normal((n, N, R), 1.0, dtype, T + 2)
    w = du.normal((N, K), K ** -0.5, dtype, T + 3) if base else None
    scales, ranks = torch.tensor([0.5, 1.0, 2.0, 1.0], device="cuda"), [24, 24, 16, 1]
    f = mx.AdapterLinear(w, a, b, scales=scales, ranks=torch.tensor(ranks, dtype=torch.int32, device="cuda"))
    clean = f.forward(x, ids, out_dtype=F)
    cols = [0, 5, 17, 70, N - 1]
    b[0, 0, 3], b[0, 5, 23], b[1, 17, 0], b[2, 70, 15] = float("inf"), float("-inf"), float("inf"), float("-inf")
    b[1, N - 1, 4], b[1, N - 1, 9], a[2, 15] = float("inf"), float("-inf"), 0.0
    b[2, 70, 16] = float("inf")   # behind the rank
    scales[3] = float("inf")
    got = f.forward(x, ids, out_dtype=F)
    low = torch.stack([torch.mm(x.double(), a[max(i, 0)].double().t()) for i in range(n)])   # [n][T][R]
    rest = torch.ones(N, dtype=torch.bool)
    rest[cols] = False
    for i in range(-1, n):
        rows = (ids == i).nonzero()[:, 0]
        if i < 0 or rows.numel() == 0:
            assert torch.equal(got[rows], clean[rows])
            continue
        r = ranks[i]
        s = scales[i].double() * low[i][rows][:, :r]
        if i == 3:
            assert torch.equal(got[rows], (s * b[i, :, 0].double()).float())
            continue
        if i != 2:
            assert torch.equal(got[rows][:, rest], clean[rows][:, rest]) and got[rows][:, rest].isfinite().all()
        want = (s[:, None, :] * b[i, cols, :r].double()).sum(2)
        at = got[rows][:, cols].double()
        assert torch.equal(at.isnan(), want.isnan()), i
        assert torch.equal(at.isposinf(), want.isposinf()) and torch.equal(at.isneginf(), want.isneginf()), i
    assert T == 3 or (ids < 0).any() and got[ids == 0].isinf().any() and (T < 100 or got[ids == 2].isnan().any())
