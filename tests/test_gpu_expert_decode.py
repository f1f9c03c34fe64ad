"""Decode of many experts: the kernel of few rows, whose blocks find their rows from the offsets, with rows in experts
behind the first 64 (a wave's lanes) and behind the first 1024 (a wave's trip), in one tile each and in several, gathered
and not.  Bounds: dense_util, for each expert's rows.

Sizes that take that kernel: sums of at least 1024, at most 16 rows an expert, few tiles of columns."""
import numpy as np
import pytest
import torch

from tests import dense_util as du
from tests import test_gpu_expert_paths as paths

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("mxfp4_weight_mixture_amd")
BF, HF, F = torch.bfloat16, torch.float16, torch.float32

H, I = 1032, 1024
ROWS = {   # expert: rows
    "256, one tile each": (256, {3: 1, 63: 1, 64: 2, 130: 1, 192: 1, 255: 3}),
    "256, the last alone": (256, {255: 1}),
    "256, several tiles late": (256, {3: 1, 200: 40, 255: 2}),
    "256, several tiles early": (256, {0: 33, 64: 1, 128: 17, 254: 1}),
    "1100, one tile each": (1100, {0: 1, 63: 1, 64: 1, 1022: 1, 1023: 2, 1024: 1, 1025: 1, 1099: 1}),
    "1100, several tiles late": (1100, {5: 1, 700: 17, 1090: 36}),
    "1100, the last alone": (1100, {1099: 9}),
}


def _within(out, gu, off, plain, f, what):
    for e in range(f.E):
        s = slice(int(off[e]), int(off[e + 1]))
        if s.start == s.stop:
            continue
        ref, bound, kept, err, _, _ = du.ffn_bounds(du.f64(plain[s]), du.f64(f.w1[e]), du.f64(f.w2[e]), f.layout, f.act,
                                                    f.dtype, f.dtype)
        du.assert_within(out[s], ref, bound, f"{what}: out of expert {e}")
        if gu is not None:
            du.assert_within(gu[s], kept, err + 1e-37, f"{what}: gate_up of expert {e}")


@pytest.mark.parametrize("name", ROWS)
@pytest.mark.parametrize("dtype,layout,act", [(BF, "split", "silu"), (HF, "interleaved", "gelu")])
def test_rows_in_late_experts(name, dtype, layout, act):
    E, some = ROWS[name]
    counts = np.zeros(E, dtype=np.int64)
    for e, n in some.items():
        counts[e] = n
    rows = int(counts.sum())
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)
    g = torch.Generator(device="cuda").manual_seed(E + rows)
    normal = lambda shape, scale: torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, scale, generator=g)
    f = mx.ExpertFFN(normal((E, 2 * I, H), H ** -0.5), normal((E, H, I), I ** -0.5), layout=layout, act=act)
    lone = torch.Generator().manual_seed(7)
    for tokens in (9, 30):                      # up to 16 rows an expert where a token comes once, and more
        x = du.normal((tokens, H), 1.0, dtype, tokens)
        gather = torch.randint(0, 2 * tokens, (rows,), generator=lone).to(torch.int32).to("cuda")
        plain = x[gather.long() // 2]
        out, gu = f.forward(x, off.to("cuda"), gather=gather, gather_div=2, save=True)
        _within(out, gu, off, plain, f, f"{tokens} tokens")
        out, gu = f.forward(plain, off.to("cuda"), save=True)
        _within(out, gu, off, plain, f, "rows in order")
        assert torch.equal(f.forward(plain, off.to("cuda")), out)


@pytest.mark.parametrize("name", [n for n in paths.CASES if n.startswith("few")])
@pytest.mark.parametrize("dtype,layout,act", [(BF, "interleaved", "silu"), (HF, "split", "gelu")])
def test_rows_in_order_of_the_cases_for_few_rows(name, dtype, layout, act):
    _, f, off, x, gather = paths._case(name, dtype, layout, act)
    plain = x[gather.long() // 2]
    out, gu = f.forward(plain, off, save=True)
    _within(out, gu, off.cpu(), plain, f, name)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_few_rows_in_order_of_a_few_experts(dtype):
    """Up to 16 rows without gather."""
    counts = [1, 0, 3, 7, 0, 2]
    w1, w2 = du.normal((6, 2 * I, H), H ** -0.5, dtype, 1), du.normal((6, H, I), I ** -0.5, dtype, 2)
    for layout in ("split", "interleaved"):
        f = mx.ExpertFFN(w1, w2, layout=layout)
        off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)
        x = du.strided(du.normal((13, H), 1.0, dtype, 3), 40)
        out, gu = f.forward(x, off.to("cuda"), save=True)
        _within(out, gu, off, x, f, layout)
