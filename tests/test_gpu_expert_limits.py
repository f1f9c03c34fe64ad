"""The experts at the limits of their sizes, and offsets that break their rule there: whatever is asked for, other
memory is not touched."""
import numpy as np
import pytest
import torch

from tests import dense_util as du

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("mxfp4_weight_mixture_amd")
BF, F = torch.bfloat16, torch.float32
GUARD = 4096


def _guarded(n, dtype=BF):
    """n values of 0 between guards."""
    buf = torch.full((n + 2 * GUARD,), 7.0, dtype=dtype, device="cuda")
    buf[GUARD: GUARD + n] = 0
    return buf, buf[GUARD: GUARD + n]


def _intact(buf):
    return bool((buf[:GUARD] == 7.0).all()) and bool((buf[-GUARD:] == 7.0).all())


@pytest.mark.parametrize("rows", [1 << 28, (1 << 27) + 12345])
def test_claims_past_2_31_tiles(rows):
    """8192 experts, every second one claims all of 2^28 rows: 2^32 row tiles of 256 (a sum that has to stop at what
    the list holds).  Weights and rows are 0, so that experts that claim the same rows write the same."""
    E, H, I = 8192, 8, 8
    f = mx.ExpertFFN(torch.zeros((E, 2 * I, H), dtype=BF, device="cuda"), torch.zeros((E, H, I), dtype=BF, device="cuda"))
    off = torch.tensor([0, rows] * (E // 2) + [0], dtype=torch.int32, device="cuda")
    x = torch.zeros((rows, H), dtype=BF, device="cuda")
    buf, out = _guarded(rows * H)
    # the call's workspace between guards, too: the list lies at its beginning
    n = mx.lib.moe_expert_ffn_workspace_size(rows, H, I, E)
    ws = torch.full((n + 2 * GUARD,), 9, dtype=torch.uint8, device="cuda")
    a = mx.ExpertFfnArgs.from_buffer_copy(f._fwd)
    a.w1, a.w2, a.rows, a.x, a.x_stride, a.out, a.out_stride = (f.w1.data_ptr(), f.w2.data_ptr(), rows, x.data_ptr(), H,
                                                                out.data_ptr(), H)
    a.expert_offsets, a.workspace, a.workspace_bytes = off.data_ptr(), ws.data_ptr() + GUARD, n
    mx._check(mx.lib.moe_expert_ffn_forward(a, mx._stream()))
    torch.cuda.synchronize()
    assert _intact(buf) and not out.any()
    assert (ws[:GUARD] == 9).all() and (ws[-GUARD:] == 9).all()
    # what the rule allows still comes out at this size: every row of one expert in the middle
    f.w1.fill_(1.0 / 8), f.w2.fill_(1.0 / 8), x.fill_(1.0)
    off = torch.tensor([0] * (E // 2 + 1) + [rows] * (E // 2), dtype=torch.int32, device="cuda")
    a.expert_offsets = off.data_ptr()
    mx._check(mx.lib.moe_expert_ffn_forward(a, mx._stream()))
    want = np.float32(1.0) / (1.0 + np.exp(-1.0))     # silu(1) * 1, eight eighths of it
    torch.cuda.synchronize()
    got = out.float()
    assert abs(float(got.min()) - want) <= 2.0 ** -7 and abs(float(got.max()) - want) <= 2.0 ** -7
    assert _intact(buf) and (ws[:GUARD] == 9).all() and (ws[-GUARD:] == 9).all()


def test_gradients_whose_tiles_are_many_together():
    """dx's, dw1's and dw2's tiles are each within one launch's limit (2^24 blocks of 256 threads), not together."""
    E, H, I = 8192, 90112, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    normal = lambda shape, scale: torch.empty(shape, dtype=BF, device="cuda").normal_(0.0, scale, generator=g)
    f = mx.ExpertFFN(normal((E, 2 * I, H), H ** -0.5), normal((E, H, I), I ** -0.5))
    x, dout = normal((E, H), 1.0), normal((E, H), 1.0)
    off = torch.arange(E + 1, dtype=torch.int32, device="cuda")     # a row an expert
    _, gu = f.forward(x, off, save=True)
    grads = [torch.full(s, float("nan"), dtype=BF, device="cuda") for s in ((E, H), (E, 2 * I, H), (E, H, I))]
    f.backward(dout, x, off, gu, dx=grads[0], dw1=grads[1], dw2=grads[2])
    assert all(bool(t.isfinite().all()) for t in grads)
    for e in (0, 1, 4097, E - 1):
        x64, d64 = du.f64(x[e: e + 1]), du.f64(dout[e: e + 1])
        refs = du.ffn_grad_bounds(d64, x64, du.f64(f.w1[e]), du.f64(f.w2[e]), "split", "silu", BF, F, BF, BF)
        for what, got, (ref, bound) in zip(("dx", "dw1", "dw2"), (grads[0][e: e + 1], grads[1][e], grads[2][e]), refs):
            du.assert_within(got, ref, bound, f"{what} of expert {e}")


def test_gradients_of_more_tokens_than_blocks():
    """A token's rows are summed by blocks that take several tokens from 2^22 on; forward takes as many."""
    T, E, H, I, rows = (1 << 22) + 77, 5, 8, 8, 3000
    g = torch.Generator().manual_seed(3)
    counts = [700, 0, 1300, 999, 1]
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    # every row is a token's only one (gather_div 1); the last tokens and those around 2^22 among them
    token = torch.randperm(T - 200, generator=g)[:rows]
    token[:200] = torch.arange(T - 200, T)
    token = token[torch.randperm(rows, generator=g)].to("cuda")
    dest = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    dest[token] = torch.arange(rows, dtype=torch.int32, device="cuda")
    f = mx.ExpertFFN(du.normal((E, 2 * I, H), H ** -0.5, BF, 1), du.normal((E, H, I), I ** -0.5, BF, 2))
    x = torch.zeros((T, H), dtype=BF, device="cuda")
    x[token] = du.normal((rows, H), 1.0, BF, 4)
    dout = du.normal((rows, H), 1.0, BF, 5)
    how = dict(gather=token.to(torch.int32), gather_div=1)
    out, gu = f.forward(x, off, save=True, **how)
    dx = torch.full((T, H), float("nan"), dtype=F, device="cuda")
    _, dw1, dw2 = f.backward(dout, x, off, gu, dest_row=dest, dx=dx, **how)
    plain = x[token]
    want, v1, v2 = f.backward(dout, plain, off, gu, dx=torch.empty((rows, H), dtype=F, device="cuda"))
    assert torch.equal(f.forward(plain, off), out) and torch.equal(dw1, v1) and torch.equal(dw2, v2)
    assert torch.equal(dx[token], want)
    dx[token] = 0.0
    assert not dx.any()
