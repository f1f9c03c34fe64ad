"""The dense operators' size queries on the CPU: 0 for sizes that no call takes, never a wrapped number."""
import pytest

mx = pytest.importorskip("mxfp4_weight_mixture_amd", reason="libmxmoe.so is not built")

TOP = 2 ** 31 - 1
WIDE, TOKENS = 1 << 18, 1 << 28   # the largest widths and token counts


@pytest.mark.parametrize("T,H,I", [(-1, 64, 32), (1, 0, 32), (1, 64, 0), (1, 64, TOP), (1, 64, 1 << 30), (1, TOP, 64),
                                   (TOP, 64, 64), (TOKENS + 1, 64, 64), (1, WIDE + 1, 64), (1, 64, WIDE + 1)])
def test_gated_ffn(T, H, I):
    assert mx.lib.moe_gated_ffn_workspace_size(T, H, I) == 0
    assert mx.lib.moe_gated_ffn_grad_workspace_size(T, H, I) == 0


@pytest.mark.parametrize("T,K,N,n,R", [(-1, 64, 64, 1, 8), (TOP, 64, 64, 1, 8), (1, TOP, 64, 1, 8), (1, 64, TOP, 1, 8),
                                       (1, 64, 64, -1, 8), (1, 64, 64, 65537, 8), (1, 64, 64, 1, 0),
                                       (1, 64, 64, 1, 257), (1, 64, 64, 1, TOP), (TOKENS + 1, 64, 64, 1, 8)])
def test_adapters(T, K, N, n, R):
    assert mx.lib.moe_adapter_workspace_size(T, K, N, n, R) == 0


def test_the_largest_sizes():
    assert mx.lib.moe_gated_ffn_workspace_size(1, WIDE, WIDE) >= 2 * WIDE
    assert mx.lib.moe_gated_ffn_workspace_size(TOKENS, 8, 8) >= 16 * TOKENS
    assert mx.lib.moe_gated_ffn_grad_workspace_size(TOKENS, 8, 8) >= 48 * TOKENS
    assert mx.lib.moe_adapter_workspace_size(TOKENS, 8, 8, 65536, 256) >= 1024 * TOKENS
