"""The linear layer on different columns of one wider matrix: x, residual and y side by side."""
import pytest
import torch

from tests import plain_ops as P

pytestmark = pytest.mark.gpu


def _check(y, ref):
    r, bound = ref
    assert bool(((y.double() - r).abs() <= bound).all())


# few tokens; pairs of blocks, y leaving by TMA (N a multiple of 8, no residual) and not
@pytest.mark.parametrize("T,K,N", [(1, 64, 72), (5, 264, 200), (700, 136, 264), (1300, 200, 2050)])
@pytest.mark.parametrize("residual", [False, True])
def test_linear_columns_of_one_matrix(T, K, N, residual, cuda_dev):
    from paged_fp8_gated_b200 import binding
    g = torch.Generator(device="cuda").manual_seed(T + N)
    n8 = (N + 7) // 8 * 8
    wide = torch.randn(T, 8 + K + 2 * n8 + 8, generator=g, device="cuda").bfloat16()
    w = (torch.randn(N, K, generator=g, device="cuda") / K ** 0.5).bfloat16()
    before = wide.clone()
    x = wide[:, 8:8 + K]
    for lo in (8 + K, 8 + K + n8):                      # y right behind x, or with the residual between
        hi = 2 * (8 + K) + n8 - lo
        r = wide[:, hi:hi + N] if residual else None
        y = wide[:, lo:lo + N]
        binding.linear(x, w, residual=r, activation="silu", out=y)
        _check(y, P.linear(before[:, 8:8 + K], w, None, before[:, hi:hi + N] if residual else None, "silu"))
        keep = torch.ones(wide.shape[1], dtype=torch.bool, device="cuda")
        keep[lo:lo + N] = False
        assert torch.equal(wide[:, keep], before[:, keep])
        wide.copy_(before)
    y = wide[:, :8]                                     # and in front of x
    binding.linear(x, w[:8], out=y)
    _check(y, P.linear(before[:, 8:8 + K], w[:8]))


def test_linear_y_between_the_rows_of_w(cuda_dev):
    """One token's y in the columns behind w."""
    from paged_fp8_gated_b200 import binding
    wide = torch.randn(96, 64 + 104, device="cuda", generator=torch.Generator("cuda").manual_seed(2)).bfloat16()
    x = torch.randn(1, 64, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).bfloat16()
    w = wide[:, :64].clone()
    binding.linear(x, wide[:, :64], out=wide[7:8, 64:160])
    _check(wide[7:8, 64:160], P.linear(x, w))
    assert torch.equal(wide[:, :64], w)
