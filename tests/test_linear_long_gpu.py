"""16-bit results of very long sums: what the tensor cores cut off of a chain stays far
below the result's own rounding.

All values are positive, so the sum is its own magnitude.  A chain of 16-product steps is
off by at most 2^-23 of it a step; chains have at most 32,768 products, or are added up from
ones of 512 (32 steps and 8 more for the sums inside a step) rounding to nearest, which is
what this K needs: 2^-24 for each of the K / 512 additions and 8 for the clusters' ones."""
import pytest
import torch

pytestmark = pytest.mark.gpu


# pairs of blocks, a K range each; a cluster of eight blocks a tile
@pytest.mark.parametrize("T,K,N", [(2048, 1 << 19, 1184), (3, 1 << 21, 100)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_linear_long_sums_with_16_bit_results(T, K, N, dtype, cuda_dev):
    from paged_fp8_gated_b200 import binding
    g = torch.Generator(device="cuda").manual_seed(5)
    # products around 2^-2 x 2^-16: the sums stay below 8
    x = torch.rand(T, K, generator=g, device="cuda", dtype=torch.float32).mul_(2.0 ** -8).to(dtype)
    w = torch.rand(N, K, generator=g, device="cuda", dtype=torch.float32).mul_(2.0 ** -8).to(dtype)
    y = binding.linear(x, w)
    rows, cols = slice(0, T, max(1, T // 48)), slice(0, N, max(1, N // 48))
    ref = x[rows].double() @ w[cols].double().T
    long_sum = 40 * 2.0 ** -23 + (K / 512 + 8) * 2.0 ** -24
    half_step = torch.finfo(dtype).eps / 2
    err = (y[rows, cols].double() - ref).abs()
    assert float((err / ref).max()) <= long_sum + half_step * (1 + long_sum)
    assert binding.linear_status() == 0
