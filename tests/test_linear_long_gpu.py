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


# two and four pairs that share a tile, odd edges; the epilogue of a cluster's blocks
@pytest.mark.parametrize("T,K,N", [(512, 1 << 18, 1024), (250, 1 << 18, 1003), (385, (1 << 17) + 40, 515), (40, 1 << 19, 131)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_linear_long_sums_with_epilogue(T, K, N, dtype, cuda_dev):
    """Bias, activation and residual behind a long sum of either sign."""
    from paged_fp8_gated_b200 import binding
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(T, K, generator=g, device="cuda").to(dtype)
    w = (torch.randn(N, K, generator=g, device="cuda") / 64).to(dtype)
    b, r = (torch.randn(*s, generator=g, device="cuda").to(dtype) for s in ((N,), (T, N)))
    y = binding.linear(x, w, bias=b, residual=r, activation="silu")
    v = torch.empty(T, N, dtype=torch.float64, device="cuda")
    mag = torch.empty_like(v)
    for n0 in range(0, N, 128):                          # (64-bit copies of w a few rows at a time)
        wd = w[n0:n0 + 128].double()
        v[:, n0:n0 + 128] = x.double() @ wd.T
        mag[:, n0:n0 + 128] = x.double().abs() @ wd.abs().T
    v += b.double()
    ref = v * torch.sigmoid(v) + r.double()
    # the sum's error through a slope of at most 1.13, the epilogue's few fp32 steps
    err = 1.13 * (40 * 2.0 ** -23 + (K / 512 + 8) * 2.0 ** -24) * mag + 2.0 ** -20 * (v.abs() + r.double().abs())
    half_step = torch.finfo(dtype).eps / 2
    assert bool(((y.double() - ref).abs() <= err + half_step * (ref.abs() + err)).all())
    assert binding.linear_status() == 0
