"""The selection's log-sum over long chains: many rows of a large vocabulary, so that a row
is one segment and a thread adds up thousands of exponentials.

Every difference d to the reference and from there to the maximum is at most `reach` in
magnitude here, so the log-sum is off by at most 2^-24 (2.5 x 2 reach) for the differences
and their scaling, 2 x (2^-22 + 2^-24) for the exponentials and the products with them, and
18 x 2^-24 for the sums (16 additions at most in fp32; the long ones keep what they round
off, but for 2).  Scores are chosen so that the best one is near 0, where rounding it to
fp32 adds nothing."""
import numpy as np
import pytest
import torch

from tests import plain_ops as P

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ROWS, V = 600, 1 << 22


def _bound(reach):
    return 2.0 ** -24 * (2.5 * 2 * reach + 18 + 2 * 5)


def _lse(row):
    x = row.double()
    m = x.max()
    return float(m + torch.log(torch.exp(x - m).sum()))


def _flat(level, dtype):
    """1,024 tokens at 0, the others at `level`: the same term again and again."""
    row = torch.full((V,), level, device="cuda", dtype=DT[dtype])
    row[:1024] = 0
    return row


@pytest.mark.parametrize("dtype,level", [("bf16", -1.3), ("bf16", -0.7), ("fp16", -1.3), ("fp32", -0.7)])
def test_beam_log_sum_of_a_long_row(dtype, level, cuda_dev):
    from paged_fp8_gated_b200 import binding
    row = _flat(level, dtype)
    lse = _lse(row)
    logits = row.expand(ROWS, 1, V).contiguous()
    scores = torch.full((ROWS, 1), lse, device="cuda")
    s, p, t = binding.beam_select(logits, scores, 2)
    exact = float(scores[0, 0].double()) - lse           # of token 0 (and 1), whose logit is 0
    assert bool((t == torch.arange(2, device="cuda")).all())
    assert bool((p == torch.arange(ROWS, device="cuda")[:, None]).all())
    assert float((s.double() - exact).abs().max()) <= _bound(1.3) + 2.0 ** -24 * abs(exact)


def test_beam_log_sum_of_a_rising_row(cuda_dev):
    """Logits that rise by 1 over the row: a new maximum in every group of a thread."""
    from paged_fp8_gated_b200 import binding
    row = torch.linspace(-1, 0, V, device="cuda", dtype=torch.float64).float()
    lse = _lse(row)
    logits = row.expand(ROWS, 1, V).contiguous()
    scores = torch.full((ROWS, 1), lse, device="cuda")
    s, _, t = binding.beam_select(logits, scores, 1)
    assert bool((t == row.argmax()).all())
    exact = float(scores[0, 0].double()) + float(row.max()) - lse
    assert float((s.double() - exact).abs().max()) <= _bound(1.0) + 2.0 ** -24 * abs(exact)


def test_beam_order_of_close_candidates(cuda_dev):
    """Two beams whose best candidates are 2.2 bounds apart come in the order of 64 bits."""
    from paged_fp8_gated_b200 import binding
    a, b = _flat(-1.3, "fp32"), _flat(-0.7, "fp32")
    la, lb = _lse(a), _lse(b)
    G, gap = ROWS // 2, 2.2 * _bound(1.3)
    logits = torch.stack([a, b]).expand(G, 2, V).contiguous()
    for first in (0, 1):                                 # which beam is ahead
        # scores near -lse' + a shared offset: exact to 2^-24 of about 1
        want = [gap, 0.0] if first == 0 else [0.0, gap]
        scores = torch.tensor([want[0] + (la - lb), want[1]], dtype=torch.float64).float().expand(G, 2)
        scores = scores.contiguous().cuda()
        exact = scores[0].double().cpu().numpy() - np.array([la, lb])
        assert (exact[0] > exact[1]) == (first == 0) and abs(exact[0] - exact[1]) > 2 * _bound(1.3)
        s, p, t = binding.beam_select(logits, scores, 1)
        assert bool((p.reshape(-1) == 2 * torch.arange(G, device="cuda") + first).all())
        assert bool((t == 0).all())


def test_beam_large_logits_and_scores(cuda_dev):
    """Logits of 1e4 and scores of 1e6: the log-sum's bound, and one rounding of the result."""
    from paged_fp8_gated_b200 import binding
    g = torch.Generator(device="cuda").manual_seed(40)
    logits = torch.randn(3, 4, 4097, generator=g, device="cuda") * 2
    scores = -torch.rand(3, 4, generator=g, device="cuda") * 8
    logits[0] *= 1e4
    logits[1] += 3e4
    scores[2] = torch.tensor([-1e6, -1e6, -2e6, 0.0], device="cuda")
    s, p, t = binding.beam_select(logits, scores, 4)
    rs, rp, rt = P.beam(logits, scores, 4)
    assert np.array_equal(p.cpu().numpy(), rp) and np.array_equal(t.cpu().numpy(), rt)
    assert (np.abs(s.cpu().numpy().astype(np.float64) - rs) <= 2.0 ** -24 * np.abs(rs) + 7e-6).all()


def test_beam_not_numbers_in_a_long_row(cuda_dev):
    """Infinities, NaN and masked stretches anywhere in a thread's chain."""
    from paged_fp8_gated_b200 import binding
    G, V1 = ROWS // 4, 300_001
    g = torch.Generator(device="cuda").manual_seed(41)
    logits = torch.randn(G, 4, V1, generator=g, device="cuda").bfloat16()
    logits[0, 0, V1 - 1] = float("nan")
    logits[1, 1, V1 // 2] = float("inf")
    logits[2, 2, : V1 - 5] = -float("inf")
    logits[3, 3] = -float("inf")
    logits[4, 0, 1000:] = torch.finfo(torch.bfloat16).min
    logits[5, 0, ::2] = torch.finfo(torch.bfloat16).max
    scores = -torch.rand(G, 4, generator=g, device="cuda")
    s, p, t = binding.beam_select(logits, scores, 4)
    rs, rp, rt = P.beam(logits[:8], scores[:8], 4)
    assert np.array_equal(p[:8].cpu().numpy(), rp) and np.array_equal(t[:8].cpu().numpy(), rt)
    live = rp >= 0
    err = np.abs(s[:8].cpu().numpy().astype(np.float64) - rs)[live]
    assert (err <= 2.0 ** -24 * np.abs(rs[live]) + 7e-6).all()
