"""gad_beam_select against a sort of every candidate in 64 bits.

Scores: one fp32 rounding of the result (2^-24 of it) plus the error of the
log-sum: exponentials of fp32 differences (2^-22 each from the exponential
itself, 2^-23 of the exponent from its scaling by log2 e, which is at most 2^-23
x 30 where a term still matters) and fp32 sums of 32 terms (2^-19 at most):
7e-6 in all.  Parents and tokens are equal."""
import math

import numpy as np
import pytest
import torch

from tests import plain_ops as P

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
INF = math.inf


def _check(logits, scores, K, finished=None, pad=0, **kw):
    from paged_fp8_gated_b200 import binding
    got = binding.beam_select(logits, scores, K, finished=finished, pad_token=pad, **kw)
    torch.cuda.synchronize()
    s, p, t = (o.cpu().numpy() for o in got)
    rs, rp, rt = P.beam(logits, scores, K, finished, pad)
    assert np.array_equal(p, rp) and np.array_equal(t, rt)
    live = rp >= 0
    assert (s[~live] == -np.inf).all()
    err = np.abs(s[live].astype(np.float64) - rs[live])
    assert (err <= 2.0 ** -24 * np.abs(rs[live]) + 7e-6).all(), err.max()
    return got


def _inputs(G, W, V, dtype, seed, scale=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = (torch.randn(G, W, V, generator=g, device="cuda") * scale).to(DT[dtype])
    return logits, -torch.rand(G, W, generator=g, device="cuda") * 8, g


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("G,W,V,K", [
    (1, 1, 1, 1), (1, 1, 5, 8), (2, 3, 7, 4), (1, 4, 2048, 4), (1, 4, 2049, 4), (3, 5, 1000, 10),
    (2, 8, 32001, 16), (5, 2, 8193, 3), (40, 8, 9001, 8), (64, 6, 16385, 12), (1, 64, 3001, 64),
    (2, 17, 20000, 33), (300, 1, 8200, 2)])
def test_beam_random(G, W, V, K, dtype, cuda_dev):
    logits, scores, _ = _inputs(G, W, V, dtype, G + W + V + K)
    _check(logits, scores, K)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("K", [1, 4, 16])
@pytest.mark.parametrize("V", [4, 9, 24, 40, 56, 72, 130, 700])
def test_beam_values_of_both_signs(V, K, dtype, cuda_dev):
    """Few places hold values, of both signs, large and tiny, so that the search for a
    bound may end anywhere: also between the last negative value and none."""
    G, W = 6, 2
    logits, scores, g = _inputs(G, W, V, dtype, V + K)
    runs = (torch.arange(V, device="cuda") // 8) % 2 * 2 - 1
    logits[:2] = logits[:2].abs() * runs                           # runs of either sign
    logits[2] = -logits[2].abs()
    logits[3] = logits[3] * (10.0 ** torch.randint(-4, 4, (W, V), generator=g, device="cuda")).to(logits.dtype)
    logits[4, :, V // 2:] = 0.0
    logits[4, :, : V // 4] = -0.0
    logits[5, 0] = -INF
    logits[5, 0, V // 2] = -1e-3
    scores[::2] = torch.tensor([5.0, -3.0], device="cuda")         # and totals of both signs
    _check(logits, scores, K)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [3001, 16400])
def test_beam_masks_finished_and_dead(V, dtype, cuda_dev):
    """Masked tokens, masks that leave one token or none, the type's lowest value as a mask,
    finished and dead beams, requests with fewer candidates than K."""
    G, W, K = 12, 4, 6
    logits, scores, g = _inputs(G, W, V, dtype, 11)
    logits[torch.rand(G, W, V, generator=g, device="cuda") < 0.5] = -INF
    logits[1] = -INF                         # nothing at all
    logits[2, 1:] = -INF
    logits[3] = -INF
    logits[3, 2, V - 1] = 0.5                # one token of one beam
    logits[4, :, 5:] = torch.finfo(DT[dtype]).min
    scores[5, 1:] = -INF                     # the first step: one live beam
    scores[6] = -INF
    scores[7, 2] = float("nan")
    finished = torch.zeros(G, W, dtype=torch.uint8, device="cuda")
    finished[8, 1] = 1
    finished[9] = 1
    finished[10, :3] = 1
    scores[10, 0] = -INF                     # finished and dead
    logits[11, :, :] = -INF
    finished[11, 3] = 1
    _check(logits, scores, K, finished, pad=V - 1)
    _check(logits, scores, K, finished.bool(), pad=0)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_beam_nan_and_infinity(dtype, cuda_dev):
    logits, scores, _ = _inputs(5, 3, 9000, dtype, 12)
    logits[0, 1, 8999] = float("nan")        # that beam has no log-sum: no candidates
    logits[1, :, 17] = float("nan")
    logits[2, 0, 4000] = INF
    logits[3] = float("nan")
    logits[4, 2, 8300:] = -INF
    logits[4, 2, 8400] = float("nan")        # a chunk of masked tokens and a NaN
    _check(logits, scores, 4)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V,K", [(1030, 5), (2500, 64), (20001, 9)])
def test_beam_ties_go_to_the_lowest_index(V, K, dtype, cuda_dev):
    """Equal logits and equal beams, whose rows start at different alignments (odd V);
    -0 and +0 are equal; more ties than the kernels' buffers hold."""
    W = 4
    for fill in ("constant", "few values", "signed zeros", "rows"):
        g = torch.Generator(device="cuda").manual_seed(3)
        if fill == "constant":
            x = torch.full((2, W, V), 0.25, device="cuda")
        elif fill == "few values":
            x = torch.randint(0, 3, (2, 1, V), generator=g, device="cuda").float().expand(2, W, V).contiguous()
        elif fill == "signed zeros":
            x = torch.zeros(2, W, V, device="cuda")
            x[..., ::3] = -0.0
        else:
            x = torch.randn(2, 1, V, generator=g, device="cuda").expand(2, W, V).contiguous()
        _check(x.to(DT[dtype]), torch.full((2, W), -1.5, device="cuda"), K)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_beam_row_strides_and_offsets(dtype, cuda_dev):
    G, W, V = 3, 4, 5000
    for lead, trail in ((0, 3), (1, 0), (5, 2), (3, 13)):
        logits, scores, _ = _inputs(G, W, V, dtype, 30 + lead)
        wide = torch.full((G, W, lead + V + trail), 60.0, device="cuda", dtype=DT[dtype])
        wide[..., lead:lead + V] = logits
        view = wide[..., lead:lead + V]
        a = _check(view, scores, 7)
        b = _check(logits, scores, 7)
        assert all(torch.equal(p, q) for p, q in zip(a, b))   # the same bits at any alignment


def test_beam_extreme_scores(cuda_dev):
    """Large logits and scores, and differences that underflow."""
    logits, scores, g = _inputs(3, 4, 4097, "fp32", 40)
    logits[0] *= 1e4
    logits[1] += 3e4
    scores[2] = torch.tensor([-1e6, -1e6, -2e6, 0.0], device="cuda")
    from paged_fp8_gated_b200 import binding
    s, p, t = binding.beam_select(logits, scores, 4)
    rs, rp, rt = P.beam(logits, scores, 4)
    assert np.array_equal(p.cpu().numpy(), rp) and np.array_equal(t.cpu().numpy(), rt)
    # the differences of the logits are rounded to fp32 once more: 2^-24 of up to 1e5
    assert (np.abs(s.cpu().numpy() - rs) <= 2.0 ** -23 * np.abs(rs) + 1e-2).all()


def test_beam_scores_that_are_not_finite(cuda_dev):
    """Beams whose score is infinite or NaN have no candidates, finished or not."""
    from paged_fp8_gated_b200 import binding
    logits, scores, _ = _inputs(3, 4, 3000, "bf16", 60)
    finished = torch.zeros(3, 4, dtype=torch.bool, device="cuda")
    scores[0, 1], scores[1, 0], scores[1, 3], scores[2, :] = INF, float("nan"), -INF, INF
    finished[1, 3] = finished[2, 0] = finished[0, 2] = True
    s, p, t = binding.beam_select(logits, scores, 5, finished=finished, pad_token=7)
    live = torch.where(scores.isfinite(), scores, -INF)
    rs, rp, rt = P.beam(logits, live, 5, finished, 7)
    assert np.array_equal(p.cpu().numpy(), rp) and np.array_equal(t.cpu().numpy(), rt)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_beam_offsets_past_32_bits(dtype, cuda_dev):
    """Rows 2^30 values apart, and the largest vocabulary."""
    from paged_fp8_gated_b200 import binding
    G, V, stride = (5, 3001, 1 << 30) if dtype == "bf16" else (3, 3001, 1 << 30)
    logits, scores, g = _inputs(G, 1, V, dtype, 70)
    big = torch.empty((G - 1) * stride + V, dtype=DT[dtype], device="cuda")
    view = big.as_strided((G, 1, V), (stride, stride, 1))
    view.copy_(logits)
    a = binding.beam_select(view, scores, 4)
    b = binding.beam_select(logits, scores, 4)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    del big, view
    V = 1 << 24
    x = torch.randn(1, 1, V, generator=g, device="cuda").to(DT[dtype])
    x[0, 0, [V - 1, 5, V // 2]] = torch.tensor([30.0, 31.0, 29.0], device="cuda", dtype=DT[dtype])
    s, p, t = binding.beam_select(x, torch.zeros(1, 1, device="cuda"), 3)
    assert t.tolist() == [[5, V - 1, V // 2]] and p.tolist() == [[0, 0, 0]]
    ref = torch.log_softmax(x.double().reshape(-1), 0)[[5, V - 1, V // 2]]
    assert bool(((s.double() - ref).abs() <= 2.0 ** -24 * ref.abs() + 7e-6).all())


def test_beam_workspace_poison_streams_and_graph(cuda_dev):
    from paged_fp8_gated_b200 import binding
    G, W, V, K = 4, 3, 12000, 5
    ins = [_inputs(G, W, V, "bf16", 50 + i)[:2] for i in range(2)]
    want = [binding.beam_select(a, b, K) for a, b in ins]
    ws = [binding.alloc_beam_workspace(G, W, V, K) for _ in range(2)]
    for w in ws:
        w.fill_(0xC3)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[binding.beam_select(*ins[k], K, workspace=ws[k], stream=streams[k]) for k in range(2)]
           for _ in range(6)]
    torch.cuda.synchronize()
    for pair in got:
        for k in range(2):
            assert all(torch.equal(a, b) for a, b in zip(pair[k], want[k]))
    x, s = ins[0][0].clone(), ins[0][1].clone()
    out = tuple(torch.empty_like(t) for t in want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.beam_select(x, s, K, out=out, workspace=ws[0])
    for k in (1, 0):
        x.copy_(ins[k][0])
        s.copy_(ins[k][1])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[k]))


def test_beam_refusals(cuda_dev):
    from paged_fp8_gated_b200 import binding
    logits, scores, _ = _inputs(2, 3, 100, "bf16", 1)
    G, W, V = logits.shape
    ws = binding.alloc_beam_workspace(2, 3, 100, 4)
    for kw, err in [
        (dict(logits=logits.to(torch.float64)), TypeError), (dict(logits=logits[0]), ValueError),
        (dict(logits=logits.transpose(1, 2)), ValueError), (dict(scores=scores[:1]), ValueError),
        (dict(scores=scores.double()), TypeError), (dict(K=0), binding.GadError), (dict(K=65), binding.GadError),
        (dict(pad_token=100), binding.GadError), (dict(pad_token=-1), binding.GadError),
        (dict(workspace=ws[:256]), binding.GadError), (dict(finished=scores), TypeError),
        (dict(workspace=ws[16:]), binding.GadError),
        (dict(K=3, out=(scores, *(torch.empty(2, 3, dtype=torch.int32, device="cuda") for _ in range(2)))),
         binding.GadError),
    ]:
        args = dict(dict(logits=logits, scores=scores, K=4), **kw)
        with pytest.raises(err):
            binding.beam_select(args.pop("logits"), args.pop("scores"), args.pop("K"), **args)
