"""gad_linear against the exact result in 64 bits (bound derived in plain_ops.linear)."""
import pytest
import torch

from tests import plain_ops as P

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _inputs(T, K, N, dtype, out, bias, residual, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rn(*s):
        return torch.randn(*s, generator=g, device="cuda")
    x, w = rn(T, K).to(DT[dtype]), (rn(N, K) / K ** 0.5).to(DT[dtype])
    return (x, w, rn(N).to(DT[dtype]) if bias else None, rn(T, N).to(DT[out]) if residual else None)


def _check(y, x, w, bias=None, residual=None, act="none"):
    ref, bound = P.linear(x, w, bias, residual, act, y.dtype)
    err = (y.double() - ref).abs()
    assert bool(y.isfinite().all())
    worst = float((err / bound).max())
    assert worst <= 1.0, f"worst error / bound {worst:.3f}"


# sizes around the tiles of both kernels: 128 weight rows, 16 to 256 tokens, 64
# values of K; 256 x 256 tiles for more tokens
SHAPES = [(1, 8, 1), (1, 64, 128), (1, 1024, 8192), (2, 72, 127), (5, 200, 129), (16, 4096, 640),
          (17, 64, 300), (33, 8192, 256), (64, 520, 4097), (100, 1000, 77), (129, 128, 128),
          (255, 264, 1000), (256, 64, 512), (257, 136, 513), (300, 8, 1), (600, 72, 1031),
          (2600, 200, 1000), (513, 64, 5001), (1025, 1096, 2304), (4000, 512, 4100)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("fp16", "fp32")])
def test_linear_shapes(shape, dtype, out, cuda_dev):
    from paged_fp8_gated_b200 import binding
    x, w, _, _ = _inputs(*shape, dtype, out, False, False, sum(shape))
    _check(binding.linear(x, w, out_dtype=DT[out]), x, w)
    assert binding.linear_status() == 0


@pytest.mark.parametrize("shape", [(3, 328, 200), (40, 2056, 1001), (1300, 136, 2050)], ids=str)
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype,out,bias,residual", [
    ("bf16", "bf16", True, True), ("fp16", "fp16", True, False), ("bf16", "fp32", False, True),
    ("fp16", "fp32", True, True)])
def test_linear_epilogues(shape, act, dtype, out, bias, residual, cuda_dev):
    from paged_fp8_gated_b200 import binding
    x, w, b, r = _inputs(*shape, dtype, out, bias, residual, 7 + sum(shape))
    _check(binding.linear(x, w, bias=b, residual=r, activation=act, out_dtype=DT[out]), x, w, b, r, act)


@pytest.mark.parametrize("T,N", [(9, 260), (1500, 2600)])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_linear_strides_and_in_place_residual(T, N, out, cuda_dev):
    """Operands that are columns of wider matrices (rows of y and residual at odd
    distances and addresses), y in place of the residual; nothing beside y is written."""
    from paged_fp8_gated_b200 import binding
    K = 200
    x, w, b, r = _inputs(T, K, N, "bf16", out, True, True, 5)
    xs, ws = torch.zeros(T, K + 24, device="cuda", dtype=x.dtype), torch.zeros(N, K + 8, device="cuda", dtype=x.dtype)
    xs[:, 8:K + 8], ws[:, :K] = x, w
    wide = torch.full((T + 2, N + 7), 9.0, device="cuda", dtype=r.dtype)
    y = wide[1:T + 1, 3:N + 3]
    y.copy_(r)
    binding.linear(xs[:, 8:K + 8], ws[:, :K], bias=b, residual=y, activation="silu", out=y)
    _check(y.contiguous(), x, w, b, r, "silu")
    assert bool((wide[0] == 9).all() and (wide[-1] == 9).all())
    assert bool((wide[:, :3] == 9).all() and (wide[:, N + 3:] == 9).all())
    z = torch.empty(T, N, device="cuda", dtype=r.dtype)   # and the aligned layout gives the same bits
    binding.linear(x, w, bias=b, residual=r, activation="silu", out=z)
    assert torch.equal(z, y)


def test_linear_matches_oproj_and_repeats(cuda_dev):
    """The projection kernel's case: the sums are the same numbers in another order, and a
    second call gives the same bits."""
    from paged_fp8_gated_b200 import binding
    x, w, _, _ = _inputs(32, 1024, 8192, "bf16", "bf16", False, False, 3)
    y = binding.linear(x, w)
    _check(y, x, w)
    _check(binding.oproj(x, w), x, w)
    for _ in range(3):
        assert torch.equal(binding.linear(x, w), y)


@pytest.mark.parametrize("shape", [(12, 1032, 700), (1400, 264, 2100)], ids=str)
def test_linear_nan_and_infinity_stay_in_their_rows(shape, cuda_dev):
    from paged_fp8_gated_b200 import binding
    T, K, N = shape
    x, w, _, _ = _inputs(*shape, "bf16", "bf16", False, False, 4)
    clean = binding.linear(x, w)
    x2 = x.clone()
    x2[T - 1, K - 1] = float("nan")
    x2[2, 0] = float("inf")
    y = binding.linear(x2, w)
    assert bool(y[T - 1].isnan().all()) and not bool(y[2].isfinite().any())
    keep = [i for i in range(T) if i not in (2, T - 1)]
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("shape", [(8, 1024, 1000), (1500, 200, 2304)], ids=str)
def test_linear_two_streams_and_graph(shape, cuda_dev):
    """Two calls at once on two streams, and a captured call replayed on new inputs."""
    from paged_fp8_gated_b200 import binding
    a = _inputs(*shape, "bf16", "bf16", True, True, 21)
    b = _inputs(*shape, "bf16", "bf16", True, True, 22)
    want = [binding.linear(q[0], q[1], bias=q[2], residual=q[3], activation="gelu") for q in (a, b)]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [[torch.empty_like(want[0]) for _ in range(8)] for _ in range(2)]
    for i in range(8):
        for k, (q, s) in enumerate(((a, s1), (b, s2))):
            binding.linear(q[0], q[1], bias=q[2], residual=q[3], activation="gelu", out=outs[k][i], stream=s)
    torch.cuda.synchronize()
    for k in range(2):
        for o in outs[k]:
            assert torch.equal(o, want[k])
    x, w, bi, r = (t.clone() for t in a)
    y = torch.empty_like(want[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.linear(x, w, bias=bi, residual=r, activation="gelu", out=y)
    for k, q in enumerate((a, b)):
        for t, v in zip((x, w, bi, r), q):
            t.copy_(v)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[k])


def test_linear_refusals(cuda_dev):
    from paged_fp8_gated_b200 import binding
    x, w, b, r = _inputs(4, 64, 96, "bf16", "bf16", True, True, 1)
    bad = [
        (dict(x=x.float()), TypeError), (dict(w=w.half()), TypeError), (dict(x=x[0]), ValueError),
        (dict(w=w[:, :56]), ValueError), (dict(bias=b[:-1]), ValueError), (dict(bias=b.float()), TypeError),
        (dict(residual=r.float()), TypeError), (dict(activation="tanh"), ValueError),
        (dict(out_dtype=torch.float16), TypeError), (dict(out=torch.empty(4, 95, device="cuda", dtype=x.dtype)), ValueError),
        (dict(x=x.cpu()), ValueError), (dict(w=w.t().contiguous().t()), ValueError),
        (dict(x=torch.randn(4, 60, device="cuda").to(x.dtype), w=torch.randn(96, 60, device="cuda").to(x.dtype)), None),
        (dict(residual=None, out=torch.as_strided(x, (4, 16), (16, 1)), w=w[:16], bias=None), None),
    ]
    for over, err in bad:
        kw = dict(dict(x=x, w=w, bias=b, residual=r), **over)
        with pytest.raises(err or binding.GadError):
            binding.linear(kw.pop("x"), kw.pop("w"), **kw)


# every form of the two kernels (a block or a cluster over K, pairs of 256 and 128
# columns, pairs that share a tile), for 16-bit results and for fp32 ones, which are
# promoted where the chains are long
FORMS = [(520, 72, 8200), (520, 2056, 4099), (1, 72, 65), (130, 2056, 8200), (1, 2056, 8200), (70, 2056, 8200),
         (1, 520, 65), (130, 8200, 2050), (1, 4104, 4099), (70, 4104, 2050), (1, 2056, 65), (1, 8200, 65),
         (300, 72, 2050), (300, 1000, 2050), (70, 72, 65), (100, 2056, 2050), (70, 200, 65), (70, 4104, 65),
         (1030, 520, 2050), (1030, 4104, 1001), (2100, 8200, 130)]


@pytest.mark.parametrize("shape", FORMS, ids=str)
def test_linear_forms(shape, cuda_dev):
    from paged_fp8_gated_b200 import binding
    x, w, b, r = _inputs(*shape, "fp16", "fp16", True, True, 11 + sum(shape))
    _check(binding.linear(x, w, bias=b, residual=r, activation="silu"), x, w, b, r, "silu")
    y = binding.linear(x, w, bias=b, residual=r.float(), activation="silu", out_dtype=torch.float32)
    _check(y, x, w, b, r.float(), "silu")
    assert binding.linear_status() == 0


@pytest.mark.parametrize("shape", [(3, 7, 5), (64, 1, 64), (5, 1001, 200), (260, 130, 2000), (300, 8193, 1000)], ids=str)
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("fp16", "fp32")])
def test_linear_what_lies_between_the_rows_is_not_read(shape, dtype, out, cuda_dev):
    """K that ends inside 16 bytes, NaN behind it in both operands."""
    from paged_fp8_gated_b200 import binding
    T, K, N = shape
    x, w, _, _ = _inputs(*shape, dtype, out, False, False, 17 + sum(shape))
    ld = (K + 7) // 8 * 8 + 8
    xs, ws = (torch.full((n, ld), float("nan"), device="cuda", dtype=x.dtype) for n in (T, N))
    xs[:, :K], ws[:, :K] = x, w
    _check(binding.linear(xs[:, :K], ws[:, :K], out_dtype=DT[out]), x, w)


# pairs' tiles that end inside y's rows and columns: 256 and 128 columns, alone and two
# or four pairs that share a tile
EDGES = [(1300, 136, 2049), (300, 328, 9001), (193, 2056, 8203), (129, 1032, 8201), (450, 1032, 2001),
         (250, 8200, 1003), (33, 520, 32001), (385, 72, 31), (1300, 136, 2056), (300, 328, 9008), (193, 2056, 8200),
         (161, 2056, 8200), (129, 1032, 8200), (450, 1032, 2008), (250, 8200, 1000), (33, 520, 32008), (385, 72, 24)]


@pytest.mark.parametrize("shape", EDGES, ids=str)
@pytest.mark.parametrize("dtype,bias,act", [("bf16", False, "none"), ("fp16", True, "gelu")])
def test_linear_rows_inside_wider_ones(shape, dtype, bias, act, cuda_dev):
    """y's rows at 16-byte distances inside wider ones: nothing beside y is written, and
    rows at odd distances get the same bits."""
    from paged_fp8_gated_b200 import binding
    T, K, N = shape
    x, w, b, _ = _inputs(*shape, dtype, dtype, bias, False, 13 + sum(shape))
    wide = torch.full((T + 2, (N + 7) // 8 * 8 + 16), 9.0, device="cuda", dtype=x.dtype)
    y = wide[1:T + 1, 8:N + 8]
    binding.linear(x, w, bias=b, activation=act, out=y)
    _check(y.contiguous(), x, w, b, None, act)
    assert bool((wide[0] == 9).all() and (wide[-1] == 9).all())
    assert bool((wide[:, :8] == 9).all() and (wide[:, N + 8:] == 9).all())
    odd = torch.full((T, N // 2 * 2 + 3), 9.0, device="cuda", dtype=x.dtype)
    binding.linear(x, w, bias=b, activation=act, out=odd[:, 1:N + 1])
    assert torch.equal(odd[:, 1:N + 1], y)
    assert bool((odd[:, 0] == 9).all() and (odd[:, N + 1:] == 9).all())
    assert binding.linear_status() == 0


@pytest.mark.parametrize("shape", FORMS, ids=str)
def test_linear_fp32_sums_do_not_lose_with_k(shape, cuda_dev):
    """A fp32 result's error does not grow with K: no chain is longer than 768 products
    (48 steps of 16, each cut off by at most 2^-23 of the magnitudes summed so far, and 8
    more for the sums inside a step), and the chains are added up rounding to nearest."""
    from paged_fp8_gated_b200 import binding
    x, w, _, _ = _inputs(*shape, "bf16", "fp32", False, False, 12 + sum(shape))
    y = binding.linear(x, w, out_dtype=torch.float32).double()
    mag = x.double().abs() @ w.double().abs().T
    bound = (56 * 2.0 ** -23 + (shape[1] / 512 + 8) * 2.0 ** -24) * mag
    assert bool(((y - x.double() @ w.double().T).abs() <= bound).all())


def test_linear_captured_behind_a_join(cuda_dev):
    """Captured behind work of two joined streams, which it must wait for."""
    from paged_fp8_gated_b200 import binding
    x, w, _, _ = _inputs(64, 2048, 2304, "bf16", "bf16", False, False, 31)
    want = binding.linear(x, w)
    xs, ws, y = torch.zeros_like(x), torch.zeros_like(w), torch.empty_like(want)
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            ws.copy_(w)
        xs.copy_(x)
        torch.cuda.current_stream().wait_stream(side)
        binding.linear(xs, ws, out=y)
    for _ in range(3):
        xs.zero_()
        ws.zero_()
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_linear_chain_of_dependent_calls(cuda_dev):
    """Each call reads what the one before wrote, the weights too: back to back they give
    what they give one at a time."""
    from paged_fp8_gated_b200 import binding
    x, w, _, _ = _inputs(64, 64, 64, "bf16", "bf16", False, False, 41)

    def chain(wait):
        a, b, every = x, w, []
        for _ in range(8):
            a = binding.linear(a, b)
            if wait:
                torch.cuda.synchronize()
            b = binding.linear(b, a)
            if wait:
                torch.cuda.synchronize()
            every += [a, b]
        return every
    want = chain(True)
    for _ in range(5):
        got = chain(False)
        torch.cuda.synchronize()
        # the same bits (towards the end the values outgrow the type: NaN compares too)
        assert all(torch.equal(p.view(torch.int16), q.view(torch.int16)) for p, q in zip(got, want))


@pytest.mark.parametrize("T,N", [(9, 70), (24_000, 264)])
def test_linear_offsets_past_32_bits(T, N, cuda_dev):
    """Rows of y and residual so far apart that their offsets pass 2^32 values."""
    from paged_fp8_gated_b200 import binding
    K, ld = 64, -(-(1 << 32) // (T - 1)) // 8 * 8 + 8
    x, w, b, r = _inputs(T, K, N, "bf16", "bf16", True, True, 51)
    big = torch.empty((T - 1) * ld + N, dtype=torch.bfloat16, device="cuda")
    y = big.as_strided((T, N), (ld, 1))
    y.copy_(r)
    binding.linear(x, w, bias=b, residual=y, out=y)
    assert torch.equal(y, binding.linear(x, w, bias=b, residual=r))
    binding.linear(x, w, bias=b, out=y)   # (by another way where rows are whole 16 bytes)
    assert torch.equal(y, binding.linear(x, w, bias=b))


@pytest.mark.parametrize("T,D", [(300, 512), (1024, 512), (700, 2048)])
def test_linear_many_tokens_read_what_the_call_before_left(T, D, cuda_dev):
    """The same with pairs' tiles, whose y leaves by TMA: a call reads the y of the one
    before it, which may still run when it starts, and adds to it in place."""
    from paged_fp8_gated_b200 import binding
    x, w, b, _ = _inputs(T, D, D, "bf16", "bf16", True, False, 43)

    def chain(wait):
        a, every = x, []
        for i in range(8):
            a = binding.linear(a, w, bias=b, activation="silu")
            if wait:
                torch.cuda.synchronize()
            every.append(a.clone())
            binding.linear(every[-1], w, residual=a, out=a)
            if wait:
                torch.cuda.synchronize()
            a = a / a.abs().max()
            every.append(a)
        return every
    want = chain(True)
    for _ in range(5):
        got = chain(False)
        torch.cuda.synchronize()
        assert all(bool(p.isfinite().all()) and torch.equal(p, q) for p, q in zip(got, want))
