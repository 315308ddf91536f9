"""Arrays of one call that lie right behind one another in one buffer overlap nowhere: the
calls take them, and give what they give on arrays of their own."""
import pytest
import torch

pytestmark = pytest.mark.gpu


class Arena:
    """Tensors cut from one buffer without a gap (but for what alignment asks)."""

    def __init__(self, size=1 << 20):
        self.buf = torch.zeros(size, dtype=torch.uint8, device="cuda")
        self.at = 0

    def like(self, t, align=4):
        self.at = -(-self.at // align) * align
        n = t.numel() * t.element_size()
        out = self.buf[self.at:self.at + n].view(t.dtype).view(t.shape)
        out.copy_(t)
        self.at += n
        return out


def _pool(page_size):
    rows, max_pages, num_pages = 5, 7, 61
    lens = torch.tensor([3 * page_size, -1, 2 * page_size - page_size // 2, 0, page_size], dtype=torch.int32, device="cuda")
    n = (lens.clamp(min=0) + page_size - 1) // page_size
    table = torch.full((rows, max_pages), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(num_pages, dtype=torch.int32, device="cuda")
    ids = torch.randperm(num_pages, generator=torch.Generator().manual_seed(page_size)).int().cuda()
    at = 0
    for r in range(rows):
        k = int(n[r])
        table[r, :k] = ids[at:at + k]
        refs[ids[at:at + k].long()] = 1
        at += k
    return table, lens, refs


@pytest.mark.parametrize("page_size", [1, 64])
def test_pages_arrays_side_by_side(page_size, cuda_dev):
    from paged_fp8_gated_b200 import binding as B

    def run(own):
        place = (lambda t, align=4: t.clone()) if own else Arena().like
        t0, l0, r0 = _pool(page_size)
        i32 = lambda *s: torch.full(s, -7, dtype=torch.int32, device="cuda")   # noqa: E731
        i64 = lambda *s: torch.full(s, -7, dtype=torch.int64, device="cuda")   # noqa: E731
        refs, table, lens = place(r0, 16), place(t0), place(l0)
        parent = place(torch.tensor([0, 0, 2, 2, -1, 4], dtype=torch.int32, device="cuda"))
        fork = tuple(place(i32(*s)) for s in ((6, 7), (6,), (6,), (6,)))
        pos, loc = place(i64(18), 8), place(i64(18), 8)
        src, dst, used, leave = place(i32(9)), place(i32(9)), place(i32(1)), place(
            torch.tensor([1, 0, 0, 1, 0, 1], dtype=torch.uint8, device="cuda"))
        ws = place(torch.zeros(B.pages_workspace_bytes(6, 61), dtype=torch.uint8, device="cuda"), 256)
        B.pages_fork(table, lens, parent, refs, page_size, out=fork, workspace=ws)
        assert B.step_status(ws) == 0
        B.pages_extend(fork[0], fork[1], refs, page_size, 3, out=(pos, loc), workspace=ws)
        assert B.step_status(ws) == 0
        B.pages_free(fork[0], fork[1], refs, page_size, leave=leave)
        B.pages_compact(fork[0], fork[1], refs, page_size, 9, out=(src, dst, used), workspace=ws)
        torch.cuda.synchronize()
        return refs, table, lens, *fork, pos, loc, src, dst, used

    for a, b in zip(run(True), run(False)):
        assert torch.equal(a, b)


def test_beam_arrays_side_by_side(cuda_dev):
    from paged_fp8_gated_b200 import binding as B
    G, W, V, K = 3, 4, 777, 5
    logits = torch.randn(G, W, V, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).bfloat16()
    scores = torch.zeros(G, W, device="cuda")
    fin = (torch.arange(G * W, device="cuda") % 5 == 0).reshape(G, W).to(torch.uint8)
    want = B.beam_select(logits, scores, K, finished=fin, pad_token=3)
    a = Arena()
    s = a.like(scores)
    out = tuple(a.like(torch.zeros_like(t)) for t in want)
    f, x = a.like(fin), a.like(logits, 2)
    ws = a.like(torch.zeros(B.beam_workspace_bytes(G, W, V, K), dtype=torch.uint8, device="cuda"), 256)
    B.beam_select(x, s, K, finished=f, pad_token=3, out=out, workspace=ws)
    assert all(torch.equal(p, q) for p, q in zip(out, want))
