"""The page operations against loops over rows and pages (plain_ops.Pool): tables,
lengths, counts, positions, cache rows and copied bytes are equal."""
import numpy as np
import pytest
import torch

from tests import plain_ops as P

pytestmark = pytest.mark.gpu


def _dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


class Both:
    """The same pool on the GPU and in plain loops, with caches that hold what each
    token's row should contain."""

    def __init__(self, rows, max_pages, page_size, num_pages, caches=2, row_bytes=128):
        from paged_fp8_gated_b200 import binding
        self.b = binding
        self.ref = P.Pool(rows, max_pages, page_size, num_pages)
        self.ps, self.num_pages = page_size, num_pages
        self.upload()
        self.ws = binding.alloc_pages_workspace(4096, num_pages)
        self.ws.fill_(0x5A)
        hkv = row_bytes // 64
        self.caches = [torch.randint(0, 256, (num_pages, page_size, hkv, 64), device="cuda", dtype=torch.uint8)
                       for _ in range(caches)]
        self.ref_caches = [c.cpu().numpy().copy() for c in self.caches]

    def upload(self):
        self.table, self.lens, self.refs = _dev(self.ref.table), _dev(self.ref.lens), _dev(self.ref.refs)

    def same(self):
        """Entries that count are equal (those behind a row's last page need not be)."""
        t = self.table.cpu().numpy()
        assert np.array_equal(self.lens.cpu().numpy(), self.ref.lens)
        assert np.array_equal(self.refs.cpu().numpy(), self.ref.refs)
        for r in range(len(self.ref.lens)):
            n = self.ref.pages(r)
            assert np.array_equal(t[r, :n], self.ref.table[r, :n]), r
        for c, rc in zip(self.caches, self.ref_caches):
            assert np.array_equal(c.cpu().numpy(), rc)

    def counts_hold(self):
        held = np.zeros(self.num_pages, np.int64)
        for r in range(len(self.ref.lens)):
            np.add.at(held, self.ref.table[r, :self.ref.pages(r)], 1)
        assert np.array_equal(held, self.ref.refs)

    def copy(self, src, dst):
        self.b.pages_copy(self.caches, src, dst)
        s, d = src.cpu().numpy(), dst.cpu().numpy()
        for rc in self.ref_caches:
            ok = (s >= 0) & (d >= 0)
            rc[d[ok]] = rc[s[ok]]

    def fork(self, parent):
        parent = np.asarray(parent)
        t, l, s, d = self.b.pages_fork(self.table, self.lens, _dev(parent), self.refs, self.ps, workspace=self.ws)
        rs, rd, short = self.ref.fork([int(p) for p in parent])
        assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(d.cpu().numpy(), rd)
        assert self.b.step_status(self.ws) == (self.b.STATUS_PAGES_POOL if short else 0)
        self.table, self.lens = t, l
        self.copy(s, d)
        return short

    def extend(self, L):
        pos, loc = self.b.pages_extend(self.table, self.lens, self.refs, self.ps, L, workspace=self.ws)
        rp, rl, short, over = self.ref.extend(L)
        assert np.array_equal(pos.cpu().numpy(), rp) and np.array_equal(loc.cpu().numpy(), rl)
        want = (self.b.STATUS_PAGES_POOL if short else 0) | (self.b.STATUS_PAGES_ROW if over else 0)
        assert self.b.step_status(self.ws) == want
        return short or over

    def free(self, leave):
        leave = np.asarray(leave)
        self.b.pages_free(self.table, self.lens, self.refs, self.ps,
                          leave=None if leave.all() else _dev(leave, torch.uint8))
        self.ref.free(leave)

    def compact(self, max_moves=None):
        s, d, u = self.b.pages_compact(self.table, self.lens, self.refs, self.ps, max_moves, workspace=self.ws)
        rs, rd, ru = self.ref.compact(max(1, self.num_pages // 2) if max_moves is None else max_moves)
        assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(d.cpu().numpy(), rd) and int(u) == ru
        assert self.b.step_status(self.ws) == 0
        self.copy(s, d)


@pytest.mark.parametrize("page_size", [1, 64])
@pytest.mark.parametrize("rows,max_pages,num_pages", [(1, 3, 4), (7, 9, 40), (33, 70, 700), (300, 13, 5000)])
def test_pages_random_walk(rows, max_pages, num_pages, page_size, cuda_dev):
    """Rounds of admitting, extending, forking, freeing and compacting, into full rows and
    full pools."""
    rng = np.random.default_rng(rows + page_size)
    b = Both(rows, max_pages, page_size, num_pages)
    full = 0
    for step in range(25):
        empty = np.nonzero(b.ref.lens < 0)[0]
        if len(empty):                                   # admit: an empty row starts at length 0
            b.ref.lens[rng.choice(empty, rng.integers(1, len(empty) + 1), replace=False)] = 0
            b.lens.copy_(_dev(b.ref.lens))
        L = int(rng.integers(1, 9 if page_size == 1 else 150))
        if b.extend(min(L, 2 * max_pages * page_size)):
            full += 1
            b.free(rng.random(rows) < 0.6)
        b.same()
        parent = np.where(rng.random(rows) < 0.5, np.arange(rows), rng.integers(-2, rows + 2, rows))
        full += b.fork(parent)
        b.same()
        b.counts_hold()
        if step % 3 == 2:
            b.compact(None if step % 2 else int(rng.integers(1, 9)))
            b.same()
            b.counts_hold()
    if num_pages <= 40:
        assert full > 0      # the walk reached full rows or pools
    b.free(np.ones(rows, bool))
    b.same()
    assert int(b.refs.abs().sum()) == 0


def test_pages_fork_shapes(cuda_dev):
    """One prompt into many rows, fewer rows out than in, partial pages to the first child,
    a pool without a page left."""
    b = Both(3, 10, 64, 24)
    b.ref.lens[:] = (130, 64, 0)
    b.ref.table[0, :3], b.ref.table[1, 0] = (20, 3, 7), 11
    b.ref.refs[[20, 3, 7, 11]] = 1
    b.upload()
    assert not b.fork([0] * 6 + [1, 1, 2, 2, -1, 3, 1 << 30, -(1 << 31)])
    b.same()
    b.counts_hold()
    assert int(b.refs[20]) == 6 and int(b.refs[11]) == 2
    assert not b.fork([5, 6])
    b.same()
    assert b.ref.lens.tolist() == [130, 64]
    assert b.fork([0] * 40)                              # 21 free pages for 39 rows
    b.same()
    b.counts_hold()
    assert (b.ref.lens == 128).sum() == 39 - 21


@pytest.mark.parametrize("page_size", [1, 64])
def test_pages_large_pool(page_size, cuda_dev):
    """More than one chunk of the pool for every block, rows longer than a block's columns."""
    rng = np.random.default_rng(5)
    num_pages = 5_000_003 if page_size == 1 else 300_001
    rows, max_pages = 6, 30_001 if page_size == 1 else 5000
    b = Both(rows, max_pages, page_size, num_pages, caches=0)
    pool = rng.permutation(num_pages)
    lens = rng.integers(1, (max_pages - 20) * page_size, rows)
    at = 0
    for r in range(rows):
        n = -(-int(lens[r]) // page_size)
        b.ref.table[r, :n] = pool[at:at + n]
        at += n
    b.ref.lens[:] = lens
    b.ref.refs[pool[:at]] = 1
    blocked = pool[at:at + num_pages // 2]               # held from outside the table
    b.ref.refs[blocked] = 3
    b.upload()
    b.caches = [torch.zeros(num_pages, 16, dtype=torch.uint8, device="cuda")]
    b.ref_caches = [b.caches[0].cpu().numpy()]
    b.extend(5)
    b.same()
    b.fork([0, 0, 1, 4, 4, 4])
    b.same()
    b.free([1, 0, 0, 1, 0, 0])
    b.extend(11)
    b.same()
    b.compact(1000)
    b.same()


def test_pages_fork_and_extend_4096_rows(cuda_dev):
    rng = np.random.default_rng(9)
    b = Both(4096, 6, 64, 30_000, caches=0)
    b.caches, b.ref_caches = [torch.zeros(30_000, 16, dtype=torch.uint8, device="cuda")], [np.zeros((30_000, 16), np.uint8)]
    b.ref.lens[:] = rng.integers(-1, 1, 4096)
    b.upload()
    b.extend(70)
    b.same()
    b.fork(rng.integers(-1, 4096, 4096))
    b.same()
    b.counts_hold()
    b.extend(64)
    b.same()


def test_pages_extend_prefill_block(cuda_dev):
    """A block of 65,536 tokens beside an empty row and a row in the middle of a page."""
    b = Both(3, 1100, 64, 4000, caches=0)
    b.ref.lens[:] = (0, -1, 63)
    b.ref.table[2, 0] = 3999
    b.ref.refs[3999] = 1
    b.upload()
    assert not b.extend(65_536)
    b.same()


@pytest.mark.parametrize("page_bytes", [16, 48, 128, 1024, 2048, 2064, 8192, 65_536, 65_552])
def test_pages_copy_sizes(page_bytes, cuda_dev):
    """Pages of any multiple of 16 bytes, 70 caches (more than one launch), pairs to skip,
    the pool's first and last pages; other pages keep their bytes."""
    from paged_fp8_gated_b200 import binding
    n, num_pages = 37, 90
    g = torch.Generator(device="cuda").manual_seed(page_bytes)
    caches = [torch.randint(0, 256, (num_pages, page_bytes), generator=g, device="cuda", dtype=torch.uint8)
              for _ in range(70 if page_bytes <= 2064 else 3)]
    want = [c.clone() for c in caches]
    ids = np.random.default_rng(page_bytes).permutation(num_pages)
    src, dst = ids[:n].astype(np.int32), ids[n:2 * n].astype(np.int32)
    src[3], dst[5], src[8], dst[9] = -1, -1, num_pages, num_pages + 5
    for w in want:
        for s, d in zip(src, dst):
            if 0 <= s < num_pages and 0 <= d < num_pages:
                w[d] = w[s]
    binding.pages_copy(caches, _dev(src), _dev(dst))
    assert all(torch.equal(c, w) for c, w in zip(caches, want))
    binding.pages_copy(caches, _dev(src[:0]), _dev(dst[:0]))   # no pairs: nothing to do


def test_pages_copy_past_32_bits(cuda_dev):
    """A cache of more than 2^32 bytes."""
    from paged_fp8_gated_b200 import binding
    num_pages, page_bytes = 600_000, 8192
    c = torch.empty(num_pages, page_bytes, dtype=torch.uint8, device="cuda")
    c[1], c[num_pages - 1] = 7, 9
    src, dst = _dev(np.array([1, num_pages - 1], np.int32)), _dev(np.array([num_pages - 2, 0], np.int32))
    binding.pages_copy([c], src, dst)
    assert bool((c[num_pages - 2] == 7).all() and (c[0] == 9).all())


def test_pages_bad_ids_are_skipped(cuda_dev):
    """Ids outside the pool in tables, and lengths past the table, touch nothing."""
    from paged_fp8_gated_b200 import binding
    table = torch.tensor([[0, -5, 1 << 30, 3], [2, 2, 2, 2]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([256, 1 << 30], dtype=torch.int32, device="cuda")
    refs = torch.tensor([1, 0, 4, 1, 0, 0, 0, 0], dtype=torch.int32, device="cuda")
    t, l, s, d = binding.pages_fork(table, lens, torch.tensor([0, 0, 1], dtype=torch.int32, device="cuda"), refs, 64)
    assert refs.tolist() == [2, 0, 4, 2, 0, 0, 0, 0] and torch.equal(t[1], table[0])
    s2, d2, used = binding.pages_compact(t, l, refs, 64)
    assert int(used) == 3 and s2.tolist() == [3, -1, -1, -1] and d2.tolist() == [1, -1, -1, -1]
    assert t[0].tolist() == [0, -5, 1 << 30, 1]
    binding.pages_free(t, l, refs, 64)
    assert refs.tolist() == [0] * 8 and l.tolist() == [-1] * 3


def test_pages_graph_and_streams(cuda_dev):
    """A captured fork + copy + extend replays on changed inputs; two pools on two streams."""
    from paged_fp8_gated_b200 import binding
    rng = np.random.default_rng(2)

    def pool(seed):
        r = np.random.default_rng(seed)
        b = Both(8, 40, 64, 200)
        b.ref.lens[:] = r.integers(1, 900, 8)
        pages = r.permutation(200)
        at = 0
        for i in range(8):
            n = b.ref.pages(i)
            b.ref.table[i, :n] = pages[at:at + n]
            at += n
        b.ref.refs[pages[:at]] = 1
        b.upload()
        return b

    a, c = pool(1), pool(2)
    parents = [rng.integers(0, 8, 8) for _ in range(4)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    par = [_dev(p) for p in parents]
    torch.cuda.synchronize()
    outs = []
    for k, (b, s) in enumerate(((a, streams[0]), (c, streams[1]))):
        with torch.cuda.stream(s):
            t, l, cs, cd = binding.pages_fork(b.table, b.lens, par[k], b.refs, 64, workspace=b.ws)
            binding.pages_copy(b.caches, cs, cd)
            outs.append((t, l, binding.pages_extend(t, l, b.refs, 64, 3, workspace=b.ws)))
    torch.cuda.synchronize()
    for k, b in enumerate((a, c)):
        s, d, _ = b.ref.fork([int(p) for p in parents[k]])
        for rc in b.ref_caches:
            rc[d[d >= 0]] = rc[s[d >= 0]]
        pos, loc, _, _ = b.ref.extend(3)
        b.table, b.lens = outs[k][0], outs[k][1]
        b.same()
        assert np.array_equal(outs[k][2][0].cpu().numpy(), pos)
        assert np.array_equal(outs[k][2][1].cpu().numpy(), loc)

    b = pool(3)
    table, lens, parent = b.table.clone(), b.lens.clone(), par[2].clone()
    out = (torch.full_like(table, -1), *(torch.empty_like(lens) for _ in range(3)))
    tok = tuple(torch.empty(8 * 3, dtype=torch.int64, device="cuda") for _ in range(2))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.pages_fork(table, lens, parent, b.refs, 64, out=out, workspace=b.ws)
        binding.pages_copy(b.caches, out[2], out[3])
        binding.pages_extend(out[0], out[1], b.refs, 64, 3, out=tok, workspace=b.ws)
    for k in (2, 3):                         # a beam loop: the new rows become the old ones
        parent.copy_(par[k])
        g.replay()
        s, d, _ = b.ref.fork([int(p) for p in parents[k]])
        for rc in b.ref_caches:
            rc[d[d >= 0]] = rc[s[d >= 0]]
        pos, loc, _, _ = b.ref.extend(3)
        b.table, b.lens = out[0], out[1]
        b.same()
        assert np.array_equal(tok[1].cpu().numpy(), loc) and np.array_equal(tok[0].cpu().numpy(), pos)
        table.copy_(out[0])
        lens.copy_(out[1])


def test_pages_refusals(cuda_dev):
    from paged_fp8_gated_b200 import binding
    table = torch.zeros(4, 8, dtype=torch.int32, device="cuda")
    lens = torch.zeros(4, dtype=torch.int32, device="cuda")
    refs = torch.zeros(64, dtype=torch.int32, device="cuda")
    par = torch.zeros(4, dtype=torch.int32, device="cuda")
    ws = binding.alloc_pages_workspace(4, 64)
    E = binding.GadError
    for call, err in [
        (lambda: binding.pages_fork(table, lens, par, refs, 16), E),
        (lambda: binding.pages_fork(table, lens, par, refs, 64, out=(table, *(torch.empty_like(lens) for _ in range(3)))), E),
        (lambda: binding.pages_fork(table, lens, par, refs, 64, workspace=ws[:512]), E),
        (lambda: binding.pages_fork(table, lens, par.long(), refs, 64), TypeError),
        (lambda: binding.pages_fork(table, lens[:3], par, refs, 64), ValueError),
        (lambda: binding.pages_fork(table, lens, par[:0], refs, 64), E),
        (lambda: binding.pages_extend(table, lens, refs, 64, 0), E),
        (lambda: binding.pages_extend(table, lens, refs, 64, 65_537), E),
        (lambda: binding.pages_extend(table, lens, refs[1:], 64, 1), E),
        (lambda: binding.pages_extend(table.t(), lens, refs, 64, 1), ValueError),
        (lambda: binding.pages_free(table, lens, refs, 64, leave=par), TypeError),
        (lambda: binding.pages_compact(table, lens, refs, 64, 0), E),
        (lambda: binding.pages_compact(table, lens, refs, 2, 1), E),
        (lambda: binding.pages_copy([], par, par), ValueError),
        (lambda: binding.pages_copy([torch.zeros(4, 24, dtype=torch.uint8, device="cuda")], par, par), E),
        (lambda: binding.pages_copy([table], par, par), TypeError),
    ]:
        with pytest.raises(err):
            call()
