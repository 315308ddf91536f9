"""Giving back the end of a row, as pages_free documents it: a verify block takes room for L
tokens, some of them stay, the others' pages go back to the pool."""
import numpy as np
import pytest
import torch

from tests import plain_ops as P

pytestmark = pytest.mark.gpu


def _shorten(binding, table, lens, refs, new, page_size, most):
    cols = torch.arange(most, device="cuda", dtype=torch.int32)
    keep, had = -(-new // page_size), -(-lens // page_size)
    tail = table.gather(1, (keep[:, None] + cols).clamp(0, table.shape[1] - 1).long())
    binding.pages_free(tail, (had - keep) * page_size, refs, page_size)
    lens.copy_(new)


@pytest.mark.parametrize("page_size,L", [(1, 8), (1, 1), (64, 8), (64, 65), (64, 200)])
def test_tokens_that_were_not_accepted_go_back(page_size, L, cuda_dev):
    """Against loops over rows and pages, in a pool that a leak would use up."""
    from paged_fp8_gated_b200 import binding
    rng = np.random.default_rng(page_size + L)
    rows, steps = 6, 20
    max_pages = -(-(steps * L // 2 + 2 * L) // page_size) + 2
    num_pages = rows * (-(-(steps * L // 2 + 2 * L) // page_size) + 1)
    ref = P.Pool(rows, max_pages, page_size, num_pages)
    ref.lens[:] = 0
    ref.lens[4] = -1                                     # an empty row gives nothing back
    table, lens, refs = (torch.from_numpy(a.copy()).cuda() for a in (ref.table, ref.lens, ref.refs))
    ws = binding.alloc_pages_workspace(rows, num_pages)
    most = -(-L // page_size) + 1
    for step in range(steps):
        before = ref.lens.copy()
        pos, loc = binding.pages_extend(table, lens, refs, page_size, L, workspace=ws)
        assert binding.step_status(ws) == 0
        rp, rl, short, over = ref.extend(L)
        assert not short and not over
        assert np.array_equal(loc.cpu().numpy(), rl) and np.array_equal(pos.cpu().numpy(), rp)
        # half of the tokens stay on average; none and all of them too
        stay = rng.integers(0, L + 1, rows) if step % 5 else np.full(rows, L * (step % 2))
        new = np.where(before < 0, -1, np.minimum(before + stay, (step + 1) * L // 2 + L)).astype(np.int32)
        new = np.maximum(new, np.where(before < 0, -1, before)).astype(np.int32)
        for r in range(rows):
            for j in range(-(-max(int(new[r]), 0) // page_size), ref.pages(r)):
                ref.refs[ref.table[r, j]] -= 1
        ref.lens[:] = new
        empty = lens < 0
        want = torch.from_numpy(new).cuda()
        _shorten(binding, table, lens, refs, want, page_size, most)
        assert torch.equal(lens < 0, empty)
        assert np.array_equal(refs.cpu().numpy(), ref.refs)
        assert int(refs.sum()) == sum(ref.pages(r) for r in range(rows))
        t = table.cpu().numpy()
        for r in range(rows):
            assert np.array_equal(t[r, :ref.pages(r)], ref.table[r, :ref.pages(r)])
