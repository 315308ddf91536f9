"""The operators together, as a beam search uses them: projection, attention step over
the forked pages, output projection with residual, vocabulary logits, selection, fork,
page copy, room for the next token.  Beside it every beam's cache is kept as a plain
list of rows that nothing shares, and the attention step is repeated on those."""
import numpy as np
import pytest
import torch

from paged_fp8_gated_b200 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page_size,window", [(64, 0), (1, 0), (64, 48)])
def test_beam_search_over_the_paged_cache(page_size, window, cuda_dev):
    from paged_fp8_gated_b200 import binding as B
    G, K, V, H, steps = 3, 4, 1003, 512, 12
    g = torch.Generator(device="cuda").manual_seed(page_size + window)

    def weight(n, k):
        return (torch.randn(n, k, generator=g, device="cuda") / k ** 0.5).bfloat16()
    emb, w_qkv, w_o, w_v = weight(V, H) * 30, weight(W.QKV_COLS, H), weight(H, 1024), weight(V, H) * 3
    prompt = [70, 1, 130]
    num_pages, max_pages = (1200, 256) if page_size == 1 else (60, 6)
    scale = torch.ones(1, device="cuda")
    kc, vc = (torch.zeros(num_pages, page_size, 2, 64, dtype=torch.uint8, device="cuda") for _ in range(2))
    refs = torch.zeros(num_pages, dtype=torch.int32, device="cuda")
    table = torch.full((G, max_pages), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(G, dtype=torch.int32, device="cuda")
    ws = B.alloc_pages_workspace(G * K, num_pages)

    def attend(h, table, lens, refs, L):
        pos, loc = B.pages_extend(table, lens, refs, page_size, L, workspace=ws)
        assert B.step_status(ws) == 0
        qkv = B.linear(h, w_qkv)
        out = B.attn_decode(qkv, pos, None, table, loc, kc, vc, scale, scale, page_size, window, True, L=L)
        return qkv, pos, loc, B.linear(out.reshape(-1, 1024), w_o, residual=h), out

    # prompts of different lengths, one by one through blocks of one request
    hist = []                                  # per row: (K rows, V rows) that it has cached
    last = []
    for i, n in enumerate(prompt):
        toks = torch.randint(0, V, (n,), generator=g, device="cuda")
        t1, l1 = table[i:i + 1], lens[i:i + 1]
        done = 0
        rows_k, rows_v = [], []
        while done < n:
            L = min(8, n - done)
            _, _, loc, y, _ = attend(emb[toks[done:done + L]], t1, l1, refs, L)
            rows_k.append(kc.reshape(-1, 128)[loc].cpu().numpy())
            rows_v.append(vc.reshape(-1, 128)[loc].cpu().numpy())
            done += L
        hist.append((np.concatenate(rows_k), np.concatenate(rows_v)))
        last.append(y[-1:])
    assert lens.tolist() == prompt
    logits = B.linear(torch.cat(last), w_v, out_dtype=torch.float32).reshape(G, 1, V)
    scores = torch.zeros(G, 1, device="cuda")

    for step in range(steps):
        scores, parent, token = B.beam_select(logits, scores, K)
        assert bool((scores[:, :-1] >= scores[:, 1:]).all()) and bool((parent >= 0).all())
        table, lens, src, dst = B.pages_fork(table, lens, parent, refs, page_size, workspace=ws)
        assert B.step_status(ws) == 0
        B.pages_copy([kc, vc], src, dst)
        par = parent.reshape(-1).cpu().numpy()
        hist = [tuple(a.copy() for a in hist[p]) for p in par]
        h = emb[token.reshape(-1).long()]
        before = lens.clone()
        qkv, pos, loc, y, out = attend(h, table, lens, refs, 1)
        assert torch.equal(pos, before.long())
        new_k, new_v = (c.reshape(-1, 128)[loc].cpu().numpy() for c in (kc, vc))
        hist = [(np.concatenate([k, new_k[r:r + 1]]), np.concatenate([v, new_v[r:r + 1]]))
                for r, (k, v) in enumerate(hist)]
        logits = B.linear(y, w_v, out_dtype=torch.float32).reshape(G, K, V)
        if step % 4 == 3:                      # now and then the pool is moved together
            src, dst, used = B.pages_compact(table, lens, refs, page_size, workspace=ws)
            B.pages_copy([kc, vc], src, dst)
            assert int((refs != 0).sum()) == int(used) and not bool((refs[int(used):] != 0).any())

        # every row reads exactly its own history through the table
        tab, ln = table.cpu().numpy(), lens.cpu().numpy()
        for r, (k, v) in enumerate(hist):
            assert ln[r] == len(k)
            i = np.arange(len(k))
            rows = torch.from_numpy(tab[r, i // page_size].astype(np.int64) * page_size + i % page_size).cuda()
            assert np.array_equal(kc.reshape(-1, 128)[rows].cpu().numpy(), k)
            assert np.array_equal(vc.reshape(-1, 128)[rows].cpu().numpy(), v)
        # and the step on caches of its own, page after page, gives the same bits
        per = -(-int(ln.max()) // page_size)
        own_k, own_v = (torch.zeros(len(hist) * per, page_size, 2, 64, dtype=torch.uint8, device="cuda")
                        for _ in range(2))
        for c, which in ((own_k, 0), (own_v, 1)):
            flat = c.reshape(len(hist), per * page_size, 128)
            for r in range(len(hist)):
                flat[r, :ln[r]] = torch.from_numpy(hist[r][which]).cuda()
        own_table = torch.arange(len(hist) * per, dtype=torch.int32, device="cuda").reshape(len(hist), per)
        own_loc = torch.arange(len(hist), device="cuda") * (per * page_size) + pos
        own = B.attn_decode(qkv, pos, None, own_table, own_loc, own_k, own_v, scale, scale, page_size, window,
                            True)
        assert torch.equal(own, out)

    B.pages_free(table, lens, refs, page_size)
    assert int(refs.abs().sum()) == 0 and lens.tolist() == [-1] * (G * K)
    assert B.linear_status() == 0


@pytest.mark.parametrize("page_size", [1, 64])
def test_step_with_empty_rows(page_size, cuda_dev):
    """Rows without a request in the batch: the step writes no cache row for them, and the
    other rows' outputs are those of a batch without them."""
    from paged_fp8_gated_b200 import binding as B
    from tests import helpers as H
    R, num_pages, max_pages = 5, 600 if page_size == 1 else 12, 120 if page_size == 1 else 3
    g = torch.Generator(device="cuda").manual_seed(9)
    scale = torch.ones(1, device="cuda")
    live = [1, 3, 4]
    outs = {}
    for rows in (list(range(R)), live):
        kc, vc = (torch.zeros(num_pages, page_size, 2, 64, dtype=torch.uint8, device="cuda") for _ in range(2))
        refs = torch.zeros(num_pages, dtype=torch.int32, device="cuda")
        table = torch.full((len(rows), max_pages), -1, dtype=torch.int32, device="cuda")
        lens = torch.tensor([0 if r in live else -1 for r in rows], dtype=torch.int32, device="cuda")
        g.manual_seed(9)
        for step, L in enumerate((8, 8, 1, 5, 1)):
            qkv = torch.randn(R, L, W.QKV_COLS, generator=g, device="cuda").bfloat16()[rows].reshape(-1, W.QKV_COLS)
            pos, loc = B.pages_extend(table, lens, refs, page_size, L)
            out = B.attn_decode(qkv, pos, None, table, loc, kc, vc, scale, scale, page_size, 0, True, L=L)
            outs.setdefault(step, []).append(out[[rows.index(r) for r in live]].float())
        assert int((refs != 0).sum()) == sum(-(-23 // page_size) for _ in live)
        written = kc.reshape(num_pages, -1).ne(0).any(1) | vc.reshape(num_pages, -1).ne(0).any(1)
        assert bool((written == (refs != 0)).all())
    for a, b in outs.values():
        assert bool(((a - b).abs() <= H.ATOL + H.RTOL * b.abs()).all())
