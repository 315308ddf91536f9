"""The operators around the paged attention step, as cases to be timed and compared.

Three families: the linear layer with its epilogue (projections of the decoder
layer, feed-forward matrices, vocabulary logits), beam search's selection over
beams and vocabulary, and the page operations of the paged cache (forking,
extending, freeing and compacting page tables, copying pages).

``listed()`` gives the named cases, ``draw(rng)`` one more of the same ranges,
``prepare(case, seed)`` what a program holds before the call, ``run(state)``
one pass, ``work(case)`` the bytes and operations of a pass, and
``exact(case, seed)`` the result in 64 bits where it is a computed number.
With ``own`` false, ``run`` computes the plain form in elementary torch
operations; with ``own`` true it calls this library.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
ROW = 128          # bytes of one cached token in K or V: 2 KV heads x 64 E4M3 codes


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _linear(T, K, N, dtype="bf16", out=None, bias=False, act="none", residual=False, name=None):
    c = dict(op="linear", T=T, K=K, N=N, dtype=dtype, out=out or dtype, bias=bias, act=act,
             residual=residual)
    return dict(c, name=name) if name else c


def _beam(G, W, V, K, dtype="bf16", masked=False, name=None):
    c = dict(op="beam", G=G, W=W, V=V, K=K, dtype=dtype, masked=masked)
    return dict(c, name=name) if name else c


def _fork(G, W, page_size, lo, hi, layers, name=None):
    c = dict(op="fork", G=G, W=W, page_size=page_size, lo=lo, hi=hi, layers=layers)
    return dict(c, name=name) if name else c


def _compact(num_pages, page_size, fill, rows, layers, name=None):
    c = dict(op="compact", num_pages=num_pages, page_size=page_size, fill=fill, rows=rows,
             layers=layers)
    return dict(c, name=name) if name else c


def _turn(rows, page_size, lo, hi, L, spare, name=None):
    c = dict(op="turn", rows=rows, page_size=page_size, lo=lo, hi=hi, L=L, spare=spare)
    return dict(c, name=name) if name else c


def listed() -> list[dict]:
    return [
        # One request's decode token through the output projection, added onto
        # its residual stream: the latency of the smallest call.
        _linear(T=1, K=1024, N=8192, residual=True, name="linear_oproj_1token"),
        # Vocabulary logits of 16 requests x 4 beams, odd vocabulary, fp32 out:
        # the weight stream.
        _linear(T=64, K=8192, N=32001, out="fp32", name="linear_vocab_logits"),
        # A feed-forward matrix over a 4,096-token prefill block, with bias and
        # activation: dense work.
        _linear(T=4096, K=8192, N=14336, dtype="fp16", bias=True, act="gelu",
                name="linear_ffn_prefill"),
        # One request, four beams, a small vocabulary: latency.
        _beam(G=1, W=4, V=32000, K=4, name="beam_1x4"),
        # A batch with an odd vocabulary, fp32 logits with masked tokens, dead
        # and finished beams.
        _beam(G=16, W=4, V=32001, K=4, dtype="fp32", masked=True, name="beam_16x4_masked"),
        # 32 requests of eight beams over a large vocabulary, twice as many
        # candidates kept as there are beams.
        _beam(G=32, W=8, V=131072, K=16, name="beam_32x8_wide"),
        # A beam step's reordering at page size 64: 16 requests x 4 beams with
        # long common prompts; the partly filled last pages are copied in the K
        # and V caches of four layers.
        _fork(G=16, W=4, page_size=64, lo=40000, hi=80000, layers=4, name="fork_16x4_page64"),
        # The same at page size 1 (nothing is partly filled, so nothing copied).
        _fork(G=32, W=4, page_size=1, lo=20000, hi=40000, layers=1, name="fork_32x4_page1"),
        # Half of a pool of 64-token pages is in use all over it: move the pages
        # together in the caches of two layers.
        _compact(num_pages=16384, page_size=64, fill=0.5, rows=32, layers=2, name="compact_page64"),
        # The same for single-token pages, three quarters used.
        _compact(num_pages=1 << 20, page_size=1, fill=0.75, rows=32, layers=1, name="compact_page1"),
        # A serving turn at page size 1: a quarter of the requests leaves, the
        # others take room for a verify block of eight tokens.
        _turn(rows=32, page_size=1, lo=40000, hi=80000, L=8, spare=100000, name="turn_page1_L8"),
        # The same at page size 64 with many short requests, one token each.
        _turn(rows=256, page_size=64, lo=1, hi=4000, L=1, spare=1000, name="turn_page64_L1"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng) -> dict:
    op = rng.choice(["linear", "linear", "beam", "beam", "fork", "compact", "turn"])
    if op == "linear":
        T = _log_int(rng, 1, 8192)
        K = 8 * _log_int(rng, 8, 1024)
        N = _log_int(rng, 32, 32768)
        while 2 * T * K * N > 9e11:
            T = max(1, T // 2)
        dtype = rng.choice(["bf16", "fp16"])
        return _linear(T, K, N, dtype, rng.choice([dtype, "fp32"]), rng.random() < 0.5,
                       rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]), rng.random() < 0.5)
    if op == "beam":
        W = rng.randint(1, 8)
        return _beam(_log_int(rng, 1, 32), W, _log_int(rng, 1000, 131072), rng.randint(1, 2 * W),
                     rng.choice(["bf16", "fp16", "fp32"]), rng.random() < 0.5)
    ps = rng.choice([1, 64])
    if op == "fork":
        hi = _log_int(rng, 100, 40000)
        return _fork(_log_int(rng, 1, 32), rng.randint(1, 4), ps, rng.randint(1, hi), hi,
                     rng.randint(1, 4) if ps == 64 else 1)
    if op == "compact":
        return _compact(_log_int(rng, 4096, 1 << 20) if ps == 1 else _log_int(rng, 64, 16384), ps,
                        rng.uniform(0.1, 0.95), rng.randint(1, 64), rng.randint(1, 2))
    hi = _log_int(rng, 10, 40000)
    return _turn(_log_int(rng, 1, 64), ps, rng.randint(0, hi), hi, rng.randint(1, 8),
                 rng.randint(1000, 100000))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(gen, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=gen, device=DEV) * scale).to(dtype)


def _caches(gen, num_pages, page_size, layers):
    return [torch.randint(0, 256, (num_pages, page_size, 2, 64), generator=gen, device=DEV,
                          dtype=torch.uint8) for _ in range(2 * layers)]


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _own_tables(rng, lens, page_size, num_pages, width):
    """Page table [rows, width] of requests that share nothing, their pages drawn
    from all over the pool, and the pool's reference counts."""
    need = -(-lens // page_size)
    pool = rng.permutation(num_pages)
    table = np.full((len(lens), width), -1, np.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = pool[at:at + n]
        at += n
    refs = np.zeros(num_pages, np.int32)
    refs[pool[:at]] = 1
    return table, refs


def prepare(case, seed) -> dict:
    # shapes follow from the case alone, values and lengths from the seed
    op = case["op"]
    gen = _gen(seed)
    st = dict(case=case)
    if op == "linear":
        T, K, N, dt = case["T"], case["K"], case["N"], DTYPES[case["dtype"]]
        st["x"] = _randn(gen, T, K, dtype=dt)
        st["w"] = _randn(gen, N, K, dtype=dt, scale=K ** -0.5)
        st["bias"] = _randn(gen, N, dtype=dt, scale=0.5) if case["bias"] else None
        st["residual"] = _randn(gen, T, N, dtype=DTYPES[case["out"]]) if case["residual"] else None
        st["y"] = torch.empty(T, N, dtype=DTYPES[case["out"]], device=DEV)
    elif op == "beam":
        G, W, V, K = case["G"], case["W"], case["V"], case["K"]
        logits = _randn(gen, G, W, V, scale=2.0)
        scores = -torch.rand(G, W, generator=gen, device=DEV) * 12
        finished = None
        if case["masked"]:
            # a third of the tokens banned, one request in five with a dead beam,
            # one beam in five finished
            logits[torch.rand(G, W, V, generator=gen, device=DEV) < 1 / 3] = -math.inf
            if W > 1:
                scores[torch.rand(G, generator=gen, device=DEV) < 0.2, W - 1] = -math.inf
            finished = (torch.rand(G, W, generator=gen, device=DEV) < 0.2).to(torch.uint8)
        st.update(logits=logits.to(DTYPES[case["dtype"]]), scores=scores, finished=finished, pad=0,
                  out_scores=torch.empty(G, K, device=DEV),
                  out_parent=torch.empty(G, K, dtype=torch.int32, device=DEV),
                  out_token=torch.empty(G, K, dtype=torch.int32, device=DEV))
        if own:
            from paged_fp8_gated_b200 import binding
            st["ws"] = binding.alloc_beam_workspace(G, W, V, K)
    elif op == "fork":
        rng = np.random.default_rng(seed)
        G, W, ps = case["G"], case["W"], case["page_size"]
        prompt = rng.integers(case["lo"], case["hi"] + 1, G)
        grown = rng.integers(1, 200)                      # tokens generated since the prompt
        lens = np.repeat(prompt + grown, W)
        shared = np.repeat(prompt // ps, W)               # full prompt pages, common to the beams
        width = -(-(case["hi"] + 200) // ps) + 4
        num_pages = G * (case["hi"] // ps) + G * W * (200 // ps + 6)
        pool = rng.permutation(num_pages)
        table = np.full((G * W, width), -1, np.int32)
        refs = np.zeros(num_pages, np.int32)
        at = 0
        for g in range(G):
            ns = int(prompt[g] // ps)
            common = pool[at:at + ns]
            at += ns
            refs[common] = W
            for r in range(g * W, (g + 1) * W):
                no = int(-(-lens[r] // ps)) - ns
                table[r, :ns] = common
                table[r, ns:ns + no] = pool[at:at + no]
                refs[pool[at:at + no]] = 1
                at += no
        parent = np.concatenate([g * W + rng.integers(0, W, W) for g in range(G)])
        R = G * W
        st.update(table=_i32(table), lens=_i32(lens), parent=_i32(parent), refs0=_i32(refs),
                  caches=_caches(gen, num_pages, ps, case["layers"]),
                  out_table=torch.full((R, width), -1, dtype=torch.int32, device=DEV),
                  out_lens=torch.empty(R, dtype=torch.int32, device=DEV),
                  src=torch.empty(R, dtype=torch.int32, device=DEV),
                  dst=torch.empty(R, dtype=torch.int32, device=DEV))
    elif op == "compact":
        rng = np.random.default_rng(seed)
        P, ps, rows = case["num_pages"], case["page_size"], case["rows"]
        share = rng.dirichlet(np.full(rows, 4.0)) * (P * case["fill"])
        width = int(4 * P * case["fill"] / rows) + 2
        pages = np.clip(np.floor(share).astype(np.int64), 0, width)
        lens = np.maximum(pages * ps - rng.integers(0, ps, rows), 0)
        table, refs = _own_tables(rng, lens, ps, P, width)
        st.update(table=_i32(table), lens=_i32(lens), refs0=_i32(refs),
                  caches=_caches(gen, P, ps, case["layers"]),
                  src=torch.empty(P // 2, dtype=torch.int32, device=DEV),
                  dst=torch.empty(P // 2, dtype=torch.int32, device=DEV),
                  used=torch.empty(1, dtype=torch.int32, device=DEV))
    else:
        rng = np.random.default_rng(seed)
        rows, ps, L = case["rows"], case["page_size"], case["L"]
        lens = rng.integers(case["lo"], case["hi"] + 1, rows)
        width = -(-(case["hi"] + L) // ps)
        P = rows * width + case["spare"] // ps
        table, refs = _own_tables(rng, lens, ps, P, width)
        st.update(table=_i32(table), lens0=_i32(lens), refs0=_i32(refs),
                  leave=torch.from_numpy((rng.random(rows) < 0.25).astype(np.uint8)).to(DEV),
                  lens=torch.empty(rows, dtype=torch.int32, device=DEV),
                  positions=torch.empty(rows * L, dtype=torch.int64, device=DEV),
                  cache_loc=torch.empty(rows * L, dtype=torch.int64, device=DEV))
    if op in ("fork", "compact", "turn"):
        st["refs"] = torch.empty_like(st["refs0"])
        if own:
            from paged_fp8_gated_b200 import binding
            st["ws"] = binding.alloc_pages_workspace(st["table"].shape[0], st["refs"].numel())
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(st):
    op = st["case"]["op"]
    if op in ("fork", "compact", "turn"):
        # the page operations change the pool's counts in place: every pass
        # starts from the same pool
        st["refs"].copy_(st["refs0"])
        if op == "turn":
            st["lens"].copy_(st["lens0"])
    return (_RUN_OWN if own else _RUN_PLAIN)[op](st)


def _act(v, act):
    if act == "relu":
        return v * (v > 0)
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * 2 ** -0.5))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh((2 / math.pi) ** 0.5 * (v + 0.044715 * v * v * v)))
    if act == "silu":
        return v / (1 + torch.exp(-v))
    return v


def _plain_linear(st):
    c = st["case"]
    v = st["x"].float() @ st["w"].float().t()
    if st["bias"] is not None:
        v = v + st["bias"].float()
    v = _act(v, c["act"])
    if st["residual"] is not None:
        v = v + st["residual"].float()
    return v.to(DTYPES[c["out"]])


def _plain_beam(st):
    c = st["case"]
    G, W, V, K = c["G"], c["W"], c["V"], c["K"]
    # 64 bits: the order of two candidates is decided by the last bits of their scores
    x = st["logits"].double()
    m = x.amax(-1, keepdim=True)
    lse = m + torch.log(torch.exp(x - m).sum(-1, keepdim=True))
    key = st["scores"].double()[..., None] + (x - lse)
    if st["finished"] is not None:
        done = (st["finished"] != 0)[..., None]
        is_pad = torch.arange(V, device=x.device) == st["pad"]
        frozen = torch.where(is_pad, st["scores"].double()[..., None], -math.inf)
        key = torch.where(done, frozen, key)
    key = torch.where(torch.isnan(key), -math.inf, key).reshape(G, W * V)
    val, idx = torch.sort(key, dim=-1, descending=True, stable=True)   # ties: lowest index first
    val, idx = val[:, :K], idx[:, :K]
    if idx.shape[1] < K:
        pad = K - idx.shape[1]
        val = torch.cat([val, val.new_full((G, pad), -math.inf)], 1)
        idx = torch.cat([idx, idx.new_zeros((G, pad))], 1)
    live = val > -math.inf
    row = torch.arange(G, device=x.device)[:, None] * W + idx // V
    return (val.float(), torch.where(live, row, -1).int(), torch.where(live, idx % V, -1).int())


def _plain_copy(caches, src, dst):
    ok = (src >= 0) & (dst >= 0)
    s, d = src[ok].long(), dst[ok].long()
    for c in caches:
        c[d] = c[s]


def _plain_fork(st):
    ps = st["case"]["page_size"]
    table, lens, parent, refs = st["table"], st["lens"].long(), st["parent"].long(), st["refs"]
    R, width = st["out_table"].shape
    dev = table.device
    col = torch.arange(width, device=dev)
    row = torch.arange(R, device=dev)
    kids = torch.zeros(table.shape[0], dtype=torch.long, device=dev)
    alive = parent >= 0
    p = parent.clamp(min=0)
    kids.index_add_(0, p, alive.long())
    first = torch.full((table.shape[0],), R, dtype=torch.long, device=dev)
    first = first.scatter_reduce(0, p, torch.where(alive, row, R), "amin")
    # references: an old row releases its pages, every child takes them; of a
    # partly filled last page only the first child takes the page itself
    n_old = -(-lens // ps)
    partial_old = lens % ps != 0
    kids_of_page = torch.where((col == (n_old - 1)[:, None]) & partial_old[:, None],
                               kids.clamp(max=1)[:, None], kids[:, None])
    held = col < n_old[:, None]
    refs.index_add_(0, table.clamp(min=0).reshape(-1).long(),
                    torch.where(held, kids_of_page - 1, 0).reshape(-1).int())
    new_lens = torch.where(alive, lens[p], -1)
    n_new = torch.where(alive, n_old[p], 0)
    last = (n_new - 1).clamp(min=0)
    fresh = alive & partial_old[p] & (first[p] != row)
    free_rank = torch.cumsum((refs == 0).int(), 0)
    k = torch.cumsum(fresh.int(), 0)
    page = torch.searchsorted(free_rank, torch.where(fresh, k, 1).to(free_rank.dtype))
    got = fresh & (k <= free_rank[-1])
    page = page.clamp(max=refs.numel() - 1)
    refs.index_add_(0, page, got.int())
    old_last = table[p, last].long()
    out = st["out_table"]
    rows = table[p]
    out.copy_(torch.where((col < n_new[:, None]) & ~(fresh[:, None] & (col == last[:, None])), rows, out))
    out.copy_(torch.where(got[:, None] & (col == last[:, None]), page[:, None].int(), out))
    st["out_lens"].copy_(torch.where(fresh & ~got, new_lens - new_lens % ps, new_lens))
    st["src"].copy_(torch.where(got, old_last, -1))
    st["dst"].copy_(torch.where(got, page, -1))
    _plain_copy(st["caches"], st["src"], st["dst"])
    return (out, st["out_lens"], refs, st["src"], st["dst"], *st["caches"])


def _plain_compact(st):
    ps = st["case"]["page_size"]
    table, refs = st["table"], st["refs"]
    dev = refs.device
    M = st["src"].numel()
    used = torch.cumsum((refs != 0).long(), 0)
    free = torch.cumsum((refs == 0).long(), 0)
    total = used[-1]
    below = torch.where(total > 0, used[(total - 1).clamp(min=0)], 0)   # used pages that stay
    k = torch.arange(1, M + 1, device=dev)
    moves = k <= total - below
    src = torch.where(moves, torch.searchsorted(used, below + k), -1)
    dst = torch.where(moves, torch.searchsorted(free, k), -1)
    st["src"].copy_(src)
    st["dst"].copy_(dst)
    st["used"].copy_(total.reshape(1))
    to = torch.arange(refs.numel() + 1, device=dev)
    to[torch.where(moves, src, refs.numel())] = torch.where(moves, dst, refs.numel())
    held = torch.arange(table.shape[1], device=dev) < (-(-st["lens"].long() // ps))[:, None]
    table.copy_(torch.where(held, to[table.clamp(min=0).long()].int(), table))
    s, d = src[moves], dst[moves]
    refs[d] = refs[s]
    refs[s] = 0
    _plain_copy(st["caches"], st["src"], st["dst"])
    return (table, refs, st["src"], st["dst"], st["used"], *st["caches"])


def _plain_turn(st):
    c = st["case"]
    ps, L = c["page_size"], c["L"]
    table, refs, lens32 = st["table"], st["refs"], st["lens"]
    R, width = table.shape
    dev = refs.device
    lens = lens32.long()
    col = torch.arange(width, device=dev)
    gone = (st["leave"] != 0)
    n_old = -(-lens // ps)
    held = (col < n_old[:, None]) & gone[:, None]
    refs.index_add_(0, table.clamp(min=0).reshape(-1).long(), -held.reshape(-1).int())
    lens = torch.where(gone, -1, lens)
    alive = ~gone
    n_new = -(-(lens + L) // ps)
    need = torch.where(alive, n_new - n_old, 0)
    free = torch.cumsum((refs == 0).long(), 0)
    ok = (need.sum() <= free[-1]) & ((n_new <= width) | ~alive).all()
    before = torch.cumsum(need, 0) - need
    # the k-th page that is handed out (row by row) is the k-th free one
    slot = (col >= n_old[:, None]) & (col < n_new[:, None]) & alive[:, None] & ok
    rank = before[:, None] + col - n_old[:, None] + 1
    page = torch.searchsorted(free, torch.where(slot, rank, 1)).clamp(max=refs.numel() - 1)
    table.copy_(torch.where(slot, page.int(), table))
    refs.index_add_(0, page.reshape(-1), slot.reshape(-1).int())
    pos = lens[:, None] + torch.arange(L, device=dev)
    pos = torch.where(alive[:, None], pos, 0)
    loc = table.gather(1, (pos // ps).clamp(max=width - 1)).long() * ps + pos % ps
    st["positions"].copy_(pos.reshape(-1))
    st["cache_loc"].copy_(torch.where(alive[:, None] & ok, loc, -1).reshape(-1))
    lens32.copy_(torch.where(alive & ok, lens + L, lens))
    return table, refs, lens32, st["positions"], st["cache_loc"]


def _own_linear(st):
    from paged_fp8_gated_b200 import binding
    return binding.linear(st["x"], st["w"], bias=st["bias"], residual=st["residual"],
                          activation=st["case"]["act"], out=st["y"])


def _own_beam(st):
    from paged_fp8_gated_b200 import binding
    return binding.beam_select(st["logits"], st["scores"], st["case"]["K"], finished=st["finished"],
                               pad_token=st["pad"],
                               out=(st["out_scores"], st["out_parent"], st["out_token"]),
                               workspace=st["ws"])


def _own_fork(st):
    from paged_fp8_gated_b200 import binding
    binding.pages_fork(st["table"], st["lens"], st["parent"], st["refs"], st["case"]["page_size"],
                       out=(st["out_table"], st["out_lens"], st["src"], st["dst"]), workspace=st["ws"])
    binding.pages_copy(st["caches"], st["src"], st["dst"])
    return (st["out_table"], st["out_lens"], st["refs"], st["src"], st["dst"], *st["caches"])


def _own_compact(st):
    from paged_fp8_gated_b200 import binding
    binding.pages_compact(st["table"], st["lens"], st["refs"], st["case"]["page_size"],
                          out=(st["src"], st["dst"], st["used"]), workspace=st["ws"])
    binding.pages_copy(st["caches"], st["src"], st["dst"])
    return (st["table"], st["refs"], st["src"], st["dst"], st["used"], *st["caches"])


def _own_turn(st):
    from paged_fp8_gated_b200 import binding
    c = st["case"]
    binding.pages_free(st["table"], st["lens"], st["refs"], c["page_size"], leave=st["leave"])
    binding.pages_extend(st["table"], st["lens"], st["refs"], c["page_size"], c["L"],
                         out=(st["positions"], st["cache_loc"]), workspace=st["ws"])
    return st["table"], st["refs"], st["lens"], st["positions"], st["cache_loc"]


_RUN_PLAIN = dict(linear=_plain_linear, beam=_plain_beam, fork=_plain_fork, compact=_plain_compact,
                  turn=_plain_turn)
_RUN_OWN = dict(linear=_own_linear, beam=_own_beam, fork=_own_fork, compact=_own_compact,
                turn=_own_turn)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case) -> dict:
    op = case["op"]
    if op == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        e, o = BYTES[case["dtype"]], BYTES[case["out"]]
        b = e * (T * K + N * K + (N if case["bias"] else 0)) + o * T * N * (2 if case["residual"] else 1)
        return dict(bytes=b, flops=2 * T * K * N)
    if op == "beam":
        G, W, V, K = case["G"], case["W"], case["V"], case["K"]
        # an exponential and a sum, a subtraction and a comparison per logit
        return dict(bytes=BYTES[case["dtype"]] * G * W * V + 4 * G * W + 12 * G * K, flops=4 * G * W * V)
    ps = case["page_size"]
    if op == "fork":
        R = case["G"] * case["W"]
        n = R * (case["lo"] + case["hi"]) // 2 // ps
        # tables read and written; a beam in three gets a copy of its last page
        pages = R // 3 if ps > 1 else 0
        return dict(bytes=2 * 4 * n + 2 * 4 * n // case["W"] + pages * 2 * case["layers"] * 2 * ps * ROW,
                    flops=n)
    if op == "compact":
        P, f = case["num_pages"], case["fill"]
        moved = int(P * f * (1 - f))
        return dict(bytes=4 * P + 3 * 4 * moved + 2 * 4 * int(P * f) + moved * 2 * case["layers"] * 2 * ps * ROW,
                    flops=P)
    R, L = case["rows"], case["L"]
    n = R * (case["lo"] + case["hi"]) // 2 // ps
    # the leaving rows' entries and counts, one look over the pool's counts, the new tokens' rows
    return dict(bytes=3 * 4 * (n // 4) + 4 * (R * -(-(case["hi"] + L) // ps) + case["spare"] // ps)
                + 16 * R * L, flops=n)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    """64-bit results of the linear layer and of the selection; the page
    operations compute no numbers (None): their tables and the bytes that they
    copy are equal or wrong."""
    if case["op"] == "linear":
        return _exact_linear(case, prepare(case, seed))
    if case["op"] == "beam":
        return _exact_beam(case, prepare(case, seed))
    return None


def _exact_linear(case, st):
    xt = st["x"].to(torch.float64)
    y = torch.empty(case["T"], case["N"], dtype=torch.float64, device=xt.device)
    for n0 in range(0, case["N"], 4096):
        n1 = min(case["N"], n0 + 4096)
        s = torch.matmul(xt, st["w"][n0:n1].to(torch.float64).T)
        if case["bias"]:
            s += st["bias"][n0:n1].to(torch.float64)
        a = case["act"]
        if a == "relu":
            s = torch.maximum(s, torch.zeros((), dtype=s.dtype, device=s.device))
        elif a == "gelu":        # x Phi(x)
            s = s * torch.special.ndtr(s)
        elif a == "gelu_tanh":
            u = math.sqrt(2.0 / math.pi) * (s + 0.044715 * s ** 3)
            s = s * torch.sigmoid(2 * u)       # (1 + tanh u) / 2 = sigmoid(2u)
        elif a == "silu":
            s = s * torch.sigmoid(s)
        if case["residual"]:
            s += st["residual"][:, n0:n1].to(torch.float64)
        y[:, n0:n1] = s
    return y


def _exact_beam(case, st):
    G, W, V, K = case["G"], case["W"], case["V"], case["K"]
    x = st["logits"].to(torch.float32).cpu().numpy()
    cum = st["scores"].cpu().numpy().astype(np.float64)
    fin = None if st["finished"] is None else st["finished"].cpu().numpy()
    val = np.full((G, K), -np.inf)
    par = np.full((G, K), -1, np.int32)
    tok = np.full((G, K), -1, np.int32)
    for g in range(G):
        cand = []
        for w in range(W):
            if fin is not None and fin[g, w]:
                cand.append((-cum[g, w], w * V + st["pad"]))
                continue
            r = x[g, w].astype(np.float64)
            top = r.max()
            if not np.isfinite(top) or cum[g, w] == -np.inf:
                continue
            norm = top + math.log(math.fsum(np.exp(r - top)))
            k = min(K, V)
            floor = np.partition(r, V - k)[V - k]          # the k-th largest logit, ties kept
            for v in np.nonzero((r >= floor) & (r > -np.inf))[0]:
                cand.append((-(cum[g, w] + (r[v] - norm)), w * V + int(v)))
        cand = sorted(c for c in cand if c[0] < np.inf)[:K]
        for i, (neg, flat) in enumerate(cand):
            val[g, i], par[g, i], tok[g, i] = -neg, g * W + flat // V, flat % V
    return (torch.from_numpy(val).to(DEV), torch.from_numpy(par).to(DEV), torch.from_numpy(tok).to(DEV))
