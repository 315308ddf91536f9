"""Argument checks of the linear layer, the beam selection and the page operations: they
run on the host before any CUDA call, so the pointers here are never followed."""
import ctypes

import pytest

FAKE = 0x100000


@pytest.fixture(scope="module")
def B():
    from paged_fp8_gated_b200 import build
    build.build()
    from paged_fp8_gated_b200 import binding
    return binding


def _linear(so, **o):
    a = dict(x=FAKE, ldx=64, w=2 * FAKE, ldw=64, bias=None, residual=None, ldr=0, y=4 * FAKE, ldy=128, T=4, K=64,
             N=128, dtype=1, out=1, act=0)
    a.update(o)
    return so.gad_linear(*(a[k] for k in ("x", "ldx", "w", "ldw", "bias", "residual", "ldr", "y", "ldy", "T", "K",
                                          "N", "dtype", "out", "act")), None)


@pytest.mark.parametrize("over,status", [
    (dict(x=None), -1), (dict(w=None), -1), (dict(y=None), -1),
    (dict(dtype=6), -8), (dict(dtype=2), -8), (dict(out=7), -8), (dict(dtype=7, out=1), -8), (dict(out=0), -8),
    (dict(T=0), -2), (dict(T=-1), -2), (dict(K=0), -2), (dict(N=0), -2), (dict(N=(1 << 22) + 1), -2),
    (dict(act=5), -4), (dict(act=-1), -4),
    (dict(ldx=60), -9), (dict(ldx=68), -9), (dict(ldw=56), -9), (dict(ldy=127), -9),
    (dict(residual=8 * FAKE, ldr=100), -9), (dict(ldx=(1 << 32) + 8), -9), (dict(ldy=1 << 33), -9),
    (dict(x=FAKE + 8), -3), (dict(w=2 * FAKE + 2), -3), (dict(y=4 * FAKE + 1), -3), (dict(out=6, y=4 * FAKE + 2), -3),
    (dict(bias=8 * FAKE + 1), -3), (dict(residual=8 * FAKE + 1, ldr=128), -3),
    (dict(y=FAKE), -4), (dict(y=2 * FAKE + 64), -4), (dict(bias=4 * FAKE + 10), -4),
    (dict(residual=4 * FAKE + 2, ldr=128), -4), (dict(residual=4 * FAKE, ldr=136), -4),
])
def test_linear_argument_checks(B, over, status):
    assert _linear(B.lib(), **over) == status
    assert B.last_error()


def _beam(so, **o):
    a = dict(logits=FAKE, dtype=1, ld=1000, scores=2 * FAKE, finished=None, pad=0, G=2, W=4, V=1000, K=4,
             s=3 * FAKE, p=4 * FAKE, t=5 * FAKE, ws=6 * FAKE, wsb=1 << 20)
    a.update(o)
    return so.gad_beam_select(*a.values(), None)


@pytest.mark.parametrize("over,status", [
    (dict(logits=None), -1), (dict(scores=None), -1), (dict(s=None), -1), (dict(p=None), -1), (dict(t=None), -1),
    (dict(dtype=5), -8), (dict(dtype=3), -8),
    (dict(G=0), -2), (dict(W=0), -2), (dict(W=65), -2), (dict(G=1025), -2), (dict(K=0), -2), (dict(K=65), -2),
    (dict(V=0), -2), (dict(V=(1 << 24) + 1, ld=1 << 25), -2), (dict(pad=-1), -2), (dict(pad=1000), -2),
    (dict(ld=999), -9), (dict(logits=FAKE + 1), -3), (dict(dtype=6, logits=FAKE + 2), -3), (dict(p=4 * FAKE + 2), -3),
    (dict(s=2 * FAKE), -4), (dict(t=2 * FAKE + 28), -4),
    (dict(ws=None), -5), (dict(ws=6 * FAKE + 16), -3), (dict(wsb=100), -5),
])
def test_beam_argument_checks(B, over, status):
    assert _beam(B.lib(), **over) == status
    assert B.last_error()


def test_beam_workspace_query(B):
    so = B.lib()
    assert so.gad_beam_workspace_bytes(0, 4, 100, 4) == 0 and B.last_error()
    assert so.gad_beam_workspace_bytes(1, 4, 100, 65) == 0
    small, large = so.gad_beam_workspace_bytes(1, 1, 1, 1), so.gad_beam_workspace_bytes(64, 64, 1 << 24, 64)
    assert 0 < small < large and small % 256 == 0 and large % 256 == 0


def _pages(so, fn, **o):
    a = dict(table=FAKE, lens=2 * FAKE, rows=4, parent=3 * FAKE, rows_out=4, L=1, max_pages=8, ps=64, refs=4 * FAKE,
             n=64, otable=5 * FAKE, olens=6 * FAKE, src=7 * FAKE, dst=8 * FAKE, pos=9 * FAKE, loc=10 * FAKE,
             leave=None, moves=4, used=11 * FAKE, ws=12 * FAKE, wsb=1 << 20)
    a.update(o)
    keys = dict(fork="table lens rows parent rows_out max_pages ps refs n otable olens src dst ws wsb",
                extend="table lens rows L max_pages ps refs n pos loc ws wsb",
                free="table lens rows leave max_pages ps refs n",
                compact="table lens rows max_pages ps refs n src dst moves used ws wsb")[fn]
    return getattr(so, f"gad_pages_{fn}")(*(a[k] for k in keys.split()), None)


@pytest.mark.parametrize("fn", ["fork", "extend", "free", "compact"])
@pytest.mark.parametrize("over,status", [
    (dict(table=None), -1), (dict(lens=None), -1), (dict(refs=None), -1),
    (dict(rows=0), -2), (dict(rows=4097), -2), (dict(max_pages=0), -2), (dict(max_pages=1 << 26), -2),
    (dict(ps=16), -4), (dict(ps=0), -4), (dict(n=0), -2), (dict(n=1 << 25), -2), (dict(ps=1, n=1 << 31), -2),
    (dict(refs=4 * FAKE + 4), -3), (dict(table=FAKE + 2), -3),
])
def test_pages_pool_checks(B, fn, over, status):
    assert _pages(B.lib(), fn, **over) == status
    assert B.last_error()


@pytest.mark.parametrize("fn,over,status", [
    ("fork", dict(parent=None), -1), ("fork", dict(otable=None), -1), ("fork", dict(dst=None), -1),
    ("fork", dict(rows_out=0), -2), ("fork", dict(rows_out=4097), -2), ("fork", dict(ws=None), -5),
    ("fork", dict(wsb=64), -5), ("fork", dict(ws=12 * FAKE + 128), -3), ("fork", dict(otable=FAKE + 4), -4),
    ("fork", dict(olens=2 * FAKE + 12), -4), ("fork", dict(parent=3 * FAKE + 1), -3),
    ("extend", dict(pos=None), -1), ("extend", dict(loc=None), -1), ("extend", dict(L=0), -2),
    ("extend", dict(L=65537), -2), ("extend", dict(pos=9 * FAKE + 4), -3), ("extend", dict(ws=None), -5),
    ("compact", dict(src=None), -1), ("compact", dict(used=None), -1), ("compact", dict(moves=0), -2),
    ("compact", dict(wsb=0), -5), ("compact", dict(used=11 * FAKE + 1), -3),
])
def test_pages_argument_checks(B, fn, over, status):
    assert _pages(B.lib(), fn, **over) == status
    assert B.last_error()


@pytest.mark.parametrize("over,status", [
    (dict(caches=None), -1), (dict(src=None), -1), (dict(dst=None), -1), (dict(m=0), -2), (dict(m=4097), -2),
    (dict(bytes=0), -2), (dict(bytes=24), -2), (dict(bytes=1 << 25), -2), (dict(n=0), -2), (dict(pairs=-1), -2),
    (dict(ptr=0), -1), (dict(ptr=FAKE + 8), -3), (dict(src=FAKE + 1), -3),
])
def test_pages_copy_argument_checks(B, over, status):
    a = dict(caches=True, m=2, bytes=128, n=64, src=FAKE, dst=2 * FAKE, pairs=4, ptr=FAKE)
    a.update(over)
    arr = (ctypes.c_void_p * 4097)(*([FAKE, a["ptr"] or None]))
    st = B.lib().gad_pages_copy(arr if a["caches"] else None, a["m"], a["bytes"], a["n"], a["src"], a["dst"],
                                a["pairs"], None)
    assert st == status
    assert B.last_error()


def test_pages_workspace_query(B):
    so = B.lib()
    assert so.gad_pages_workspace_bytes(0, 100) == 0 and so.gad_pages_workspace_bytes(4097, 100) == 0
    assert so.gad_pages_workspace_bytes(4, 0) == 0 and B.last_error()
    assert so.gad_pages_workspace_bytes(4, 1 << 20) > so.gad_pages_workspace_bytes(4, 100) > 0
