"""Arrays of one call that overlap: refused on the host, before any CUDA call, wherever one
block could read what another has written already.  The pointers here are never followed."""
import pytest

F = 0x100000     # one MiB apart: nothing overlaps unless a test says so


@pytest.fixture(scope="module")
def B():
    from paged_fp8_gated_b200 import build
    build.build()
    from paged_fp8_gated_b200 import binding
    return binding


def _refused(B, status):
    assert status == -4 and b"overlap" in B.lib().gad_last_error()


BEAM = dict(logits=F, dtype=1, ld=1000, scores=2 * F, finished=9 * F, pad=0, G=2, W=4, V=1000, K=4,
            s=3 * F, p=4 * F, t=5 * F, ws=6 * F, wsb=1 << 20)


@pytest.mark.parametrize("over", [
    dict(s=9 * F), dict(p=9 * F + 4), dict(t=9 * F - 28),              # finished [8 bytes]
    dict(s=2 * F + 28), dict(p=2 * F - 28), dict(t=2 * F),             # scores [32]
    dict(s=4 * F), dict(p=5 * F + 16), dict(t=3 * F - 16),             # one another [32 each]
    dict(ws=2 * F), dict(s=6 * F + 256), dict(finished=6 * F + 300), dict(ws=F + 15872),   # the workspace; logits [16,000]
], ids=str)
def test_beam_overlaps_are_refused(B, over):
    _refused(B, B.lib().gad_beam_select(*dict(BEAM, **over).values(), None))


PAGES = dict(table=F, lens=2 * F, rows=4, parent=3 * F, rows_out=6, L=3, max_pages=8, ps=64, refs=4 * F, n=64,
             otable=5 * F, olens=6 * F, src=7 * F, dst=8 * F, pos=9 * F, loc=10 * F, leave=13 * F, moves=5, used=11 * F,
             ws=12 * F, wsb=1 << 20)
KEYS = dict(fork="table lens rows parent rows_out max_pages ps refs n otable olens src dst ws wsb",
            extend="table lens rows L max_pages ps refs n pos loc ws wsb",
            free="table lens rows leave max_pages ps refs n",
            compact="table lens rows max_pages ps refs n src dst moves used ws wsb")
# bytes of each array at these sizes
SIZE = dict(fork=dict(table=128, lens=16, parent=24, refs=256, otable=192, olens=24, src=24, dst=24, ws=4096),
            extend=dict(table=128, lens=16, refs=256, pos=96, loc=96, ws=4096),
            free=dict(table=128, lens=16, leave=4, refs=256),
            compact=dict(table=128, lens=16, refs=256, src=20, dst=20, used=4, ws=4096))
READ = dict(fork={"table", "lens", "parent"}, extend=set(), free={"table", "leave"}, compact={"lens"})
FIXED = {"refs": 16, "ws": 256, "pos": 8, "loc": 8, "leave": 1}     # alignments (others 4)
PAIRS = [(fn, a, b) for fn in KEYS for a in SIZE[fn] for b in SIZE[fn]
         if a != b and not {a, b} <= READ[fn]]


def _pages(B, fn, **over):
    a = dict(PAGES, **over)
    return getattr(B.lib(), f"gad_pages_{fn}")(*(a[k] for k in KEYS[fn].split()), None)


@pytest.mark.parametrize("fn,a,b", PAIRS, ids=lambda v: str(v))
def test_pages_overlaps_are_refused(B, fn, a, b):
    """Array a at b's last place that a's alignment allows."""
    align = FIXED.get(a, 4)
    at = PAGES[b] + (SIZE[fn][b] - 1) // align * align
    _refused(B, _pages(B, fn, **{a: at}))


@pytest.mark.parametrize("which", [0, 1])
def test_pages_copy_lists_inside_a_cache_are_refused(B, which):
    import ctypes
    caches = (ctypes.c_void_p * 2)(F, 2 * F)
    lists = [3 * F, 4 * F]
    lists[which] = 2 * F + 64 * 128 - 4
    _refused(B, B.lib().gad_pages_copy(caches, 2, 128, 64, *lists, 4, None))


def _linear(B, **o):
    a = dict(x=F, ldx=256, w=2 * F, ldw=64, bias=None, residual=None, ldr=0, y=4 * F, ldy=256, T=4, K=64, N=100,
             dtype=1, out=1, act=0)
    a.update(o)
    return B.lib().gad_linear(*a.values(), None)


@pytest.mark.parametrize("over", [
    dict(y=F), dict(y=F + 126), dict(y=F - 198), dict(y=F + 3 * 512 + 126), dict(y=F - 3 * 512),   # x: 128 of 512 bytes
    dict(y=F + 314), dict(y=F + 3 * 512 - 2),                      # y's 200 bytes reach x's next row
    dict(y=F + 128, ldy=264), dict(y=F + 128, ldx=264),            # side by side, but rows at different distances
    dict(out=6, y=F + 128, ldy=128),                               # fp32: 400 of 512 bytes
    dict(y=2 * F + 200), dict(residual=4 * F + 198, ldr=256), dict(residual=4 * F + 314, ldr=256),
    dict(bias=4 * F + 320), dict(T=1, y=F + 126), dict(T=1, y=2 * F + 120, ldw=256), dict(T=1, y=2 * F + 400, ldw=256),
], ids=str)
def test_linear_overlaps_are_refused(B, over):
    _refused(B, _linear(B, **over))
