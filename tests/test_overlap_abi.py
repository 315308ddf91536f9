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
