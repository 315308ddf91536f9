"""The linear layer's bounded waits give up instead of hanging, and gad_linear_status
reports it: every kernel form on the build of the library in which a pipeline wait gives
up at its first miss (see test_wait_giveup_gpu.py), in a child process that loads only
that build.  The waiting warps stop, the copies and tensor-core operations in flight are
waited for (also where only one block of a pair has asked for a stage), tensor memory is
freed, the bit is set and cleared by the read, and the context stays usable."""
import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16, F32 = 1, 6
LINEAR = 16  # GAD_STATUS_LINEAR_WAIT
# one block a tile; a cluster over K; promoted chains, of 64, 128 and 256 tokens; pairs,
# with 256 and 128 columns; two and four pairs that share a tile; promoted pairs, alone
# and sharing
CALLS = [("narrow", 8, 1024, 40000, BF16), ("cluster", 16, 8192, 1024, BF16), ("promote", 16, 8192, 8192, F32),
         ("wide", 2048, 1024, 4096, BF16), ("wide128", 256, 1024, 8192, BF16), ("split", 512, 8192, 1024, BF16),
         ("wide_promote", 1024, 4096, 4096, F32), ("promote128", 96, 8192, 4096, F32),
         ("promote256", 160, 4096, 8192, F32), ("split256", 192, 2048, 8192, BF16), ("split4", 256, 8192, 1024, BF16),
         ("promote_pairs", 96, 1024, 40000, F32), ("promote_split", 128, 4096, 4096, F32),
         ("promote_split4", 128, 8192, 128, F32)]


def test_linear_waits_give_up_and_report(cuda_dev):
    from paged_fp8_gated_b200 import build
    build.build_short_wait()
    proc = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "linear_giveup_child.py"), json.dumps(CALLS)],
                          cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert proc.returncode == 0, proc.stderr[-3000:]
    res = json.loads(proc.stdout.strip().splitlines()[-1])
    for name, *_ in CALLS:
        first, second, seconds = res[name]
        assert first & LINEAR and second == 0, (name, res)
        assert seconds < 30, (name, res)     # at most a teardown wait of 2 s per stage
    assert res["after"] == 999000.0
