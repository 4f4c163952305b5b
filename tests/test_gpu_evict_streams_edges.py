"""Eviction's calls on several host threads."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FIRST_CALLS = """
import threading, torch
from tests.eviction_common import Cache, check_mass, lse_of
caches = [Cache([400, 300 + i], 2, d, 16, seed=i) for i, d in enumerate((64, 128) * 4)]
pools = [c.pool() for c in caches]
qs = [c.randn(2, 300, 8, c.d) for c in caches]
lses = [lse_of(c, q, 0.1, True) for c, q in zip(caches, qs)]
torch.cuda.synchronize()
got, go = [None] * len(caches), threading.Barrier(len(caches))
def call(i):
    torch.cuda.set_device(0)
    with torch.cuda.stream(torch.cuda.Stream()):
        go.wait()
        got[i] = pools[i].prefill_mass(qs[i], lses[i], None, scale=0.1)
threads = [threading.Thread(target=call, args=(i,)) for i in range(len(caches))]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
for c, p, q, lse, m in zip(caches, pools, qs, lses, got):
    assert p.check_errors() == 0
    check_mass(c, q, lse, 0.1, True, 1.0, None, m)
print("all right")
"""


def test_the_first_calls_of_a_process_on_several_threads():
    """Each thread has a pool; what the library asks of a kernel's build once, all ask for at the same time."""
    out = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.stdout.endswith("all right\n"), out.stderr[-2000:]
