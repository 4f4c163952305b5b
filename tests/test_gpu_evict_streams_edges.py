"""Eviction's calls right behind one another, and on several host threads."""
import os
import subprocess
import sys

import pytest
import torch

from .eviction_common import Cache, lse_of
from .test_gpu_evict import spare_table

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


@pytest.mark.parametrize("T", [2003, 2000])
def test_calls_right_behind_one_another_give_what_calls_that_wait_give(T):
    """Every kernel may start while the one before is finishing: what that one still writes, masses in place and
    indexes, is read as it is in the end, also where two tokens' masses share 32 bytes."""
    lens = [2000 - 37 * b for b in range(24)]
    c = Cache(lens, 8, 128, 16, seed=T, spare=24 * 63)
    pool = c.pool()
    scale = 0.2
    qs = [c.randn(24, 2, 32, 128) for _ in range(3)]
    lses = [lse_of(c, q, scale, True) for q in qs]
    keep = [500 + 20 * b for b in range(24)]
    new = spare_table(c, keep, lens)
    table = c.table.cuda()

    def steps(wait):
        mass = torch.zeros(24, 8, T, device="cuda")
        index = torch.zeros(24, 8, max(keep), dtype=torch.int32, device="cuda")
        moved = torch.zeros_like(mass)
        got = []
        for i in range(60):
            q, lse = qs[i % 3], lses[i % 3]
            (pool.decode_mass if i % 2 else pool.prefill_mass)(
                *((q.view(24, 64, 128), lse.view(24, 64), 2) if i % 2 else (q, lse)), mass, decay=0.3, scale=scale)
            wait()
            pool.select_tokens(mass, keep, sink=2, recent=5, out=index)
            wait()
            pool.evict_tokens(index, keep, new, mass=mass, out=moved, source=(table, lens))
            wait()
            got.append((mass.clone(), index.clone(), moved.clone(), pool.k_pages[new[3, :20].long()].clone()))
            pool.set_seq_lens(lens)
            pool.block_table.copy_(table)
        torch.cuda.synchronize()
        assert pool.check_errors() == 0
        return got

    want = steps(torch.cuda.synchronize)
    for _ in range(3):
        for i, (a, b) in enumerate(zip(steps(lambda: None), want)):
            assert all(torch.equal(x, y) for x, y in zip(a, b)), i
