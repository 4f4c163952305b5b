"""Index arithmetic of the masses' kernels over the whole range of lengths, compiled for the host."""
import os
import subprocess

import pytest

from cross_model_shared_gb300 import build as B

PROGRAM = r"""
#include <cstdio>
#include "evict.cuh"
int main()
{
    int t, past, i0, group;
    while (std::scanf("%d %d %d %d", &t, &past, &i0, &group) == 4)
        std::printf("%d\n", shkv::mass_first_row(t, past, i0, group));
}
"""


@pytest.fixture(scope="module")
def first_rows(tmp_path_factory):
    d = tmp_path_factory.mktemp("bounds")
    (d / "bounds.cu").write_text(PROGRAM)
    exe = str(d / "bounds")
    subprocess.check_call([B._nvcc(), *B.ARCH, "-std=c++17", "-I", B.INCLUDE, "-I", B.CSRC, "-o", exe, str(d / "bounds.cu")])

    def ask(cases):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout
        return [int(x) for x in out.split()]
    return ask


def test_rows_that_see_a_token_of_the_longest_requests(first_rows):
    """Row r of a block, query token i0 + r // group at position past + that, sees token t if it is not before it."""
    longest = 1 << 30
    cases = []
    for L in (1, 129, 1 << 24, (1 << 25) + 1, longest):
        for group in (1, 5, 64, 100, 128):
            for n in (1, 2, 8, 255):
                tpt = min(128 // group, n)
                if n > L or not 1 <= -(-n // tpt) <= 2:
                    continue
                for past in (L, L - n):                        # of a decode, and of a chunk
                    for i0 in range(0, n, tpt):
                        # tokens of a tile may lie up to 127 behind the request's last
                        ts = {0, 1, 31, L // 2, L // 3, L - 1, L - 33, L - n, L - n + i0, L - n + i0 + 1, L + 126,
                              L - (1 << 25), L - (1 << 24), L - (1 << 25) // 64 * 63}
                        cases += [(t, past, i0, group, tpt) for t in sorted(ts) if 0 <= t <= L + 126]
    got = first_rows([c[:4] for c in cases])
    for (t, past, i0, group, tpt), first in zip(cases, got):
        for r in {0, 1, group - 1, group, tpt * group - 1}:
            if 0 <= r < tpt * group:
                assert (r >= first) == (i0 + r // group >= t - past), (t, past, i0, group, r, first)
        assert first >= 0
    assert len(cases) > 500
