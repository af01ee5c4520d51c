"""How the attention's key tiles are cut into runs (csrc/runs.h), compiled for
the host: every tile belongs to the run that starts at or before it, whatever
their number."""
import ctypes
import os
import shutil
import subprocess

import pytest

from block_diffusion_speculative_draft_gb300 import build

SOURCE = """
#include "runs.h"
extern "C" long long start(long long all, long long runs, long long c) { return dfl::Runs{all, runs}.start(c); }
extern "C" long long of(long long all, long long runs, long long u) { return dfl::Runs{all, runs}.of(u); }
extern "C" long long ratio(long long x, long long y) { return dfl::Runs::ratio(x, y); }
"""


@pytest.fixture(scope="module")
def runs(tmp_path_factory):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("needs g++")
    at = tmp_path_factory.mktemp("runs")
    (at / "runs.cpp").write_text(SOURCE)
    out = str(at / "libruns.so")
    subprocess.run([cxx, "-O2", "-fPIC", "-shared", "-I", build.CSRC, str(at / "runs.cpp"), "-o", out], check=True)
    lib = ctypes.CDLL(out)
    for fn, n in ((lib.start, 3), (lib.of, 3), (lib.ratio, 2)):
        fn.argtypes, fn.restype = [ctypes.c_longlong] * n, ctypes.c_longlong
    return lib


# up to 2^22 kv heads, 2^13 query tiles of a head and 2^18 key tiles of an item,
# as far as a device's memory holds their keys and rows
@pytest.mark.parametrize("n", [1, 2, 151, 152, 4097, 10 ** 6 + 1, 2 ** 31, 2 ** 32 - 1, 2 ** 32, 2 ** 32 + 5, 2 ** 33 + 7,
                               5 * 2 ** 33, 2 ** 38 + 11])
@pytest.mark.parametrize("most", [1, 2, 7, 152, 304, 320])
def test_a_tile_belongs_to_the_run_that_holds_it(runs, n, most):
    r = min(n, most)
    starts = [runs.start(n, r, c) for c in range(r + 1)]
    assert starts == [c * n // r for c in range(r + 1)]
    for c in range(r):
        for u in {starts[c], starts[c + 1] - 1, (starts[c] + starts[c + 1]) // 2}:
            assert runs.of(n, r, u) == c, u


def test_ratio(runs):
    for x in (0, 1, 9, 2 ** 32 - 1, 2 ** 32, 2 ** 40 + 3, 2 ** 62):
        for y in (1, 2, 320, 2 ** 32 - 1, 2 ** 32, 2 ** 32 + 1, 2 ** 45):
            assert runs.ratio(x, y) == x // y, (x, y)


@pytest.mark.parametrize("shape", [(4096, 256, 4096, 64, 64), (16384, 256, 65536, 256, 64), (4, 256, 1 << 18, 1 << 8, 64)])
def test_no_size_is_refused_for_the_joins_sake(shape):
    """The launch that joins parts has a grid of its own, whatever the rows."""
    from block_diffusion_speculative_draft_gb300 import api
    build.build()
    b, N, nq, nkv, d = shape
    assert api.dflash_tree_attention_workspace_size(*shape) == api.dflash_tree_attention_workspace_size(1, N, nq, nkv, d)
