"""The step kernel's plan and walk on the CPU: the kernel's own index
arithmetic (flint_paged_walk.cuh), compiled for the host, over random
boundaries and lengths.  Every sequence, row, position and tile that a share's
walk names lies within the call's arrays, the walks take just the pairs that
the plan counted, and each ends, whatever cu_new and cache_len hold."""
import os
import subprocess

import pytest

from full_gqa_learned_b200 import build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("walk") / "paged_walk_host")
    subprocess.check_call([build.nvcc_path(), "-O1", "-std=c++17", *build.ARCH, "-I", build.INCLUDE, "-o", exe,
                           os.path.join(HERE, "paged_walk_host.cu")])
    return exe


@pytest.mark.parametrize("kind", ["good", "ill"])
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_walk_stays_within_the_call(walk, kind, seed):
    r = subprocess.run([walk, kind, str(seed), "4000"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.endswith("OK\n"), "exit %d: %s" % (r.returncode, r.stdout[-2000:])
