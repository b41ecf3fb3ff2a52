"""The ring of key stages of the attention for few rows (csrc/kv4_ring.cuh), walked through
on the host in every interleaving of a group of warps and of the copies."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ is not installed")
    exe = str(tmp_path_factory.mktemp("ring") / "ring_walk")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror",
                    "-I", os.path.join(ROOT, "cache_gating_kv_b200", "csrc"),
                    "-o", exe, os.path.join(ROOT, "tests", "c", "ring_walk.cpp")],
                   check=True, capture_output=True, text=True)

    def run(*args):
        r = subprocess.run([exe, *map(str, args)], capture_output=True, text=True, timeout=120)
        return r.returncode, r.stdout.strip()

    return run


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tail", [1, 33, 65, 96, 97, 128])
def test_no_copy_meets_a_reader(walk, d, tail):
    """Up to 13 stages, the last with keys for one to four warps, behind 0 or 5 stages of
    other pieces: no wait is answered early, no stage overwritten while a warp has it to
    read, nobody waits for ever, and every phase has its arrivals at the end."""
    for base in (0, 5):
        for stages in (1, 2, 6, 7, 8, 9, 10, 13):
            rc, out = walk(d, (stages - 1) * 128 + tail, base)
            assert rc == 0 and out.startswith("states "), (base, stages, out)


@pytest.mark.parametrize("d,slots", [(64, 8), (128, 6)])
def test_walk_finds_a_release_without_its_wait(walk, d, slots):
    """The walk sees the fault that the wait is there for: a warp that releases a last
    stage without keys for it unread and unwaited-for lets a copy overwrite its slot."""
    for tail in (1, 33, 65, 96):
        rc, out = walk(d, slots * 128 + tail, 0, "skip")
        assert rc == 1 and "overwritten" in out, out
        assert walk(d, (slots - 1) * 128 + tail, 0, "skip")[0] == 0  # the ring is not used twice
    assert walk(d, 10 * 128, 0, "skip")[0] == 0  # all warps have keys
