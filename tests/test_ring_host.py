"""The bookkeeping of a ring's copies (csrc/ring.cuh), compiled for the host: after a wait that ran out, the
drain waits for every copy in flight, in its phase, and for no other."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = """#include "ring.cuh"
extern "C" int stage(int n, int s) { return dsa::ring_stage(n, s); }
extern "C" unsigned parity(int n, int s) { return dsa::ring_parity(n, s); }
extern "C" int end(int landed, int s, int copies) { return dsa::ring_end(landed, s, copies); }
"""


@pytest.fixture(scope="module")
def ring(tmp_path_factory):
    gxx = shutil.which("g++")
    assert gxx, "g++ not found"
    lib = str(tmp_path_factory.mktemp("ring") / "ring.so")
    cmd = [gxx, "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-x", "c++", "-", "-o", lib,
           "-I", os.path.join(ROOT, "sparse_attention_09_b200", "csrc")]
    res = subprocess.run(cmd, input=SOURCE, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    return ctypes.CDLL(lib)


@pytest.mark.parametrize("stages", range(2, 9))
def test_drain_waits_for_exactly_the_copies_in_flight(ring, stages):
    for copies in range(1, 4 * stages + 3):
        for fails in range(copies + 1):  # the wait for this copy runs out; == copies: none does
            completed, flying = [0] * stages, {}  # per stage: phases of its barrier that are complete; its copy in flight

            def issue(n):
                s = ring.stage(n, stages)
                assert s not in flying and completed[s] == n // stages
                flying[s] = n

            def passes(n):  # a wait for a phase of this parity returns when the current phase has the other one
                s = ring.stage(n, stages)
                return completed[s] & 1 != ring.parity(n, stages)

            def land(n):
                s = ring.stage(n, stages)
                assert flying.pop(s) == n
                completed[s] += 1

            for n in range(min(copies, stages)):
                issue(n)
            for n in range(fails):
                assert not passes(n)
                land(n)
                assert passes(n)
                if n + stages < copies:
                    issue(n + stages)
            drained = range(fails, ring.end(fails, stages, copies))
            assert sorted(flying.values()) == list(drained)
            for n in drained:
                assert not passes(n)  # it does not return while the copy is in flight
                land(n)
                assert passes(n)      # and returns at once when it has landed
            assert not flying


def test_no_overflow_at_the_longest_runs(ring):
    for landed, copies in ((2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31 - 3, 2 ** 31 - 1)):
        assert ring.end(landed, 8, copies) == copies
