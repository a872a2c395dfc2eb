"""The mbarrier phases that the paged kernels wait for (csrc/fa_paged_phases.h), walked on
the host over every order of completions. No kernel is launched.

A barrier counts the phases it has completed; a wait for a parity passes while the phase
in progress has the other one."""

import ctypes
import os
import shutil
import subprocess

import pytest

import exact_attention_80_gb300 as fa

CSRC = os.path.join(os.path.dirname(os.path.abspath(fa.__file__)), "csrc")

SOURCE = """
#include "fa_paged_phases.h"
extern "C" {
int pv_barrier(int j, int n) { return fa::wide_pv_barrier(j, n); }
unsigned pv_parity(int j, int n) { return fa::wide_pv_parity(j, n); }
int slot(int k, int stages) { return fa::ring_slot(k, stages); }
unsigned parity(int k, int stages) { return fa::ring_parity(k, stages); }
int issued(int k, int stages, int tiles) { return fa::ring_issued(k, stages, tiles); }
}
"""


@pytest.fixture(scope="module")
def phases(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    at = tmp_path_factory.mktemp("phases")
    src, lib = at / "phases.cpp", at / "phases.so"
    src.write_text(SOURCE)
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(lib)],
                   check=True)
    return ctypes.CDLL(str(lib))


def passes(completed, parity):
    """Whether a wait for ``parity`` passes on a barrier with ``completed`` phases behind it."""
    return (completed & 1) != parity


def test_wide_heads_wait_for_the_last_product(phases):
    """d = 256: behind its last arrival a softmax warp reads O once every product of P and V is done, and it
    gets there wherever the tensor core is when the warp comes to poll."""
    for n in range(1, 12):
        bar, parity = phases.pv_barrier(n - 1, n), phases.pv_parity(n - 1, n)
        for done in range(max(0, n - 2), n + 1):  # products finished at a poll: S of the last tile told of n - 2
            completed = [sum(phases.pv_barrier(j, n) == b for j in range(done)) for b in range(2)]
            assert passes(completed[bar], parity) == (done == n), (n, done)


def test_wide_heads_wait_for_the_product_before(phases):
    """d = 256: a warp that rescales O at step j waits for the product of step j - 1, and gets there; those of
    step j and later wait for its P."""
    for n in range(2, 12):
        for j in range(1, n):
            bar, parity = phases.pv_barrier(j - 1, n), phases.pv_parity(j - 1, n)
            for done in (j - 1, j):
                completed = [sum(phases.pv_barrier(i, n) == b for i in range(done)) for b in range(2)]
                assert passes(completed[bar], parity) == (done == j), (n, j, done)


@pytest.mark.parametrize("stages", [2, 3])
def test_a_warp_that_gives_up_waits_for_its_copies(phases, stages):
    """Few rows: a warp whose wait for tile k ran out leaves its ring only when all copies that it started have
    landed, whatever the tile, and whichever of them land first."""
    for tiles in range(1, 4 * stages + 2):
        for k in range(tiles):
            # The loop's own order: the first `stages` tiles, then tile i + stages behind tile i.
            started = list(range(min(stages, tiles))) + [i + stages for i in range(k) if i + stages < tiles]
            flying = [e for e in started if e >= k]  # tiles before k were waited for one by one
            assert flying == list(range(k, phases.issued(k, stages, tiles)))
            for landed in range(1 << len(flying)):
                done = set(range(k)) | {e for i, e in enumerate(flying) if landed >> i & 1}
                completed = [sum(e % stages == s for e in done) for s in range(stages)]
                waits = [passes(completed[phases.slot(e, stages)], phases.parity(e, stages))
                         for e in range(k, phases.issued(k, stages, tiles))]
                assert all(waits) == (len(done) == len(started))
