"""The shared-prefix kernel's slots under copies and products that complete at random times, simulated on the host
(prefix_ring_sim.cpp): every ring size, segments of one and two q tiles in any mix.  Two rings that are known to be wrong
have to fail, or the simulation could not tell."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "paged_gqa_decode_05_gb300", "csrc")


@pytest.fixture(scope="module")
def sim(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("sim") / "prefix_ring_sim")
    subprocess.run(["g++", "-std=c++20", "-O2", "-I", CSRC, os.path.join(HERE, "prefix_ring_sim.cpp"), "-o", exe], check=True)
    return lambda runs, seed, ring: subprocess.run([exe, str(runs), str(seed), ring], capture_output=True, text=True, timeout=300)


@pytest.mark.parametrize("seed", [0, 1000, 2000, 3000])
def test_no_slot_is_taken_too_early_and_nobody_waits_for_ever(sim, seed):
    r = sim(75, seed, "own")
    assert r.returncode == 0, r.stdout
    assert r.stdout == "450 runs\n"


@pytest.mark.parametrize("ring", ["one", "eager"])
def test_wrong_rings_fail(sim, ring):
    r = sim(200, 0, ring)
    assert r.returncode == 1 and "slot" in r.stdout, r.stdout
