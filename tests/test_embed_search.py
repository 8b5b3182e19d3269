"""The search of the embedding gradient for codes without rows, on the host.

Its steps (gmm_search.h) are compiled with g++ and run for many numbers of keys and first places: every
probe that reads a key reads one of them, also while other searches of the wave go on, and the search
ends where it should.
"""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "gmm_em_amd", "csrc")


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("search") / "driver")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-I", CSRC,
                    os.path.join(HERE, "embed_search_driver.cpp"), "-o", exe], check=True)
    return exe


@pytest.mark.parametrize("extra", [0, 1, 12])
def test_probes_are_keys(driver, extra):
    r = subprocess.run([driver, str(extra)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr

