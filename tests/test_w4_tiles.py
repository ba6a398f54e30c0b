"""Addresses of the weights' loads in products with group-scaled 4-bit weights, on the host: the
functions that the kernels form them with (csrc/w4_tiles.h), for every lane, at every number of
columns up to 600 and several lengths, each workgroup's shape and each wave."""
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))


def test_loads_stay_within_the_weights(tmp_path):
    exe = tmp_path / "w4_tiles"
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-o", str(exe), os.path.join(HERE, "w4_tiles_main.cpp")], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout
