"""Rows of 16-bit elements that are copied to another pitch, on the CPU: the loads stay inside the row."""
import os
import subprocess

from zero_partitioned_optimizer_shard_gb300 import _build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_rows_are_read_inside_their_ends(tmp_path):
    exe = str(tmp_path / "pad_host")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", _build.CSRC,
                    os.path.join(HERE, "pad_host.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
