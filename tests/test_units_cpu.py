"""How the paged prompt attention divides a call among its CTAs: the closed sums of
units.cuh against enumeration, in a program of its own."""
import os
import subprocess

from grouped_query_kv_gb300 import build as gbuild

HERE = os.path.dirname(os.path.abspath(__file__))


def test_the_division_of_a_call_against_enumeration(tmp_path):
    exe = str(tmp_path / "units_check")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-I", gbuild.CSRC,
                    os.path.join(HERE, "units_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
