"""The library's record of how much shared memory a kernel may be launched with, under host threads that ask for different
sizes at the same time (the Python calls run without the interpreter lock): built on the host against a runtime that
tests/csrc/smem_attribute.cpp makes up."""
import os
import subprocess

from hadamard_rotation_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_threads_that_ask_for_different_sizes(tmp_path):
    exe = tmp_path / "smem_attribute"
    cuda = os.path.join(os.path.dirname(os.path.dirname(build.nvcc_path())), "include")
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", build.CSRC, "-I", build.INCLUDE, "-I", cuda, "-x", "c++",
                    os.path.join(HERE, "csrc", "smem_attribute.cpp"), os.path.join(build.CSRC, "hq_smem.cu"),
                    "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stdout
    assert out.stdout.strip() == "ok"
