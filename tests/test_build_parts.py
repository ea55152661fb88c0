"""libhq.so and the module of its torch calls are built apart: what the module needs and does not find must not cost a C
caller the library, and a module of another torch is built again."""
import os
import subprocess

import pytest

from hadamard_rotation_gb300 import build


@pytest.fixture
def small(tmp_path, monkeypatch):
    """A library of one small source, and a module beside it, in a folder of their own."""
    src = tmp_path / "hq_small.cu"
    src.write_text('extern "C" __attribute__((visibility("default"))) int hq_small() { return 7; }\n')
    monkeypatch.setattr(build, "CSRC", str(tmp_path))
    monkeypatch.setattr(build, "SOURCES", [str(src)])
    monkeypatch.setattr(build, "DEPS", [str(src)])
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libhq.so"))
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "_torch_calls.so"))
    return tmp_path


def left(folder):
    return sorted(p for p in os.listdir(folder) if not p.endswith(".cu"))


def test_a_module_that_does_not_compile(small, monkeypatch):
    monkeypatch.setattr(build, "calls_compile_command", lambda src, obj: ["false"])
    with pytest.raises(subprocess.CalledProcessError, match="hq_torch"):
        build.build()
    assert left(small) == ["libhq.so"]


def test_no_compiler_and_no_headers_for_the_module(small, monkeypatch):
    def nothing(src, obj):
        raise ImportError("no torch")

    monkeypatch.setattr(build, "calls_compile_command", nothing)
    with pytest.raises(ImportError, match="no torch"):
        build.build()
    assert left(small) == ["libhq.so"]
    os.remove(build.LIB)
    monkeypatch.setattr(build, "calls_compile_command", lambda src, obj: ["/nowhere/g++"])
    with pytest.raises(OSError):
        build.build()
    assert left(small) == ["libhq.so"]


def test_the_library_alone(small, monkeypatch):
    monkeypatch.setattr(build, "calls_compile_command", None)  # not asked for
    assert build.build(calls=False) == build.LIB
    assert left(small) == ["libhq.so"]


def test_a_library_that_does_not_compile(small):
    (small / "hq_small.cu").write_text("this is no C++\n")
    with pytest.raises(subprocess.CalledProcessError, match="hq_small"):
        build.build(calls=False)
    assert left(small) == []


def test_a_module_of_another_torch_is_built_again(monkeypatch):
    import torch

    build.build()
    assert build.up_to_date()
    monkeypatch.setattr(torch, "__version__", "0.0.1+none")
    assert not build.up_to_date() and build.library_up_to_date()
