"""The in-tree build: what it leaves behind when a compiler fails, and that no compiled file is kept in the repository.
The compilers are stand-ins that write their output file, or fail."""
import os
import shutil
import subprocess

import pytest
import torch

from paged_kv_cache_185_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# writes "made" into the file after -o; fails if one of its arguments is $FAIL_ON (with the output already there)
COMPILER = """#!/bin/sh
rc=0; out=
for a in "$@"; do
  if [ "$prev" = "-o" ]; then out=$a; fi
  case "$a" in *"$FAIL_ON") rc=1;; esac
  prev=$a
done
echo made > "$out"
exit $rc
"""


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A package folder of its own with stand-in compilers."""
    pkg, tools = tmp_path / "pkg", tmp_path / "tools"
    for d in (pkg, tools):
        d.mkdir()
    for name in ("nvcc", "g++"):
        (tools / name).write_text(COMPILER)
        (tools / name).chmod(0o755)
    monkeypatch.setenv("PATH", f"{tools}{os.pathsep}{os.environ['PATH']}")
    monkeypatch.setenv("NVCC", str(tools / "nvcc"))
    monkeypatch.setenv("FAIL_ON", "nothing")
    for name, file in (("BUILD", "_build"), ("LIB", "libwllm.so"), ("DESCRIBE", "_describe.so"),
                       ("STAMP", "_build/describe.stamp")):
        monkeypatch.setattr(build, name, str(pkg / file))
    return pkg


def test_a_build_leaves_its_outputs_alone_in_the_package(tree):
    assert build.build() == str(tree / "libwllm.so")
    assert sorted(os.listdir(tree)) == ["_build", "_describe.so", "libwllm.so"]
    assert not [f for f in os.listdir(tree / "_build") if f.endswith(".tmp")]
    assert build.up_to_date()


def test_another_torch_or_python_means_a_rebuild(tree, monkeypatch):
    build.build()
    assert build.described_for() == build.describe_key() and build.up_to_date()
    monkeypatch.setattr(torch, "__version__", "9.9")
    assert not build.up_to_date()
    build.build()
    assert build.up_to_date() and "9.9" in build.described_for()
    monkeypatch.setattr(build.sysconfig, "get_config_var", lambda name: "cpython-399")
    assert not build.up_to_date()
    os.remove(build.STAMP)
    assert not build.up_to_date()  # a module of which nothing says what it was made for


def test_calls_refuse_a_module_made_for_another_torch(monkeypatch):
    from paged_kv_cache_185_gb300 import binding
    build.build()
    monkeypatch.setattr(binding, "_invoke", None)
    monkeypatch.setattr(build, "described_for", lambda: "cpython-399 torch 9.9")
    with pytest.raises(ImportError, match="built for 'cpython-399 torch 9.9'"):
        binding._load_calls()


@pytest.mark.parametrize("fail", ["select.cu", "describe.cpp", "-shared"])
def test_a_failed_build_leaves_nothing_behind(tree, monkeypatch, fail):
    (tree / "libwllm.so").write_text("before")
    (tree / "_describe.so").write_text("before")
    monkeypatch.setenv("FAIL_ON", fail)
    with pytest.raises(RuntimeError, match="failed"):
        build.build(force=True)
    assert sorted(os.listdir(tree)) == ["_build", "_describe.so", "libwllm.so"]
    assert not [f for f in os.listdir(tree / "_build") if f.endswith(".tmp")]
    for name in ("libwllm.so", "_describe.so"):
        assert (tree / name).read_text() == "before"


def test_no_compiled_file_is_tracked():
    if shutil.which("git") is None or not os.path.isdir(os.path.join(ROOT, ".git")):
        pytest.skip("no repository here")
    files = subprocess.run(["git", "ls-files", "-z"], cwd=ROOT, capture_output=True, check=True).stdout.split(b"\0")
    compiled = []
    for name in filter(None, files):
        try:
            with open(os.path.join(ROOT.encode(), name), "rb") as f:
                if f.read(4) == b"\x7fELF":
                    compiled.append(name)
        except FileNotFoundError:
            pass
    assert not compiled
