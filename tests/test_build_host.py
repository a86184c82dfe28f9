"""The build script without torch and without a C++ compiler: the library needs nvcc
alone.  nvcc is a stand-in here that only writes its output file."""
import os
import shutil
import subprocess
import sys

import pytest

import mixed_precision_quantized_quantize_b200 as q

PACKAGE = os.path.dirname(q.LIB_PATH)


@pytest.fixture
def tree(tmp_path):
    """A copy of the sources, a stand-in nvcc and a torch that cannot be imported."""
    package = tmp_path / "package"
    shutil.copytree(os.path.join(PACKAGE, "csrc"), package / "csrc")
    shutil.copy(os.path.join(PACKAGE, "build.py"), package)
    shutil.copytree(os.path.join(os.path.dirname(PACKAGE), "include"), tmp_path / "include")
    nvcc = tmp_path / "nvcc"
    nvcc.write_text('#!/bin/sh\nwhile [ "$1" != -o ]; do shift; done\necho built > "$2"\n')
    nvcc.chmod(0o755)
    (tmp_path / "no_torch").mkdir()
    (tmp_path / "no_torch" / "torch.py").write_text('raise ImportError("no torch here")\n')

    def run(*options, torch=False):
        env = dict(os.environ, NVCC=str(nvcc), CXX=str(tmp_path / "no_compiler"))
        if not torch:
            env["PYTHONPATH"] = str(tmp_path / "no_torch")
        return subprocess.run([sys.executable, str(package / "build.py"), *options], env=env, capture_output=True,
                              text=True, timeout=300)

    return package, run


def test_the_library_needs_neither_torch_nor_a_compiler(tree):
    package, run = tree
    for options, lib in (((), "libquik_b200.so"), (("--checks",), "libquik_b200_checked.so"),
                         (("--force",), "libquik_b200.so")):
        r = run(*options)
        assert r.returncode == 0, r.stderr
        assert r.stdout.strip().endswith(lib) and (package / lib).read_text() == "built\n"
        # the part that was left out is named, unless it was not asked for
        assert ("_calls" in r.stderr) == (options != ("--checks",))
    assert not (package / "_calls.so").exists()


def test_a_compiler_that_is_missing_leaves_the_library(tree):
    package, run = tree
    r = run(torch=True)
    assert r.returncode == 0 and "_calls" in r.stderr, r.stderr
    assert (package / "libquik_b200.so").exists()


def test_an_extension_of_older_sources_does_not_stay(tree):
    """What cannot be built again is not left to be loaded against another header."""
    package, run = tree
    old = package / "_calls.so"
    old.write_text("old")
    os.utime(old, (0, 0))
    assert run().returncode == 0
    assert not old.exists()
