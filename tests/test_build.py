"""The built modules: that they belong together wherever the tree lies.  Runs on the CPU: nothing is launched."""
import os
import shutil
import subprocess
import sys

import pytest

from lossless_draft_verification_online_amd import build

NAME = os.path.basename(build.PKG)


@pytest.fixture(scope="module", autouse=True)
def _built():
    if build.is_stale():
        pytest.fail("libsdv.so or _marshal.so is missing or older than its sources; run __graft_entry__.build()")


@pytest.fixture
def copy(tmp_path):
    """The built package in another directory."""
    shutil.copytree(build.PKG, tmp_path / NAME, ignore=shutil.ignore_patterns("csrc", "__pycache__"))
    return tmp_path


def run(where, code):
    return subprocess.run([sys.executable, "-c", code], cwd=where, capture_output=True, text=True, timeout=300)


def test_modules_name_no_directory():
    said = subprocess.run(["readelf", "-d", build.LIBRARY, build.MARSHAL], capture_output=True, text=True, check=True).stdout
    needed = [line.split("[")[1].split("]")[0] for line in said.splitlines() if "(NEEDED)" in line]
    assert "libsdv.so" in needed and not [n for n in needed if "/" in n]


def test_a_copy_uses_its_own_library(copy):
    got = run(copy, f"from {NAME} import _native\n_native.marshal()\n"
                    "print(*sorted({line.split()[-1] for line in open('/proc/self/maps') if 'libsdv' in line}))")
    assert got.returncode == 0, got.stderr
    assert got.stdout.split() == [str(copy.resolve() / NAME / "libsdv.so")]


def test_a_module_that_does_not_load_says_why(copy):
    at = copy / NAME / "_marshal.so"
    at.write_bytes(bytes(4096))
    got = run(copy, f"from {NAME} import _native\n_native.marshal()")
    assert got.returncode != 0 and "RuntimeError" in got.stderr
    last = got.stderr.strip().splitlines()[-1]
    assert "is not built" not in last and f"{at.resolve()}: invalid ELF header" in last, last
    at.unlink()
    got = run(copy, f"from {NAME} import _native\n_native.marshal()")
    assert "_marshal.so is not built; run __graft_entry__.build()" in got.stderr.strip().splitlines()[-1]


def test_a_module_older_than_its_sources_is_stale(tmp_path, monkeypatch):
    module = tmp_path / "_marshal.so"
    monkeypatch.setattr(build, "MARSHAL", str(module))
    assert build.is_stale()  # none there
    module.write_bytes(b"")
    for source in (build.MARSHAL_SOURCE, os.path.join(build.ROOT, "include", "sdv.h")):
        t = os.path.getmtime(source)
        os.utime(module, (t - 1, t - 1))
        assert build.is_stale(), source
    os.utime(module, (2 ** 31, 2 ** 31))
    assert not build.is_stale()


def test_the_library_alone_can_be_asked_for(monkeypatch):
    monkeypatch.setattr(build, "MARSHAL", "/nowhere/_marshal.so")
    assert not build.is_stale(build.LIBRARY)
