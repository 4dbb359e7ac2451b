"""The committed sources compile, and a build that fails leaves nothing to load."""
import concurrent.futures as cf
import os
import shutil
import subprocess

import pytest

from conftest import ROOT
from vq_dequant_matmul_amd import _build

PACKAGE = "vq_dequant_matmul_amd"


def _sources():
    """Files of the native library: the tracked ones where there is a checkout."""
    dirs = ["include", f"{PACKAGE}/csrc"]
    if os.path.isdir(os.path.join(ROOT, ".git")):
        out = subprocess.run(["git", "-C", ROOT, "ls-files", "-z", "--", *dirs],
                             capture_output=True, text=True, check=True).stdout
        return [f for f in out.split("\0") if f]
    return [os.path.join(d, f) for d in dirs for f in os.listdir(os.path.join(ROOT, d))]


def test_every_source_compiles_from_a_copy(tmp_path):
    for f in _sources():
        dst = tmp_path / f
        dst.parent.mkdir(parents=True, exist_ok=True)
        shutil.copyfile(os.path.join(ROOT, f), dst)

    def check(src):
        r = subprocess.run([*_build.compile_command(src, str(tmp_path)), "-fsyntax-only"],
                           capture_output=True, text=True)
        return src, r.returncode, r.stderr

    with cf.ThreadPoolExecutor(4) as ex:
        results = list(ex.map(check, _build.SOURCES))
    bad = [f"{src}:\n{err[-2000:]}" for src, rc, err in results if rc]
    assert not bad, "\n".join(bad)


def test_every_native_source_is_built():
    units = {os.path.basename(f) for f in _sources() if f.endswith((".hip", ".cpp"))}
    assert units == set(_build.SOURCES)


def test_a_failed_build_leaves_no_library(tmp_path, monkeypatch):
    csrc = tmp_path / PACKAGE / "csrc"
    csrc.mkdir(parents=True)
    (csrc / "a.cpp").write_text("int f() { return 1; }\n")
    (csrc / "b.cpp").write_text("int g() { return no_such_name; }\n")
    monkeypatch.setattr(_build, "BUILD", str(tmp_path / "obj"))
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(_build, "SOURCES", ["a.cpp", "b.cpp"])
    command = _build.compile_command
    monkeypatch.setattr(_build, "compile_command", lambda src: command(src, str(tmp_path)))
    (tmp_path / "obj").mkdir()
    for old in ("lib.so", "obj/b.o"):
        (tmp_path / old).write_text("of an earlier build")
    with pytest.raises(RuntimeError, match="no_such_name"):
        _build.build()
    assert not (tmp_path / "lib.so").exists() and not (tmp_path / "obj" / "b.o").exists()
    (csrc / "b.cpp").write_text("int g() { return 2; }\n")
    assert os.path.getsize(_build.build()) > 0
