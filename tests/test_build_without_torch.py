"""The C library builds, and the calls that need no compiled module work, where that
module cannot be had: no torch, a torch without CUDA, no Python headers, or a module
built against another torch.  The calls that need it say so."""
import importlib.machinery
import importlib.util
import os
import subprocess
import sys

import pytest

from paged_kv_cache_215_gb300 import build as pkv_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _without(monkeypatch, spec):
    real = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec",
                        lambda name, *a: spec if name == "torch" else real(name, *a))


@pytest.mark.parametrize("kind", ["no torch", "a folder of that name", "no CUDA"])
def test_the_library_builds(monkeypatch, tmp_path, kind):
    pkv_build.build()
    monkeypatch.setattr(pkv_build, "BINDING", str(tmp_path / "pkv_tensors.so"))
    spec = None
    if kind != "no torch":
        spec = importlib.machinery.ModuleSpec("torch", None)
        if kind == "no CUDA":
            (tmp_path / "lib").mkdir()
            spec.origin = str(tmp_path / "__init__.py")
    _without(monkeypatch, spec)
    assert pkv_build._binding_job() is None
    assert pkv_build.build() == pkv_build.SO and os.path.exists(pkv_build.SO)


def test_no_python_headers(monkeypatch, tmp_path):
    monkeypatch.setattr(pkv_build, "BINDING", str(tmp_path / "pkv_tensors.so"))
    paths = dict(pkv_build.sysconfig.get_paths(), include=str(tmp_path))
    monkeypatch.setattr(pkv_build.sysconfig, "get_paths", lambda *a: paths)
    assert pkv_build._binding_job() is None


def test_a_torch_of_unknown_version(monkeypatch):
    def unknown(name):
        raise importlib.metadata.PackageNotFoundError(name)

    monkeypatch.setattr(pkv_build.importlib.metadata, "version", unknown)
    where, version = pkv_build._torch()
    assert os.path.isdir(where) and version


CALLS = """
import sys
from paged_kv_cache_215_gb300 import build
build.BINDING = sys.argv[1]
from paged_kv_cache_215_gb300 import pkv
assert pkv.kv_pool_bytes(pkv.geometry(1, 4, 2, 64, 16, 8, "bf16")) > 0
rope, pool = pkv.Rope(16, device="cpu"), object.__new__(pkv.KVPool)
pool.handle = pool.storage = None
for call in (lambda: pkv.rope_apply(None, None, None, rope),
             lambda: pool.append_rope(0, None, None, None, None, rope, None, None),
             lambda: pkv.verify_drafts(None, None, None, None, None, None, None)):
    try:
        call()
    except ImportError as e:
        assert sys.argv[1] in str(e), e
    else:
        raise AssertionError("no error")
print("ok")
"""


@pytest.mark.parametrize("kind", ["missing", "not loadable"])
def test_only_the_calls_that_need_the_module_fail(tmp_path, kind):
    pkv_build.build()
    path = tmp_path / "pkv_tensors.so"
    if kind == "not loadable":
        path.write_text("no library")
    r = subprocess.run([sys.executable, "-c", CALLS, str(path)], cwd=ROOT, capture_output=True,
                       text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr
