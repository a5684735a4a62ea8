"""The paged cache's extension module beside the library: who needs it, when it is built."""
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAME = "blockwise_exact_attention_block_b200"


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__._build_module().build()


def package(where, module=None):
    """The package in `where`, with its library but with `module` in the place of the extension module."""
    pkg = where / NAME
    pkg.mkdir()
    for f in os.listdir(os.path.join(ROOT, NAME)):
        if f.endswith((".py", ".so")) and f != "_paged.so":
            os.symlink(os.path.join(ROOT, NAME, f), pkg / f)
    if module is not None:
        (pkg / "_paged.so").write_bytes(module)
    return where


USE = f"""
import sys, torch
import {NAME} as ra
assert ra.__file__.startswith(sys.argv[1])
assert ra.ra_status_string(0) and ra.ra_paged_decode_workspace(1, 1, 8, 2, 128) > 0
try:
    ra.ra_merge_partial(*(torch.zeros(4, 64) for _ in range(4)))
except ValueError:
    pass  # (host tensors: the older calls' own refusal)
for _ in range(2):
    try:
        ra.ra_cache_read(*(torch.zeros(1) for _ in range(4)), 1)
    except ImportError as e:
        assert "_paged" in str(e)
    else:
        raise SystemExit("the paged call did not fail")
print("done")
"""


@pytest.mark.parametrize("module", [None, b"not a shared object"])
def test_older_calls_do_not_need_the_module(tmp_path, module):
    """Without the extension module, or with one that does not load, the package imports, its other
    calls work and the paged ones fail loudly."""
    where = package(tmp_path, module)
    res = subprocess.run([sys.executable, "-c", USE, str(where)], cwd=where, capture_output=True, text=True,
                         env=dict(os.environ, PYTHONPATH=str(where)))
    assert res.returncode == 0 and "done" in res.stdout, res.stdout + res.stderr


def build_module(where):
    """build.py as it is, for a tree of its own in `where`."""
    import importlib.util
    pkg = where / NAME
    pkg.mkdir()
    for d, to in (("csrc", pkg), ):
        os.symlink(os.path.join(ROOT, NAME, d), to / d)
    os.symlink(os.path.join(ROOT, "include"), where / "include")
    path = pkg / "build.py"
    path.write_bytes(open(os.path.join(ROOT, NAME, "build.py"), "rb").read())
    spec = importlib.util.spec_from_file_location("a_build", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


class Compilers:
    """Stands in for subprocess.run: notes what would be compiled and writes its output."""

    def __init__(self, monkeypatch, mod, text=b""):
        self.made = []
        monkeypatch.setattr(mod.subprocess, "run", self.run)
        self.text = text

    def run(self, cmd, **_):
        out = cmd[cmd.index("-o") + 1]
        tags = [x[len("-DRA_BINDING_TAG="):].strip('"').encode() + b"\0" for x in cmd if x.startswith("-DRA_BINDING_TAG=")]
        with open(out, "wb") as f:
            f.write(b"".join(tags))
        self.made.append(os.path.basename(out).removesuffix(".tmp"))
        return subprocess.CompletedProcess(cmd, 0, "", "")


def test_the_checked_build_makes_the_module_too(tmp_path, monkeypatch):
    mod = build_module(tmp_path)
    c = Compilers(monkeypatch, mod)
    mod.build(debug_bounds=True)
    assert sorted(c.made) == ["_paged.so", "libra_b200_debug.so"]
    mod.build(debug_bounds=True)
    mod.build()
    assert sorted(c.made) == ["_paged.so", "libra_b200.so", "libra_b200_debug.so"]


def test_another_torch_or_python_has_the_module_made_anew(tmp_path, monkeypatch):
    import importlib.metadata
    mod = build_module(tmp_path)
    c = Compilers(monkeypatch, mod)
    mod.build_binding()
    mod.build_binding()
    assert c.made == ["_paged.so"]
    version = importlib.metadata.version("torch")
    monkeypatch.setattr(importlib.metadata, "version", lambda name: version + ".1")
    mod.build_binding()
    mod.build_binding()
    assert c.made == ["_paged.so"] * 2


def test_the_module_names_what_it_was_built_for():
    import __graft_entry__
    import blockwise_exact_attention_block_b200 as ra
    assert ra._paged().built_for == __graft_entry__._build_module().binding_tag()
    assert torch.__version__ in ra._paged().built_for
