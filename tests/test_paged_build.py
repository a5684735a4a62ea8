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
