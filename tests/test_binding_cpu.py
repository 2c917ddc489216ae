"""The Python binding on the host: what loading it needs and how it refuses a
library that does not fit."""
import os
import subprocess
import sys
import types

import pytest

from pruned_expert_backward_amd import lrmoe as L

if not os.path.exists(L.LIB_PATH):
    pytest.skip("liblrmoe.so not built (run __graft_entry__.build())", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def python(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                          timeout=300)


def test_host_side_without_cuda_streams_in_torch():
    """A CPU build of torch has no stream handles; planning needs none."""
    r = python("import torch\n"
               "del torch._C._cuda_getCurrentRawStream\n"
               "from pruned_expert_backward_amd import lrmoe as L\n"
               "print(L.plan_quota([10, 0, 5], ('ratio', 4, 5)))")
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip() == str(L.plan_quota([10, 0, 5], ("ratio", 4, 5)))


def test_library_of_an_older_version_is_named_as_such(monkeypatch):
    """Version 4 has no forward side: loading it says what to do, and does not
    end at the first symbol that it lacks."""
    def version():
        return 4

    monkeypatch.setattr(L, "_lib_handle", None)
    monkeypatch.setattr(L.C, "CDLL", lambda path: types.SimpleNamespace(lrmoe_abi_version=version))
    with pytest.raises(RuntimeError, match="rebuild"):
        L.lib()
