"""The Python binding on the host: what loading it needs and how it refuses a
library that does not fit."""
import os
import subprocess
import sys
import types

import pytest
import torch

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


@pytest.fixture
def host_calls(monkeypatch):
    """The forward side's binding on CPU tensors: entry points called, none run."""
    calls = []
    monkeypatch.setattr(L, "_device", lambda t: t.device)
    monkeypatch.setattr(L, "_call", lambda fn, dev, *args: calls.append(fn))
    return calls


def z(*shape, dt=torch.bfloat16):
    return torch.zeros(shape, dtype=dt)


def test_options_that_out_has_no_buffer_for(host_calls):
    seg, f32, i32 = z(3, dt=torch.int32), torch.float32, torch.int32
    x, W, y = z(4, 8), z(2, 16, 8), z(4, 16)
    half = dict(y=z(4, 8), pre_a=z(4, 8))
    ids, w = z(4, 2, dt=i32), z(4, 2, dt=f32)
    sort = dict(counts=z(3, dt=torch.int64), seg_offsets=z(4, dt=i32), row_index=z(8, dt=i32),
                pos=z(4, 2, dt=i32))
    bad = [
        (ValueError, lambda: L.grouped_forward(seg, x, W, save_pre=True, out=dict(y=y))),
        (ValueError, lambda: L.grouped_forward(seg, x, W, act=L.ACT_SWIGLU, save_pre=True,
                                               out=half)),
        (ValueError, lambda: L.act_backward(seg, y, dbias=True, out=dict(dz=y))),
        (ValueError, lambda: L.act_backward(seg, y, dbias=True, out=dict(dz=y, dbias=None))),
        (TypeError, lambda: L.act_backward(seg, y, dz_dtype=f32, out=dict(dz=z(4, 16)))),
        (ValueError, lambda: L.route_sort(ids, 3, weights=w, out=sort)),
    ]
    for n, (err, call) in enumerate(bad):
        with pytest.raises(err):
            call()
            pytest.fail(f"call {n} was taken")
    assert host_calls == []


def test_out_decides_what_is_stored(host_calls):
    """Buffers that stand in out are filled whatever the options' defaults."""
    seg, f32 = z(3, dt=torch.int32), torch.float32
    y = z(4, 16)
    L.grouped_forward(seg, z(4, 8), z(2, 16, 8), out=dict(y=y, pre_a=z(4, 16)))
    L.grouped_forward(seg, z(4, 8), z(2, 16, 8), out=dict(y=y))
    assert "dbias" not in L.act_backward(seg, y, out=dict(dz=z(4, 16)))
    both = dict(dz=z(4, 16, dt=f32), dbias=z(2, 16, dt=f32))
    assert L.act_backward(seg, y, dz_dtype=f32, out=both) is both
    assert L.act_backward(seg, y)["dbias"].shape == (2, 16)
    assert L.act_backward(seg, y, dbias=False)["dbias"] is None
    assert len(host_calls) == 6
