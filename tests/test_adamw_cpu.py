"""The AdamW step's refusals on the host that concern more than one argument: nothing is
launched before all of them are checked."""
import ctypes as C
import os

import pytest
import torch

from pruned_expert_backward_amd import lrmoe as L

if not os.path.exists(L.LIB_PATH):
    pytest.skip("liblrmoe.so not built (run __graft_entry__.build())", allow_module_level=True)

FAKE = 0x7F0000001000   # 16-byte aligned; validation fails before any use
SHAPE = 3


@pytest.mark.parametrize("n", [2 ** 36, 2 ** 37, 2 ** 62])
@pytest.mark.parametrize("bits", [32, 8])
def test_a_tensor_of_too_many_elements(n, bits):
    """More elements than a launch holds are refused by their number."""
    cfg = L.AdamW(1e-3, 0.9, 0.95, 1e-8, 0.1, 1, 0)
    scales = (FAKE, FAKE) if bits == 8 else (None, None)
    table = (L.AdamWTensor * 1)(L.AdamWTensor(n, FAKE, FAKE, FAKE, FAKE, *scales, None, L.F32, L.F32))
    assert L.lib().lrmoe_adamw_step(C.byref(cfg), table, 1, None) == SHAPE


def test_a_tensor_that_is_there_twice(monkeypatch):
    """One launch works on all tensors at once: the same parameter or state twice would be a
    race.  Empty ones, and one gradient for several parameters, are none."""
    calls = []
    monkeypatch.setattr(L, "_device", lambda t: t.device)
    monkeypatch.setattr(L, "_call", lambda fn, dev, *args: calls.append(fn))
    p, q, none = (torch.zeros(n) for n in (10, 10, 0))
    g = torch.zeros(10)
    for bits in (32, 8):
        st, s2, s0 = (L.adamw_state(x, bits) for x in (p, q, none))
        with pytest.raises(ValueError, match="params"):
            L.adamw_step([p, p], [g, g], [st, s2], 1, 1e-3)
        with pytest.raises(ValueError, match="states"):
            L.adamw_step([p, none, q], [g, none, g], [st, s0, st], 1, 1e-3)
        with pytest.raises(ValueError, match="params"):
            L.adamw_step([none, p, none, p.view(10)], [none, g, none, g], [s0, st, s0, s2], 1, 1e-3)
        assert calls == []
        L.adamw_step([p, none, q, none], [g, none, g, none], [st, s0, s2, s0], 1, 1e-3)
        assert calls.pop() == "lrmoe_adamw_step"
