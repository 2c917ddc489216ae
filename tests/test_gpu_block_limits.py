"""Calls near the ends of the documented ranges on the GPU: more rows than one launch's
grid holds."""
import gc

import pytest
import torch

from pruned_expert_backward_amd import lrmoe as L

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from tests.test_gpu_forward import BF16, DEV, gen, normal  # noqa: E402

U8, I32 = torch.uint8, torch.int32


@pytest.fixture(autouse=True)
def memory():
    """These take tens of GB: nothing of them stays for the next test."""
    yield
    gc.collect()
    torch.cuda.empty_cache()


def test_quantize_more_rows_than_a_grid():
    """2^30 rows and more of one block each; the rows around the places where one
    launch ends (2^30 - 64 rows) and the call does are as if they were alone."""
    T, D, n = 2 ** 30 + 70, 16, 300
    x = torch.zeros(T, D, dtype=BF16, device=DEV)
    tail = normal(gen(3), (n, D), BF16).to(DEV)
    x[-n:], x[:n] = tail, tail.flip(0)
    out, ref = L.quantize_rows(x), L.quantize_rows(tail)
    assert torch.equal(out["q"][-n:].view(U8), ref["q"].view(U8))
    assert torch.equal(out["scale"][-n:], ref["scale"])
    assert torch.equal(out["q"][:n].view(U8), ref["q"].view(U8).flip(0))
    assert torch.equal(out["scale"][:n], ref["scale"].flip(0))
    assert bool((out["scale"][n:-n].view(I32) == 0x7F7F7F7F).all())
    assert int(out["q"][n:-n].view(U8).view(-1).view(torch.int64).max()) == 0
    assert int(out["q"][n:-n].view(U8).view(-1).view(torch.int64).min()) == 0
