"""Calls near the ends of the documented ranges on the GPU: more rows than one launch's
grid holds, pair rows up to 2^31."""
import gc

import pytest
import torch

from pruned_expert_backward_amd import lrmoe as L

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from tests.test_gpu_forward import BF16, DEV, F32, gen, normal  # noqa: E402

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


def every_fifth(y, want, P):
    """y's rows are want's five in turn."""
    whole = P // 5
    step = 1 << 24
    for i in range(0, whole, step):
        part = y[5 * i:5 * min(i + step, whole)].view(-1, *want.shape)
        assert bool((part == want).all()), i
    assert torch.equal(y[5 * whole:P], want[:P - 5 * whole])


def fives(P, pick):
    """int32 [P]: the five of pick in turn."""
    at = torch.tensor(pick, dtype=I32, device=DEV).repeat(P // 5 + 1)
    return at[:P].contiguous()


def test_quantized_product_of_more_pairs_than_a_grid():
    """2^30 pairs and more that pick rows of an x beyond a buffer's 2 GiB."""
    P, D, N, T = 2 ** 30 + 77, 16, 8, 2 ** 27 + 3
    g = gen(5)
    x8 = L.quantize_rows(normal(g, (5, D), BF16).to(DEV))
    W8 = L.quantize_weights(normal(g, (2, N, D), BF16).to(DEV))
    pick = [0, T - 1, T - 2, 5, T // 2]
    q = torch.zeros(T, D, dtype=U8, device=DEV)
    s = torch.full((T, 4), 127, dtype=U8, device=DEV)
    for i, t in enumerate(pick):
        q[t], s[t] = x8["q"].view(U8)[i], x8["scale"][i]
    # the second expert has the last 3 to 7 rows, from a multiple of five on
    first = (P - 3) // 5 * 5
    seg = torch.tensor([0, first, P], dtype=I32, device=DEV)
    y = L.grouped_forward_quantized(seg, dict(q=q.view(L.FP8), scale=s), W8,
                                    row_index=fives(P, pick))["y"]
    small = torch.tensor([0, 5, 10], dtype=I32, device=DEV)
    want = L.grouped_forward_quantized(small, x8, W8, row_index=fives(10, list(range(5))))["y"]
    every_fifth(y[:first], want[:5], first)
    assert torch.equal(y[first:], want[5:][torch.arange(P - first) % 5])


@pytest.mark.parametrize("dt,P,T", [(BF16, 2 ** 31 - 1, 0), (BF16, 2 ** 30 + 77, 2 ** 27 + 3),
                                    (F32, 2 ** 30 + 77, 0)])
def test_product_of_more_pairs_than_a_grid(dt, P, T):
    """As many pairs as a call may have: rows in place (T = 0), or picked from an x
    beyond a buffer's 2 GiB."""
    D = N = 16 // dt.itemsize
    g = gen(6)
    few, W = normal(g, (5, D), dt).to(DEV), normal(g, (2, N, D), dt).to(DEV)
    row = None
    if T:
        pick = [0, T - 1, T - 2, 5, T // 2]
        x = torch.zeros(T, D, dtype=dt, device=DEV)
        for i, t in enumerate(pick):
            x[t] = few[i]
        row = fives(P, pick)
    else:
        x = torch.empty(P, D, dtype=dt, device=DEV)
        x[:P // 5 * 5].view(-1, 5, D)[:] = few
        x[P // 5 * 5:] = few[:P % 5]
    first = (P - 3) // 5 * 5
    seg = torch.tensor([0, first, P], dtype=I32, device=DEV)
    y = L.grouped_forward(seg, x, W, row_index=row)["y"]
    small = torch.tensor([0, 5, 10], dtype=I32, device=DEV)
    want = L.grouped_forward(small, few.repeat(2, 1), W)["y"]
    every_fifth(y[:first], want[:5], first)
    assert torch.equal(y[first:], want[5:][torch.arange(P - first) % 5])
