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


@pytest.mark.parametrize("d_out,d_in", [(2056, 2 ** 20), (2 ** 20, 2064)])
@pytest.mark.parametrize("P", [3, 300])
def test_quantized_product_of_an_expert_beyond_a_buffer(d_out, d_in, P):
    """Weights of more than 2 GiB: zeros but for blocks at their ends, whose product alone is
    within one buffer.  (The blocks of zeros add nothing; the others' sums may come in
    another order, each side off by the product's own bound.)"""
    from oracle import block_oracle as B
    from oracle import forward_oracle as O
    from tests.test_gpu_block import product_error
    g = gen(d_in % 1000)
    near, n = 256 + d_in % 128, 256
    W = normal(g, (1, n, near), BF16, 0.1)
    x = normal(g, (P, near), BF16)
    x8, W8 = L.quantize_rows(x.to(DEV)), L.quantize_weights(W.to(DEV))
    last = d_in % 128 or 128                  # columns of the last block
    cols = torch.cat([torch.arange(near - last), torch.arange(d_in - last, d_in)])
    # the first and the last block of rows, where the last one is whole
    rows = torch.arange(256) if d_out % 128 else torch.cat([torch.arange(128),
                                                            torch.arange(d_out - 128, d_out)])
    big = dict(q=torch.zeros(1, d_out, d_in, dtype=U8, device=DEV),
               scale=torch.full((1, -(-d_out // 128), L.scale_row_bytes(d_in)), 127, dtype=U8,
                                device=DEV))
    wide = dict(q=torch.zeros(P, d_in, dtype=U8, device=DEV),
                scale=torch.full((P, L.scale_row_bytes(d_in)), 127, dtype=U8, device=DEV))
    big["q"][0, rows.to(DEV)[:, None], cols.to(DEV)] = W8["q"].view(U8)[0]
    wide["q"][:, cols.to(DEV)] = x8["q"].view(U8)
    kb, nb = cols[::128] // 128, rows[::128] // 128
    wide["scale"][:, kb.to(DEV)] = x8["scale"][:, :len(kb)]
    big["scale"][0, nb.to(DEV)[:, None], kb.to(DEV)] = W8["scale"][0, :, :len(kb)]
    as8 = lambda t: dict(q=t["q"].view(L.FP8), scale=t["scale"])   # noqa: E731
    seg = torch.tensor([0, P], dtype=I32, device=DEV)
    y = L.grouped_forward_quantized(seg, as8(wide), as8(big))["y"]
    want = L.grouped_forward_quantized(seg, x8, W8)["y"].cpu().double()
    ref = O.linear([0, P], B.row_values(x8["q"].cpu(), x8["scale"].cpu()),
                   B.weight_values(W8["q"].cpu(), W8["scale"].cpu()))
    e = product_error([0, P], x8, W8, None, ref["mag"])
    assert bool(((y[:, rows.to(DEV)].cpu().double() - want).abs()
                 <= 2 * e + 2 ** -7 * want.abs()).all())
    y[:, rows.to(DEV)] = 0
    assert int(y.count_nonzero()) == 0


def test_norms_of_rows_beyond_32_bits():
    """Rows whose elements pass 2^32: the first and the last ones as if they were alone."""
    T, D, n = 2 ** 21 + 37, 2048, 70
    g = gen(9)
    few = {k: normal(g, (n, D), BF16).to(DEV) for k in ("x", "y", "ds", "dh")}
    w, wb = (1 + normal(g, (D,), F32, 0.1)).to(BF16).to(DEV), normal(g, (D,), BF16).to(DEV)
    gate = normal(g, (n, 1), F32).to(DEV)
    wide = {k: torch.zeros(T, D, dtype=BF16, device=DEV) for k in few}
    wide["gate"] = torch.zeros(T, 1, device=DEV)
    for k, t in {**few, "gate": gate}.items():
        wide[k][-n:], wide[k][:n] = t, t.flip(0)

    def calls(t, gate):
        out = L.residual_norm(t["x"], y=t["y"], weight=w, branch_weight=wb, gate=gate, scale=0.5)
        d = L.residual_norm_backward(out["s"], ds=t["ds"], dh=t["dh"], y=t["y"], weight=w,
                                     branch_weight=wb, gate=gate, scale=0.5)
        return dict(s=out["s"], h=out["h"], dx=d["dx"], dy=d["dy"], dgate=d["dgate"])
    got, want = calls(wide, wide["gate"]), calls(few, gate)
    for k in want:
        assert torch.equal(got[k][-n:], want[k]), k
        assert torch.equal(got[k][:n], want[k].flip(0)), k
        assert int(got[k][n:-n].count_nonzero()) == 0, k
