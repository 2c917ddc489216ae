"""The grouped product's tile kernels on the GPU against the float64 oracle:
single-row tiles, long K, every epilogue, rows by index and in place, more pair
capacity than pairs, offsets out of order.

The shapes go by the launch's rule, the workgroups that a call is expected to
have; error bounds are those of test_gpu_forward.py."""
import pytest
import torch

from oracle import forward_oracle as O
from pruned_expert_backward_amd import lrmoe as L

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from tests.test_gpu_forward import (  # noqa: E402
    ACTS, BF16, DEV, F32, HALF, U, act_bound, check_linear, gen, linear_inputs, normal, within)

# name: (segments, columns of y without SwiGLU).  Each holds one-row segments.
TILES = {
    "few rows": ([0, 1, 3, 20, 21], 136),
    "32x256": ([0, 1, 2] + list(range(10, 508, 8)) + [510, 512], 776),
    "32x64": ([0, 1, 120, 121, 300], 1032),
    "64x64": ([0, 1, 600, 601, 1200], 1032),
    "64x128": ([0, 1, 1250, 1251, 2500], 1032),
    "128 rows": ([0, 1, 2045, 2046, 4090], 1032),   # one round of them
    # whole 256-row tiles, ends of each class, one row
    "256 rows": ([0, 1500, 1501, 1600, 4200], 2056),
}


def inputs(tile, name, dt, d_in, seed, index, spare=0):
    seg, F = TILES[tile]
    F = F // 16 * 8 if name == "swiglu" else F   # as many rows of W
    return (seg,) + linear_inputs(seg, d_in, 2 * F if name == "swiglu" else F, dt, seed,
                                  spare=spare, index=index, name=name)


@pytest.mark.parametrize("tile", list(TILES))
@pytest.mark.parametrize("name,d_in", [("none", 8), ("swiglu", 776)])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_one_row_tiles_in_place(tile, name, d_in, dt):
    """A tile of one row without a row index reads one row of x: the loads
    ahead of the products go on past the end of K, behind that row."""
    seg, x, W, _, bias, res = inputs(tile, name, dt, d_in, 101, index=False)
    check_linear(seg, x, W, None, bias, res, name, True)


@pytest.mark.parametrize("tile", list(TILES))
@pytest.mark.parametrize("name", ["none", "swiglu"])
@pytest.mark.parametrize("d_in", [776, 2056])
def test_long_rows(tile, name, d_in):
    """13 and 33 steps of K with a ragged end: every LDS stage is refilled many
    times.  Bias, residual and pre-activations all on."""
    seg, x, W, row, bias, res = inputs(tile, name, BF16, d_in, 102, index=True)
    check_linear(seg, x, W, row, bias, res, name, True)


@pytest.mark.parametrize("tile", ["few rows", "64x64"])
@pytest.mark.parametrize("name", ["none", "swiglu"])
@pytest.mark.parametrize("d_in", [388, 1028])
def test_long_rows_float32(tile, name, d_in):
    seg, x, W, row, bias, res = inputs(tile, name, F32, d_in, 103, index=True)
    check_linear(seg, x, W, row, bias, res, name, True)


@pytest.mark.parametrize("tile", list(TILES))
@pytest.mark.parametrize("name", list(ACTS))
@pytest.mark.parametrize("bias,residual,pre,index", [(False, False, True, True),
                                                     (True, True, False, False)])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_epilogues(tile, name, bias, residual, pre, index, dt):
    seg, x, W, row, b, r = inputs(tile, name, dt, 136, 104, index=index)
    check_linear(seg, x, W, row, b if bias else None, r if residual else None, name, pre)


@pytest.mark.parametrize("tile", list(TILES))
@pytest.mark.parametrize("name", ["silu", "swiglu"])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_rows_out_of_range_and_masked_values(tile, name, dt):
    """Indices outside x read zero rows; NaN in rows of x that no pair names
    and in the weights of an expert without rows reach nothing."""
    seg, F = TILES[tile]
    seg = seg + [seg[-1]]                     # one more expert, no rows
    F = F // 16 * 8 if name == "swiglu" else F
    x, W, row, bias, _ = linear_inputs(seg, 200, 2 * F if name == "swiglu" else F, dt, 105,
                                       name=name)
    T, P = x.shape[0], row.numel()
    for u, r in ((0, -1), (P // 2, T), (P - 1, 2 ** 31 - 1), (P // 3, -2 ** 31)):
        row[u] = r
    named = torch.zeros(T, dtype=torch.bool)
    named[row[(row >= 0) & (row < T)].long()] = True
    x[~named] = float("nan")
    bad = W.clone()
    bad[-1] = float("nan")
    # the oracle skips experts without rows, so it takes the same weights
    check_linear(seg, x, bad, row, bias, None, name, True)


@pytest.mark.parametrize("tile", list(TILES))
@pytest.mark.parametrize("name", ["gelu", "swiglu"])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_an_eighth_of_the_capacity(tile, name, dt):
    """Pair rows for eight times the pairs, as a rank that holds an eighth of
    the experts gets them from the sort: token -1 behind the last pair.  The
    rows there stay as they were."""
    full, F = TILES[tile]
    seg = [o // 8 for o in full]
    F = F // 16 * 8 if name == "swiglu" else F
    x, W, row, bias, res = linear_inputs(seg, 136, 2 * F if name == "swiglu" else F, dt, 106,
                                         spare=full[-1] - seg[-1], name=name)
    row[seg[-1]:] = -1
    check_linear(seg, x, W, row, bias, res, name, True)


def covered(seg, P):
    """Clamped segments as the kernels read them: the expert of each row of P
    (-1: none, -2: several)."""
    at = [min(max(o, 0), P) for o in seg]
    e = torch.full((P,), -1)
    for i in range(len(seg) - 1):
        for u in range(at[i], at[i + 1]):
            e[u] = i if e[u] == -1 else -2
    return e


@pytest.mark.parametrize("tile", list(TILES))
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("order", [0, 1, 2])
def test_offsets_out_of_order_in_tiles(tile, dt, order):
    """Offsets that do not ascend or leave the rows are bounded: nothing outside
    y is written, rows of no segment stay, and a row of one segment holds that
    expert's values or, where the order names more tiles than P rows can have,
    what it held before."""
    F, guard, E = TILES[tile][1], 300, 4
    P = TILES[tile][0][-1]
    seg = [[-5, P // 3, P // 3, 2 ** 31 - 1, 0],             # every row once
           [0, P // 2, P // 4, P + 50, P - P // 8],          # some twice
           [P + 50, P + 60, -7, -9, -2 ** 31]][order]        # none
    g = gen(107)
    x, W = normal(g, (P, 72), dt), normal(g, (E, F, 72), dt, 0.1)
    buf = torch.full((P + 2 * guard, F), 5.0, dtype=dt, device=DEV)
    s = torch.tensor(seg, dtype=torch.int32, device=DEV)
    L.grouped_forward(s, x.to(DEV), W.to(DEV), out=dict(y=buf[guard:guard + P]))
    got = buf.cpu().double()
    assert (got[:guard] == 5.0).all() and (got[guard + P:] == 5.0).all()
    got, own = got[guard:guard + P], covered(seg, P)
    assert torch.isfinite(got).all()
    assert (got[own == -1] == 5.0).all()
    for e in range(E):
        at = own == e
        ref = O.linear([0, int(at.sum())], x[at], W[e:e + 1])
        bound = 74 * 2 * U * ref["mag"]
        right = (got[at] - ref["y"]).abs() <= bound + HALF[dt] * (ref["y"].abs() + bound)
        assert (right | (got[at] == 5.0) & (order == 1)).all()
    # the epilogue's gradient over the same offsets
    dy = normal(g, (P, 40), dt)
    buf = torch.full((P + 2 * guard, 40), 5.0, dtype=dt, device=DEV)
    db = torch.empty((E, 40), device=DEV)
    L.act_backward(s, dy.to(DEV), act=L.ACT_NONE, out=dict(dz=buf[guard:guard + P], dbias=db))
    got = buf.cpu()
    assert (got[:guard] == 5.0).all() and (got[guard + P:] == 5.0).all()
    got = got[guard:guard + P]
    assert (got[own == -1] == 5.0).all()
    once = own >= 0
    assert ((got[once] == dy[once]) | (got[once] == 5.0) & (order == 1)).all()
    if order != 1:
        for e in range(E):   # float32 sums of at most P terms in some order
            rows = dy[own == e].double()
            assert ((db[e].cpu() - rows.sum(0)).abs() <= (len(rows) + 1) * U
                    * rows.abs().sum(0)).all()


@pytest.mark.parametrize("dt,T", [(BF16, 1_100_000), (F32, 550_000)])
def test_swiglu_of_rows_beyond_a_buffer(dt, T):
    """Picked rows of an x beyond 2 GiB through the gated product, also indices
    out of range, with bias, residual and pre-activations."""
    d_in, F, n = 2048, 1032, 300
    g = gen(108)
    x = torch.zeros((T, d_in), dtype=dt, device=DEV)
    tail = normal(g, (n, d_in), dt)
    x[T - n:] = tail.to(DEV)
    W, bias = normal(g, (2, 2 * F, d_in), dt, 0.1), normal(g, (2, 2 * F), dt)
    res = normal(g, (n, F), dt)
    row = torch.arange(T - n, T, dtype=torch.int32, device=DEV)
    row[5], row[250] = T, -3
    tail[5] = tail[250] = 0
    seg = [0, 1, n]
    out = L.grouped_forward(torch.tensor(seg, dtype=torch.int32, device=DEV), x, W.to(DEV),
                            row_index=row, bias=bias.to(DEV), residual=res.to(DEV),
                            act=L.ACT_SWIGLU, save_pre=True)
    ref = O.linear(seg, tail, W, None, bias, res, "swiglu")
    ez = (d_in + 2) * 2 * U * ref["mag"]
    pre = torch.cat([out["pre_a"], out["pre_b"]], 1)
    within(pre, ref["z"], ez + HALF[dt] * (ref["z"].abs() + ez), "pre")
    y, ey = act_bound("swiglu", ref["z"], ez, HALF[dt])
    ey = ey + U * (ref["y"].abs() + ey)
    within(out["y"], ref["y"], ey + HALF[dt] * (ref["y"].abs() + ey), "y")


@pytest.mark.parametrize("name", ["relu", "swiglu"])
@pytest.mark.parametrize("dt,out", [(BF16, BF16), (F32, F32), (BF16, F32)])
def test_epilogue_gradient_at_an_eighth_of_the_capacity(name, dt, out):
    seg, P, F = [0, 0, 70, 71, 300], 2400, 264
    g = gen(109)
    dy, a, b = (normal(g, (P, F), dt, s) for s in (1.0, 2.0, 1.0))
    glu = name == "swiglu"
    n = seg[-1]
    for t in (dy, a, b):
        t[n:] = float("nan")      # what a buffer holds behind the last pair
    bufs = dict(dz=torch.full((P, 2 * F if glu else F), 4.0, dtype=out, device=DEV),
                dbias=torch.empty((len(seg) - 1, 2 * F if glu else F), device=DEV))
    L.act_backward(torch.tensor(seg, dtype=torch.int32, device=DEV), dy.to(DEV), a.to(DEV),
                   b.to(DEV) if glu else None, act=ACTS[name], out=bufs)
    dy, a, b = dy[:n].double(), a[:n].double(), b[:n].double()
    ref = O.act_grad(seg, dy, a, b if glu else None, name)
    e = 16 * U * dy.abs() * (1 + a.abs()) * (1 + a ** 2)   # as in test_act_gradient
    e = torch.cat([e * b.abs(), e], 1) if glu else e * 0
    dz = ref["dz"]
    within(bufs["dz"][:n], dz, e + HALF[out] * (dz.abs() + e) + 1e-38, "dz")
    assert (bufs["dz"][n:] == 4.0).all()
    es = torch.stack([e[seg[i]:seg[i + 1]].sum(0) for i in range(len(seg) - 1)])
    within(bufs["dbias"], ref["dbias"], es + (19 + n // 64 + 1) * U * (ref["mag"] + es) + 1e-38,
           "dbias")


@pytest.mark.parametrize("T", [1, 37, 700])
def test_layer_of_ranks_that_hold_some_experts(T):
    """Gate ids are global and the sort takes local ones: a rank that holds
    experts first .. first + n - 1 sorts ids - first.  Its product runs at the
    capacity of all slots, its combine sums its own slots only."""
    E, K, d, f, ranks = 12, 3, 64, 48, 3
    g = gen(T)
    x, logits = normal(g, (T, d), BF16), normal(g, (T, E), F32)
    Wgu, Wd = normal(g, (E, 2 * f, d), BF16, 0.1), normal(g, (E, d, f), BF16, 0.1)
    gt = L.gate_topk(logits.to(DEV), K)
    ids, w = O.gate(logits, K, "softmax")
    assert torch.equal(gt["ids"].cpu().long(), ids)
    total, n = 0, E // ranks
    for first in range(0, E, n):
        mine = slice(first, first + n)
        rt = L.route_sort(gt["ids"] - first, n, weights=gt["weights"])
        up = L.grouped_forward(rt["seg_offsets"], x.to(DEV), Wgu[mine].contiguous().to(DEV),
                               row_index=rt["row_index"], act=L.ACT_SWIGLU)
        down = L.grouped_forward(rt["seg_offsets"], up["y"], Wd[mine].contiguous().to(DEV))
        y = L.combine(down["y"], rt["pos"], gt["weights"])
        want = torch.zeros((T, d), dtype=torch.float64)
        bound = torch.zeros((T, d), dtype=torch.float64)
        for t in range(T):
            for k in range(K):
                e = int(ids[t, k])
                if not first <= e < first + n:
                    continue
                z = O.linear([0, 1], x[t:t + 1], Wgu[e:e + 1])
                h, eh = act_bound("swiglu", z["z"], (d + 2) * 2 * U * z["mag"], HALF[BF16])
                # h, the pair row and y are rounded to bf16; 1 % covers the
                # roundings' products and the float32 sums of f and K terms
                size = Wd[e].double().abs() @ h[0].abs()
                want[t] += w[t, k] * (Wd[e].double() @ h[0])
                bound[t] += w[t, k] * (Wd[e].double().abs() @ eh[0] + 3.03 * HALF[BF16] * size)
        within(y, want, bound, "y")
        total += int(rt["seg_offsets"][-1])
    assert total == T * K
