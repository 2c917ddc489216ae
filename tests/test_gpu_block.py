"""Operators around the expert products on the GPU against the float64 oracle: 8-bit
rows, weights and their grouped product, the norms around a block, the AdamW step;
edges, refusals of what the host cannot see, graphs, streams, and a run of
them together.

Error bounds: u = 2^-24 (half a float32 step), h = half a step of the output
type (2^-8 for bf16, u for float32), derived where they are used."""
import math

import pytest
import torch

from oracle import block_oracle as B
from oracle import forward_oracle as O
from pruned_expert_backward_amd import lrmoe as L

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from tests.test_gpu_forward import (  # noqa: E402
    ACTS, BF16, DEV, F32, HALF, U, act_bound, gen, normal, within, zipf_seg)

NAN, INF = float("nan"), float("inf")
U8 = torch.uint8


def put(t):
    return None if t is None else t.to(DEV)


def same(got, want, what=""):
    """Equal values, NaN at the same places."""
    got = got.cpu()
    got = got.double() if got.dtype in (L.FP8, BF16, F32) else got
    assert got.shape == want.shape, what
    ok = (got == want) | ((got != got) & (want != want))
    assert bool(ok.all()), f"{what}: {int((~ok).sum())} differ, first at {(~ok).nonzero()[0].tolist()}"


# ------------------------------------------------------------- quantisation

def odd_values(x):
    """Zeros, subnormals, the type's extremes, infinities and NaN among x's blocks."""
    T, D = x.shape
    big = torch.finfo(x.dtype).max
    x = x.clone()
    x[0] = 0
    if T > 5:
        x[1] = 0
        x[1, D - 1] = -1e-38
        x[2] *= 1e30
        x[3, D // 2], x[3, 0] = INF, NAN
        x[4] = NAN
        x[5, 0] = big
        x[5, 1] = -big
    if T > 8:
        x[6] = 448.0
        x[7] = 449.0 if x.dtype == F32 else 450.0
        x[8] = torch.tensor([0.0, -0.0, 1.0, 1.0625, 17.0, 19.0, -0.01953125, 2.0 ** -10] * (D // 8))
    return x


@pytest.mark.parametrize("T,D", [(1, 16), (1, 128), (2, 144), (9, 16), (33, 272), (11, 2048),
                                 (7, 4112), (300, 528)])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_quantize_rows(T, D, dt):
    x = odd_values(normal(gen(T + D), (T, D), dt))
    q, byte = B.quantize_rows(x)
    out = L.quantize_rows(put(x))
    same(out["scale"], byte, "scale")
    same(out["q"], q, "q")


def test_quantize_every_bf16():
    """All bfloat16 values, sixteen to a block."""
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF16).view(-1, 16)
    out = L.quantize_rows(put(x))
    q, byte = B.quantize_rows(x)
    same(out["scale"], byte, "scale")
    same(out["q"], q, "q")


@pytest.mark.parametrize("E,N,K", [(1, 16, 16), (2, 128, 128), (3, 144, 272), (1, 400, 1040),
                                   (2, 8, 144), (1, 520, 48), (4, 256, 512)])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_quantize_weights(E, N, K, dt):
    W = normal(gen(N + K), (E, N, K), dt, 0.02)
    W[0, : N // 2, : K // 2] = 0
    W[E - 1, N - 1, K - 1], W[E - 1, N - 1, 0] = INF, 3.0
    q, byte = B.quantize_weights(W)
    turn = N % 16 == 0
    out = L.quantize_weights(put(W), transpose=turn)
    same(out["scale"], byte, "scale")
    same(out["q"], q, "q")
    if turn:
        qt, bt = B.quantize_weights(W.transpose(1, 2))
        same(out["scale_t"], bt, "scale_t")
        same(out["qt"], qt, "qt")


# ----------------------------------------------------------------- product

def eights(q, byte):
    """Largest code of each run of 8 in a row, at least 2^-6, times its scale."""
    n = q.shape[-1]
    top = torch.nan_to_num(q.double()).abs().unflatten(-1, (n // 8, 8)).amax(-1).clamp_min(2.0 ** -6)
    return top * torch.exp2(byte.double() - 127).repeat_interleave(16, -1)[..., : n // 8]


def product_error(seg, x8, W8, row, mag):
    """Bound of a product's error, given the sum of absolute terms.

    The matrix instruction brings eight products a_i b_i of a run of 8 to one scale: with
    e the largest exponent (of a_i's code plus b_i's; a code below 2^-6 has exponent -6),
    what lies below 2^(e - 13) is cut off.  (Measured: beside 2^16 a second product
    in the run counts in multiples of 2^3, without rounding, of either sign; the sums of
    runs and the accumulator keep 24 bits.)  At most seven terms lose something, the
    one of the largest exponent has 6 bits behind its leading one and loses nothing:
    7 * 2^-13 * max(|a|, 2^-6) max(|b|, 2^-6) for each run.  The float32 sums of the
    runs and of K's steps: a term each, off by one float32 step at most."""
    n = x8["q"].shape[1]
    ax = eights(x8["q"].cpu(), x8["scale"].cpu())
    N = W8["q"].shape[1]
    aw = eights(W8["q"].cpu(), W8["scale"].cpu().repeat_interleave(128, 1)[:, :N])
    cut = torch.zeros_like(mag)
    for e in range(len(seg) - 1):
        at = torch.arange(seg[e], seg[e + 1])
        r = at if row is None else row[at].long()
        ok = (r >= 0) & (r < ax.shape[0])
        v = torch.where(ok[:, None], ax[r.clamp(0, ax.shape[0] - 1)], 0.0)
        cut[at] = v @ aw[e].t()
    return 7 * 2.0 ** -13 * cut + (n + 2) * 2 * U * mag


def check_product(seg, x, W, row, bias, res, name, pre):
    """x and W are values before quantisation; the oracle multiplies what the codes
    stand for."""
    x8, W8 = L.quantize_rows(put(x)), L.quantize_weights(put(W))
    xv = B.row_values(x8["q"].cpu(), x8["scale"].cpu())
    Wv = B.weight_values(W8["q"].cpu(), W8["scale"].cpu())
    ref = O.linear(seg, xv, Wv, row, bias, res, name)
    P, d_out = ref["z"].shape
    F = d_out // 2 if name == "swiglu" else d_out
    out = dict(y=torch.full((P, F), 5.0, dtype=BF16, device=DEV))
    if pre:
        out["pre_a"] = torch.full((P, F), 6.0, dtype=BF16, device=DEV)
        if name == "swiglu":
            out["pre_b"] = torch.full((P, F), 7.0, dtype=BF16, device=DEV)
    L.grouped_forward_quantized(put(torch.tensor(seg, dtype=torch.int32)), x8, W8, put(row),
                                put(bias), put(res), ACTS[name], out=out)
    ez = product_error(seg, x8, W8, row, ref["mag"])
    y, ey = act_bound(name, ref["z"], ez, HALF[BF16])
    if res is not None:
        ey = ey + U * (ref["y"].abs() + ey)
    n = seg[-1]
    within(out["y"][:n], ref["y"][:n], (ey + HALF[BF16] * (ref["y"].abs() + ey))[:n] + 1e-38, "y")
    if pre:
        z = torch.cat([out["pre_a"], out["pre_b"]], 1) if name == "swiglu" else out["pre_a"]
        within(z[:n], ref["z"][:n], (ez + HALF[BF16] * (ref["z"].abs() + ez))[:n] + 1e-38, "pre")
        assert (out["pre_a"][n:] == 6.0).all()
    assert (out["y"][n:] == 5.0).all()     # rows behind the last segment
    return out


def product_inputs(seg, d_in, d_out, seed, spare=0, index=True, name="none"):
    """Rows and weights whose blocks have scales of their own."""
    g = gen(seed)
    E, P = len(seg) - 1, seg[-1] + spare
    T = max(1, P // 2) if index else P
    blocks = (d_in + 127) // 128
    size = torch.exp2(torch.randint(-6, 7, (T, blocks), generator=g).float())
    x = normal(g, (T, d_in), F32) * size.repeat_interleave(128, 1)[:, :d_in]
    wsize = torch.exp2(torch.randint(-3, 4, (E, (d_out + 127) // 128, blocks), generator=g).float())
    wsize = wsize.repeat_interleave(128, 1)[:, :d_out].repeat_interleave(128, 2)[:, :, :d_in]
    W = normal(g, (E, d_out, d_in), F32, 0.1) * wsize
    row = torch.randint(0, T, (P,), generator=g).int() if index else None
    F = d_out // 2 if name == "swiglu" else d_out
    return x.to(BF16), W.to(BF16), row, normal(g, (E, d_out), BF16), normal(g, (P, F), BF16)


SEGS = [[0, 1], [0, 0, 0, 1], [0, 3, 3, 20, 21], [0, 16, 33], [0, 40, 41, 41, 170],
        [0, 127, 255, 384], [0, 300], [0, 5, 600, 1100], [0, 0, 0]]


@pytest.mark.parametrize("seg", SEGS, ids=str)
@pytest.mark.parametrize("d_in,d_out", [(16, 8), (128, 40), (144, 136), (528, 264), (1040, 520)])
def test_product_shapes(seg, d_in, d_out):
    x, W, row, bias, res = product_inputs(seg, d_in, d_out, len(seg) + d_in, spare=3)
    check_product(seg, x, W, row, bias, res, "none", False)


# (segments, columns of y) of every tile shape: by the workgroups that the launch expects
TILES = {
    "few rows": ([0, 1, 3, 20, 21], 136),
    "32x256": ([0, 1, 2] + list(range(10, 508, 8)) + [510, 512], 776),
    "32x64": ([0, 1, 120, 121, 300], 1032),
    "64x64": ([0, 1, 600, 601, 1200], 1032),
    "64x128": ([0, 1, 1250, 1251, 2500], 1032),
    "128 rows": ([0, 1, 2045, 2046, 4090], 1032),
    "256 rows": ([0, 1500, 1501, 1600, 4200], 2056),
    "cut in four": ([0, 4100, 8200], 2304),
    "zipf": (zipf_seg(6000, 12), 1160),
}


def tile_inputs(tile, name, d_in, seed, index=True, spare=0):
    seg, F = TILES[tile]
    F = F // 16 * 8 if name == "swiglu" else F   # as many rows of W
    return (seg,) + product_inputs(seg, d_in, 2 * F if name == "swiglu" else F, seed, spare,
                                   index, name)


@pytest.mark.parametrize("tile", list(TILES))
@pytest.mark.parametrize("name,d_in", [("none", 16), ("swiglu", 144), ("none", 656)])
@pytest.mark.parametrize("index", [True, False])
def test_product_tiles(tile, name, d_in, index):
    seg, x, W, row, bias, _ = tile_inputs(tile, name, d_in, 5 + d_in, index)
    check_product(seg, x, W, row, bias, None, name, name == "swiglu")


@pytest.mark.parametrize("tile", ["few rows", "32x256", "32x64", "64x128", "256 rows"])
@pytest.mark.parametrize("d_in", [4096, 4112, 8720])
def test_product_long_rows(tile, d_in):
    """More K steps than the scales in LDS at a time, and a last group of every length."""
    seg, F = TILES[tile]
    seg = [s // 4 for s in seg] if seg[-1] > 2000 else seg
    x, W, row, bias, res = product_inputs(seg, d_in, 264, 9)
    check_product(seg, x, W, row, None, res, "none", False)


@pytest.mark.parametrize("name", list(ACTS))
@pytest.mark.parametrize("tile", ["few rows", "64x64", "256 rows"])
@pytest.mark.parametrize("bias,residual,pre", [(1, 1, 1), (0, 1, 0), (1, 0, 1), (0, 0, 0)])
def test_product_epilogues(name, tile, bias, residual, pre):
    seg, x, W, row, b, r = tile_inputs(tile, name, 272, 31, spare=2)
    check_product(seg, x, W, row, b if bias else None, r if residual else None, name, bool(pre))


@pytest.mark.parametrize("tile", ["few rows", "32x64", "64x128", "256 rows"])
def test_product_rows_out_of_range_and_nan(tile):
    """Rows by index that are not there are zeros; NaN in a row or a weight reaches
    exactly the results that read it."""
    seg, x, W, row, bias, _ = tile_inputs(tile, "none", 272, 8)
    row[::7] = -1
    row[3::11] = x.shape[0]
    check_product(seg, x, W, row, bias, None, "none", False)
    x[0, 5], W[0, 3, 200] = NAN, INF
    P = seg[-1]
    x8, W8 = L.quantize_rows(put(x)), L.quantize_weights(put(W))
    y = L.grouped_forward_quantized(put(torch.tensor(seg, dtype=torch.int32)), x8, W8,
                                    put(row))["y"].cpu()
    want = (row == 0)[:, None].repeat(1, W.shape[1])
    want[: seg[1], 3] = True       # an index that is not there reads zeros: 0 * NaN
    assert torch.equal(torch.isnan(y[:P]), want)


@pytest.mark.parametrize("tile", ["few rows", "64x64", "256 rows"])
@pytest.mark.parametrize("order", ["back", "past", "negative"])
def test_product_offsets_out_of_order(tile, order):
    """Offsets that do not ascend or leave the rows: every access stays inside; segments
    that are in order are right."""
    seg, x, W, row, bias, _ = tile_inputs(tile, "none", 144, 3)
    E, P = len(seg) - 1, seg[-1]
    bad = list(seg)
    if order == "back":
        bad[E // 2] = 0
    elif order == "past":
        bad[-1] = P + 1000
    else:
        bad[0] = -5
    x8, W8 = L.quantize_rows(put(x)), L.quantize_weights(put(W))
    y = torch.full((P + 8, W.shape[1]), 5.0, dtype=BF16, device=DEV)
    L.grouped_forward_quantized(put(torch.tensor(bad, dtype=torch.int32)), x8, W8, put(row),
                                out=dict(y=y[:P]))
    assert bool((y[P:] == 5.0).all())
    if order != "back":
        ref = L.grouped_forward_quantized(put(torch.tensor(seg, dtype=torch.int32)), x8, W8,
                                          put(row))["y"]
        assert torch.equal(ref, y[:P])


def test_product_scales_at_their_ends():
    """Blocks of the largest and smallest scales: products of 2^(e + f) that float32
    holds, zero blocks beside them."""
    g = gen(4)
    x, W = normal(g, (5, 384), F32), normal(g, (1, 24, 384), F32)
    x[:, :128] *= 2.0 ** 60
    W[:, :, :128] *= 2.0 ** -60
    x[:, 128:256] *= 2.0 ** -110
    W[:, :, 256:] = 0
    x[4] = 0
    check_product([0, 5], x, W, None, None, None, "none", False)


def test_product_is_the_same_in_any_company():
    """A row's result does not depend on the rows beside it, within a tile shape."""
    x, W, _, _, _ = product_inputs([0, 4096], 1040, 520, 12, index=False)
    x8, W8 = L.quantize_rows(put(x)), L.quantize_weights(put(W))
    seg = put(torch.tensor([0, 4096], dtype=torch.int32))
    y = L.grouped_forward_quantized(seg, x8, W8)["y"]
    flip = torch.arange(4095, -1, -1, dtype=torch.int32, device=DEV)
    z = L.grouped_forward_quantized(seg, x8, W8, row_index=flip)["y"]
    assert torch.equal(y, z.flip(0))


def test_product_input_gradient():
    """dx through the transposed weights against the formula and against
    differences of the product (linear in x: exact but for roundings)."""
    seg, d_in, d_out = [0, 70, 71, 200], 272, 144
    x, W, _, _, _ = product_inputs(seg, d_in, d_out, 21, index=False)
    dy = normal(gen(2), (200, d_out), BF16)
    W8 = L.quantize_weights(put(W), transpose=True)
    d8 = L.quantize_rows(put(dy))
    off = put(torch.tensor(seg, dtype=torch.int32))
    dx = L.grouped_forward_quantized(off, d8, L.transposed_weights(W8))["y"]
    Wv = B.weight_values(W8["q"].cpu(), W8["scale"].cpu())
    dv = B.row_values(d8["q"].cpu(), d8["scale"].cpu())
    ref = O.linear(seg, dv, Wv.transpose(1, 2).contiguous())
    Wt8 = L.transposed_weights(W8)
    within(dx, ref["z"], product_error(seg, d8, Wt8, None, ref["mag"]) + HALF[BF16] * ref["z"].abs() * 1.01
           + 1e-38, "dx")
    u, k = 130, 200
    e = 2
    y = lambda v: float((Wv[e] @ v * dv[u]).sum())   # noqa: E731
    one = torch.zeros(d_in, dtype=torch.float64)
    one[k] = 1.0
    base = x[u].double()
    assert abs(y(base + one) - y(base) - float(dx[u, k])) <= 2 ** -7 * float(ref["mag"][u, k])


def test_product_beyond_a_buffer():
    """x beyond 2 GiB behind a row index, and rows' addresses beyond 32 bits."""
    T, D = 2 ** 31 // 2048 + 3, 2048
    q = torch.zeros(T, D, dtype=U8, device=DEV)
    s = torch.full((T, 16), 127, dtype=U8, device=DEV)
    pick = [0, T - 1, T - 2, 5, T // 2]
    x, W, _, _, _ = product_inputs([0, 5], D, 40, 3, index=False)
    x8, W8 = L.quantize_rows(put(x)), L.quantize_weights(put(W))
    seg = put(torch.tensor([0, 5], dtype=torch.int32))
    want = L.grouped_forward_quantized(seg, x8, W8)["y"]
    for i, t in enumerate(pick):
        q[t], s[t] = x8["q"].view(U8)[i], x8["scale"][i]
    big = dict(q=q.view(L.FP8), scale=s)
    row = put(torch.tensor(pick, dtype=torch.int32))
    assert torch.equal(L.grouped_forward_quantized(seg, big, W8, row_index=row)["y"], want)
    # as many rows as make tiles of them
    P, W = 4096, product_inputs([0, 1], D, 1032, 4)[1]
    W8 = L.quantize_weights(put(W))
    at = torch.tensor(pick, dtype=torch.int32)[torch.arange(P) % 5]
    seg = put(torch.tensor([0, P], dtype=torch.int32))
    y = L.grouped_forward_quantized(seg, big, W8, row_index=put(at))["y"]
    ref = L.grouped_forward_quantized(seg, x8, W8, row_index=put((torch.arange(P) % 5).int()))["y"]
    # two tile shapes: float32 sums in the same order of K steps, so equal but for a
    # start of the loop elsewhere
    mag = O.linear([0, 5], B.row_values(x8["q"].cpu(), x8["scale"].cpu()),
                   B.weight_values(W8["q"].cpu(), W8["scale"].cpu()))["mag"]
    e = product_error([0, 5], x8, W8, None, mag)[torch.arange(P) % 5]
    got, z = y.cpu().double(), ref.cpu().double()
    assert bool(((got - z).abs() <= 2 * e + 2 ** -7 * z.abs()).all())


@pytest.mark.parametrize("tile", list(TILES))
@pytest.mark.parametrize("name", ["none", "swiglu"])
def test_product_at_an_eighth_of_the_capacity(tile, name):
    """As many pair rows again seven times, behind the last segment: left as they were."""
    seg, F = TILES[tile]
    seg, F = [s // 8 for s in seg], F // 16 * 8 if name == "swiglu" else F
    x, W, row, bias, _ = product_inputs(seg, 272, 2 * F if name == "swiglu" else F, 6,
                                        spare=TILES[tile][0][-1] - seg[-1], name=name)
    check_product(seg, x, W, row, bias, None, name, False)


def test_product_many_experts():
    """256 experts, most of them without rows, one with most."""
    seg = [0] * 40 + [3] * 100 + [900] * 50 + [901 + i for i in range(67)]
    x, W, row, bias, _ = product_inputs(seg, 144, 72, 14)
    check_product(seg, x, W, row, bias, None, "silu", True)


def test_quantize_beyond_32_bits():
    """Rows and weights whose elements pass 2^32: the last ones as if they were alone."""
    D = 4096
    T = 2 ** 32 // D + 70
    x = torch.zeros(T, D, dtype=BF16, device=DEV)
    tail = normal(gen(3), (70, D), BF16)
    x[-70:] = put(tail)
    out, ref = L.quantize_rows(x), L.quantize_rows(put(tail))
    assert torch.equal(out["q"][-70:].view(U8), ref["q"].view(U8))
    assert torch.equal(out["scale"][-70:], ref["scale"])
    assert int((out["scale"][:-70] != 127).sum()) == 0
    del out
    W = x[: T // 128 * 128].view(1, -1, D)     # one expert's, transposed as well
    W8 = L.quantize_weights(W, transpose=True)
    end = W[0, -128:]
    want = L.quantize_weights(end[None].contiguous(), transpose=True)
    assert torch.equal(W8["q"][0, -128:].view(U8), want["q"][0].view(U8))
    assert torch.equal(W8["scale"][0, -1], want["scale"][0, 0])
    assert torch.equal(W8["qt"][0, :, -128:].contiguous().view(U8), want["qt"][0].view(U8))
    last = W.shape[1] // 128 - 1
    assert torch.equal(W8["scale_t"][0, :, last], want["scale_t"][0, :, 0])


def test_results_into_given_buffers():
    """out's buffers are the results, and nothing beside them is written."""
    x = put(normal(gen(5), (33, 272), BF16))
    ref = L.quantize_rows(x)
    q, s = torch.full((35, 272), 9, dtype=U8, device=DEV), torch.full((35, 4), 9, dtype=U8, device=DEV)
    out = dict(q=q[1:34].view(L.FP8), scale=s[1:34])
    with pytest.raises(L.LrmoeError):          # a row of scales is no 16-byte border
        L.quantize_rows(x, out=out)
    q, s = torch.full((48, 272), 9, dtype=U8, device=DEV), torch.full((48, 4), 9, dtype=U8, device=DEV)
    out = dict(q=q[4:37].view(L.FP8), scale=s[4:37])
    assert L.quantize_rows(x, out=out) is out
    assert torch.equal(q[4:37], ref["q"].view(U8)) and torch.equal(s[4:37], ref["scale"])
    assert bool((q[:4] == 9).all() and (q[37:] == 9).all() and (s[:4] == 9).all()
                and (s[37:] == 9).all())


# ------------------------------------------------------------------- norms

NORMS = [(1, 8), (3, 64), (5, 520), (33, 512), (130, 1032), (9, 2048), (6, 2056), (1100, 136),
         (4, 8192), (3, 8200), (2, 16384)]
KINDS = [dict(y=1, w=1, wb=1, gate="channel"), dict(y=1, w=1, wb=1, gate="token"),
         dict(y=1, w=1, wb=0, gate=None), dict(y=1, w=0, wb=1, gate=None),
         dict(y=1, w=0, wb=0, gate="token"), dict(y=1, w=1, wb=0, gate="channel"),
         dict(y=0, w=1, wb=0, gate=None)]
K_SUM = 60   # float32 sums over a row: at most 32 in a lane's registers (16 values, two of
#              them squared), 6 in a wave, 16 over waves, and the mean, root and reciprocal


def norm_inputs(T, D, dt, kind, seed):
    g = gen(seed)
    v = dict(x=normal(g, (T, D), dt, 2.0))
    if kind["y"]:
        v["y"] = normal(g, (T, D), dt)
    if kind["w"]:
        v["weight"] = (1 + normal(g, (D,), F32, 0.2)).to(dt)
    if kind["wb"]:
        v["branch_weight"] = (1 + normal(g, (D,), F32, 0.2)).to(dt)
    if kind["gate"] == "channel":
        v["gate"] = normal(g, (D,), dt)
    elif kind["gate"] == "token":
        v["gate"] = normal(g, (T, 1), F32)
    return v


def rms(v):
    return v.square().mean(1, keepdim=True).sqrt()


@pytest.mark.parametrize("T,D", NORMS)
@pytest.mark.parametrize("kind", KINDS, ids=lambda k: "".join(f"{a}{b}" for a, b in k.items()))
@pytest.mark.parametrize("dt", [BF16, F32])
def test_norm(T, D, kind, dt):
    v = norm_inputs(T, D, dt, kind, T + D)
    c = 0.75 if kind["y"] else 1.0
    s, h = B.residual_norm(**v, scale=c, eps=1e-5)
    out = L.residual_norm(**{k: put(t) for k, t in v.items()}, scale=c, eps=1e-5)
    assert set(out) == {k for k, on in (("s", kind["y"]), ("h", kind["w"])) if on}
    # s: the branch is good to (K_SUM + 4) u of itself, the sum rounds twice more
    es = torch.zeros_like(s)
    if kind["y"]:
        es = U * (2 * (c * v["x"].double()).abs() + (K_SUM + 6) * (s - c * v["x"].double()).abs()
                  + s.abs())
        within(out["s"], s, es + HALF[dt] * (s.abs() + es) + 1e-38, "s")
    if kind["w"]:
        # h: s's error, that of the root (s's errors against its size) and the products
        eh = h.abs() * ((K_SUM + 4) * U + rms(es) / rms(s)) + \
            es * (h / s).abs().nan_to_num(0)
        within(out["h"], h, eh + HALF[dt] * (h.abs() + eh) + 1e-38, "h")


def check_norm_grad(v, ds, dh, c, eps, dt):
    """Every output against its formula; a float32 computation's error is within K u
    of the sum of absolute terms that the oracle gives: K_SUM for each of the two
    means on the way and a dozen products, T more for sums over rows."""
    T, D = v["x"].shape
    rest = {k: t for k, t in v.items() if k != "x"}
    s = B.residual_norm(**v, scale=c, eps=eps)[0].to(dt) if "y" in v else v["x"]
    ref = B.residual_norm_grad(s, ds, dh, scale=c, eps=eps, **rest)
    out = L.residual_norm_backward(put(s), ds=put(ds), dh=put(dh), scale=c, eps=eps,
                                   **{k: put(t) for k, t in rest.items()})
    assert set(out) == {k for k in ref if not k.endswith("_mag")}
    for k, got in out.items():
        rows = T if k in ("dweight", "dbranch_weight") or (k == "dgate" and got.dim() == 1) else 0
        half = HALF[dt] if k in ("dx", "dy") else U
        e = (2 * K_SUM + 12 + rows) * U * ref[k + "_mag"]
        within(got, ref[k], e + half * (ref[k].abs() + e) + 1e-38, k)
    return out


@pytest.mark.parametrize("T,D", NORMS)
@pytest.mark.parametrize("kind", KINDS, ids=lambda k: "".join(f"{a}{b}" for a, b in k.items()))
@pytest.mark.parametrize("dt", [BF16, F32])
def test_norm_gradient(T, D, kind, dt):
    v = norm_inputs(T, D, dt, kind, T + D + 1)
    g = gen(7)
    ds = normal(g, (T, D), dt) if kind["y"] or T % 2 else None
    dh = normal(g, (T, D), dt) if kind["w"] else None
    check_norm_grad(v, ds, dh, 0.75 if kind["y"] else 1.0, 1e-5, dt)


def test_norm_gradient_many_rows():
    """More rows than groups of waves, and nothing arriving at s but through h."""
    kind = dict(y=1, w=1, wb=1, gate="channel")
    for T, D in ((5000, 64), (2500, 1040)):
        v = norm_inputs(T, D, BF16, kind, 3)
        check_norm_grad(v, None, normal(gen(1), (T, D), BF16), 1.0, 1e-6, BF16)


def test_norm_gradient_against_differences():
    """float32 results against differences of the float64 loss at the stored s."""
    T, D, c, eps = 6, 48, 0.5, 1e-5
    v = norm_inputs(T, D, F32, dict(y=1, w=1, wb=1, gate="token"), 11)
    g = gen(12)
    ds, dh = normal(g, (T, D), F32), normal(g, (T, D), F32)

    def loss(**over):
        a = {k: t.double() for k, t in {**v, **over}.items()}
        s, h = B.residual_norm(**a, scale=c, eps=eps)
        return float((s * ds).sum() + (h * dh).sum())
    s = B.residual_norm(**v, scale=c, eps=eps)[0].float()
    rest = {k: put(t) for k, t in v.items() if k != "x"}
    out = L.residual_norm_backward(put(s), ds=put(ds), dh=put(dh), scale=c, eps=eps, **rest)
    for name, at in (("x", (2, 5)), ("y", (4, 40)), ("weight", (7,)), ("branch_weight", (47,)),
                     ("gate", (3, 0))):
        d = torch.zeros(v[name].shape, dtype=torch.float64)
        d[at] = 1e-4
        diff = (loss(**{name: v[name].double() + d}) - loss(**{name: v[name].double() - d})) / 2e-4
        # float32 and the rounded s: 2^-20 of the terms; central differences 1e-8 of the third slope
        assert abs(float(out["d" + name][at]) - diff) <= 2e-4 * (1 + abs(diff)), name


def test_norm_zero_rows_and_extremes():
    """Rows of zeros are 0 through eps; an infinity or NaN stays in its row."""
    T, D = 6, 136
    kind = dict(y=1, w=1, wb=1, gate="channel")
    v = norm_inputs(T, D, F32, kind, 5)
    v["x"][0], v["y"][0] = 0, 0
    v["y"][2, 7] = INF
    v["x"][3, 9] = NAN
    out = L.residual_norm(**{k: put(t) for k, t in v.items()})
    s, h = out["s"].cpu(), out["h"].cpu()
    assert bool((s[0] == 0).all()) and bool((h[0] == 0).all())
    ok = [0, 1, 4, 5]
    assert bool(torch.isfinite(s[ok]).all()) and bool(torch.isfinite(h[ok]).all())
    assert bool(torch.isnan(h[2]).any()) and bool(torch.isnan(h[3]).all())
    g = L.residual_norm_backward(put(torch.zeros(T, D)), ds=put(v["x"] * 0 + 1), dh=put(v["x"] * 0 + 1),
                                 y=put(torch.zeros(T, D)), weight=put(v["weight"]),
                                 branch_weight=put(v["branch_weight"]), gate=put(v["gate"]))
    assert bool(torch.isfinite(g["dy"][ok]).all())


def test_norm_gradient_of_chosen_parts():
    """A given out says which sums over rows are computed; the others need no workspace."""
    T, D = 20, 264
    v = {k: put(t) for k, t in norm_inputs(T, D, BF16, KINDS[0], 2).items()}
    s = L.residual_norm(**v)["s"]
    rest = {k: t for k, t in v.items() if k != "x"}
    ds = put(normal(gen(3), (T, D), BF16))
    full = L.residual_norm_backward(s, ds=ds, dh=ds, **rest)
    new = lambda *sh, dt=F32: torch.zeros(sh, dtype=dt, device=DEV)   # noqa: E731
    for names in ((), ("dweight",), ("dgate",), ("dbranch_weight", "dgate")):
        out = dict(dx=new(T, D, dt=BF16), dy=new(T, D, dt=BF16), **{n: new(D) for n in names})
        L.residual_norm_backward(s, ds=ds, dh=ds, out=out, **rest)
        for k, t in out.items():
            assert torch.equal(t, full[k]), k


# ------------------------------------------------------------------- AdamW

def state_of(m, v, bits):
    """A state that holds m and v (8-bit: their nearest codes)."""
    if bits == 32:
        return dict(m=put(m), v=put(v))
    out = {}
    for name, x in (("m", m), ("root", v.sqrt())):
        s, byte = B.blocks_of(x)
        out[name] = put((B.e4m3(x.double() / s)).float().to(L.FP8))
        out[name + "_scale"] = put(byte)
    return out


def values_of(st, n):
    """(m, v) that a state stands for, float64."""
    if "v" in st:
        return st["m"].cpu().double(), st["v"].cpu().double()
    val = [B.row_values(st[k].cpu().view(1, -1), st[k + "_scale"].cpu().view(1, -1))[0]
           for k in ("m", "root")]
    return val[0], val[1] ** 2


def check_codes(q, byte, x, ex, u, root, what):
    """Codes of a block's values x (float64, known to ex): the scale byte, and one of
    the two neighbours, the upper one where the fraction passes 1 - u.  Where x is too near
    a border to tell, either neighbour will do."""
    s, want = B.blocks_of(x)
    top = torch.nn.functional.pad(x.abs(), (0, -x.numel() % 128)).view(-1, 128).amax(1)
    sure = (top / (448 * torch.exp2(want.double() - 127)) < 1 - 1e-6) & \
        (top / (224 * torch.exp2(want.double() - 127)) > 1 + 1e-6) | (top == 0)
    assert torch.equal(byte.cpu()[sure], want[sure]), what
    assert bool(sure.all()), f"{what}: inputs at a scale's border"
    a = (x / s).abs()
    step = B.e4m3_step(a)
    t = a / step
    lo, up = torch.floor(t), t - torch.floor(t) + u >= 1
    code = (lo + up) * step
    if root:
        code = torch.where((x > 0) & (code == 0), 2.0 ** -9, code)
    got = q.cpu().double()
    near = ((t + u - torch.round(t + u)).abs() <= ex / s / step + 2.0 ** -18)
    right = (got.abs() == code) | near & ((got.abs() - a).abs() <= step * (1 + 1e-6))
    assert bool(right.all()), f"{what}: {int((~right).sum())} codes"
    assert bool((near.double().mean() < 0.01)), what
    sign = torch.sign(got) * torch.sign(x)
    assert bool((sign >= 0).all()), what


SIZES = [1, 7, 8, 127, 128, 129, 2047, 2048, 2049, 5000, 8192, 20011]


@pytest.mark.parametrize("pdt", [F32, BF16])
@pytest.mark.parametrize("gdt", [F32, BF16])
@pytest.mark.parametrize("bits", [32, 8])
def test_adamw(pdt, gdt, bits):
    """Tensors of every kind of length in one call, each against the formula."""
    g = gen(17)
    step, lr, betas, eps, wd, gs, seed = 37, 1e-2, (0.9, 0.95), 1e-8, 0.1, 0.8125, 91
    ps = [normal(g, (n,), pdt, 0.5) for n in SIZES]
    gr = [normal(g, (n,), F32, 0.01).to(gdt) for n in SIZES]
    ms = [normal(g, (n,), F32, 0.003) for n in SIZES]
    vs = [(normal(g, (n,), F32, 0.01)) ** 2 for n in SIZES]
    gr[4][:] = 0                       # an expert without pairs
    ms[5][:], vs[5][:] = 0, 0          # a first step
    gr[6][:], ms[6][:], vs[6][:] = 0, 0, 0
    sts = [state_of(m, v, bits) for m, v in zip(ms, vs)]
    old = [values_of(st, n) for st, n in zip(sts, SIZES)]
    dp = [put(p) for p in ps]
    copies = [torch.zeros(n, dtype=BF16, device=DEV) if pdt == F32 and n % 3 else None
              for n in SIZES]
    L.adamw_step(dp, [put(x) for x in gr], sts, step, lr, betas, eps, wd, copies=copies,
                 grad_scale=torch.tensor([gs], device=DEV), seed=seed)
    for k, n in enumerate(SIZES):
        p, m, v = B.adamw(ps[k], gr[k], *old[k], step, lr, betas, eps, wd, gs)
        # two products, a sum, beta's own rounding: 4 u of the terms; v three more
        am = betas[0] * old[k][0].abs() + (1 - betas[0]) * gs * gr[k].double().abs()
        em, ev = 4 * U * am + 1e-44, 8 * U * v + 1e-44
        # the update: m's error, sqrt (half of v's error and its own), reciprocal 2 u, products
        upd = lr / (1 - betas[0] ** step) / (torch.sqrt(v / (1 - betas[1] ** step)) + eps)
        ep = upd * (em + 16 * U * m.abs()) + 4 * U * ps[k].double().abs()
        dice = B.dice(seed, step, k, n)
        if pdt == F32:
            within(dp[k], p, ep + U * p.abs(), f"p {n}")
            if copies[k] is not None:
                same(copies[k], dp[k].cpu().to(BF16).double(), "copy")
        else:
            _, e = torch.frexp(p)
            bf = torch.exp2((e - 8).double())
            t = p.abs() / bf
            u = B.chance(B.second_dice(dice))
            want = (torch.floor(t) + ((t - torch.floor(t) + u) >= 1)) * bf
            got = dp[k].cpu().double()
            near = (t + u - torch.round(t + u)).abs() <= ep / bf + 2.0 ** -15
            ok = (got.abs() == want) | near & ((got.abs() - p.abs()).abs() <= bf * 1.001)
            assert bool(ok.all()), f"p {n}"
            assert float(near.double().mean()) < 0.01 or n < 1000
        if bits == 32:
            within(sts[k]["m"], m, em, f"m {n}")
            within(sts[k]["v"], v, ev, f"v {n}")
        else:
            root = torch.sqrt(v)
            check_codes(sts[k]["m"], sts[k]["m_scale"], m, em, B.chance(dice >> 16), False, f"m {n}")
            check_codes(sts[k]["root"], sts[k]["root_scale"], root, 8 * U * root,
                        B.chance(dice & 0xFFFF), True, f"root {n}")


def test_adamw_many_tensors_of_all_kinds():
    """More tensors than a launch takes, kinds mixed, empty ones among them: each as if
    it were alone at its place in the list."""
    g = gen(3)
    n = 130
    sizes = [0 if k % 13 == 5 else 1 + 37 * k % 4001 for k in range(n)]
    make = []
    for k, size in enumerate(sizes):
        pdt, gdt, bits = (F32, BF16)[k % 2], (F32, BF16)[k // 2 % 2], (32, 8)[k // 4 % 2]
        make.append((normal(g, (size,), pdt), normal(g, (size,), gdt, 0.1), bits))
    runs = []
    for alone in (False, True):
        p, gr = [put(a) for a, _, _ in make], [put(b) for _, b, _ in make]
        st = [L.adamw_state(a, bits) for a, (_, _, bits) in zip(p, make)]
        for t in (1, 2):
            if alone:
                blank = torch.zeros(0, device=DEV)
                for k in range(n):   # at place k, behind empty tensors
                    L.adamw_step([blank] * k + [p[k]], [blank] * k + [gr[k]],
                                 [L.adamw_state(blank)] * k + [st[k]], t, 1e-2, seed=5)
            else:
                L.adamw_step(p, gr, st, t, 1e-2, seed=5)
        runs.append((p, st))
    for k in range(n):
        assert torch.equal(runs[0][0][k], runs[1][0][k]), k
        for name in runs[0][1][k]:
            a, b = runs[0][1][k][name], runs[1][1][k][name]
            assert torch.equal(a.view(U8) if a.dtype == L.FP8 else a,
                               b.view(U8) if b.dtype == L.FP8 else b), (k, name)


def test_adamw_rounding_is_even_handed():
    """The mean of many stochastic roundings is the value: the error of the mean of n
    roundings within a step has a standard deviation of at most half a step / sqrt(n);
    six of those are allowed."""
    n, step = 128 * 512, 1
    p = torch.full((n,), 1.0, dtype=BF16, device=DEV)
    gr = torch.zeros(n, device=DEV)
    gr.view(-1, 128)[:] = torch.linspace(0.011, 1.0, 128, device=DEV)
    st = L.adamw_state(p, bits=8)
    L.adamw_step([p], [gr], [st], step, 1e-3, (0.9, 0.96), 1e-8, 0.0, seed=123)
    m, v = values_of(st, n)
    want = 0.1 * gr.cpu().double().view(-1, 128)[0]
    gap = B.e4m3_step(want / torch.exp2(st["m_scale"].cpu().double()[0] - 127)) * \
        torch.exp2(st["m_scale"].cpu().double()[0] - 127)
    off = (m.view(-1, 128).mean(0) - want).abs()
    assert bool((off <= 6 * gap / 2 / math.sqrt(512) + 1e-6 * want).all())
    root = 0.2 * gr.cpu().double().view(-1, 128)[0]
    s = torch.exp2(st["root_scale"].cpu().double()[0] - 127)
    off = (v.sqrt().view(-1, 128).mean(0) - root).abs()
    assert bool((off <= 6 * B.e4m3_step(root / s) * s / 2 / math.sqrt(512) + 1e-6 * root).all())
    # p = 1 - 1e-3 (the first step's update is lr g / |g|): bf16 steps of 2^-8 below 1
    off = abs(float(p.double().mean()) - (1 - 1e-3))
    assert off <= 6 * 2.0 ** -9 / math.sqrt(n) + 1e-6


def test_adamw_second_moment_stays_above_zero():
    """Elements far below their block's largest keep a non-zero root, so that their
    first moment is never divided by eps alone."""
    n = 256
    p, gr = torch.zeros(n, device=DEV), torch.full((n,), 1e-9, device=DEV)
    gr[::128] = 1.0
    st = L.adamw_state(p, bits=8)
    for t in range(1, 30):
        L.adamw_step([p], [gr], [st], t, 1e-3, weight_decay=0.0, seed=t)
    root = st["root"].cpu().float()
    assert bool((root > 0).all())
    assert float(p.abs().max()) <= 29 * 1.3e-3   # m / root is about 1 where both are exact


def test_adamw_not_finite():
    """NaN and infinity stay with their elements in either kind of state."""
    for bits in (32, 8):
        n = 300
        p, gr = torch.ones(n, device=DEV), torch.full((n,), 0.5, device=DEV)
        gr[3], gr[200] = NAN, INF
        st = L.adamw_state(p, bits)
        L.adamw_step([p], [gr], [st], 1, 1e-2)
        m, v = values_of(st, n)
        bad = torch.zeros(n, dtype=torch.bool)
        bad[3] = bad[200] = True
        assert torch.equal(~torch.isfinite(m), bad) and torch.equal(~torch.isfinite(v), bad)
        assert bool(torch.isfinite(p.cpu()[~bad]).all()) and bool(torch.isnan(p.cpu()[3]))


def test_adamw_skip_and_scalars_on_the_device():
    g = gen(8)
    p0, gr = put(normal(g, (1000,), F32)), put(normal(g, (1000,), F32))
    one = lambda v, dt: torch.tensor([v], dtype=dt, device=DEV)   # noqa: E731
    for bits in (32, 8):
        host, dev, kept = (dict(p=p0.clone(), st=L.adamw_state(p0, bits)) for _ in range(3))
        for t in (1, 2, 3):
            lr = float(torch.tensor(1e-2 / t))
            L.adamw_step([host["p"]], [gr], [host["st"]], t, lr, seed=4)
            L.adamw_step([dev["p"]], [gr], [dev["st"]], one(t, torch.int64), one(lr, F32), seed=4,
                         skip=one(0.0, F32))
            L.adamw_step([kept["p"]], [gr], [kept["st"]], t, lr, seed=4,
                         skip=one((1.0, NAN, -2.0)[t - 1], F32))
        assert torch.equal(host["p"], dev["p"]) and torch.equal(kept["p"], p0)
        for k, t in host["st"].items():
            u = (lambda x: x.view(U8) if x.dtype == L.FP8 else x)
            assert torch.equal(u(t), u(dev["st"][k])), k
            assert torch.equal(u(kept["st"][k]), u(L.adamw_state(p0, bits)[k])), k


def test_adamw_beyond_32_bits():
    """Elements behind 2^32 of one tensor (bf16 parameters and gradients, 8-bit states)."""
    n = 2 ** 32 + 3000
    p = torch.zeros(n, dtype=BF16, device=DEV)
    gr = torch.zeros(n, dtype=BF16, device=DEV)
    st = L.adamw_state(p, bits=8)
    tail = 3000
    g = normal(gen(1), (tail,), BF16)
    gr[-tail:] = put(g)
    L.adamw_step([p], [gr], [st], 1, 1e-2, (0.9, 0.95), 1e-8, 0.0, seed=7)
    _, m, v = B.adamw(torch.zeros(tail), g, torch.zeros(tail), torch.zeros(tail), 1, 1e-2,
                      (0.9, 0.95), 1e-8, 0.0)
    assert int((p[:1000] != 0).sum()) == 0 and int((st["m"][:1000].view(U8) & 127).sum()) == 0
    # the tail starts at a block's border (2^32 is one); the hash takes the index mod 2^32
    dice = B.dice(7, 1, 0, tail)
    check_codes(st["m"][-tail:], st["m_scale"][2 ** 25:], m, 4 * U * m.abs(), B.chance(dice >> 16),
                False, "m")
    check_codes(st["root"][-tail:], st["root_scale"][2 ** 25:], torch.sqrt(v), 8 * U * torch.sqrt(v),
                B.chance(dice & 0xFFFF), True, "root")


# -------------------------------------------------------- graphs, streams, empties

def block_calls(t):
    """One pass through every operator on the tensors of t."""
    n = L.residual_norm(t["x"], y=t["y"], weight=t["w"], branch_weight=t["w"], gate=t["gate"])
    x8 = L.quantize_rows(n["h"])
    W8 = L.quantize_weights(t["W"], transpose=True)
    up = L.grouped_forward_quantized(t["seg"], x8, W8, act=L.ACT_SWIGLU, save_pre=True)
    dz = L.act_backward(t["seg"], t["dy"], up["pre_a"], up["pre_b"], act=L.ACT_SWIGLU,
                        dbias=False)["dz"]
    dh = L.grouped_forward_quantized(t["seg"], L.quantize_rows(dz), L.transposed_weights(W8))["y"]
    d = L.residual_norm_backward(n["s"], ds=t["x"], dh=dh, y=t["y"], weight=t["w"],
                                 branch_weight=t["w"], gate=t["gate"])
    return dict(s=n["s"], h=n["h"], y=up["y"], dh=dh, **d)


def block_tensors(seed, T=200, D=256, f=64):
    g = gen(seed)
    return dict(x=put(normal(g, (T, D), BF16)), y=put(normal(g, (T, D), BF16)),
                w=put((1 + normal(g, (D,), F32, 0.1)).to(BF16)), gate=put(normal(g, (D,), BF16)),
                W=put(normal(g, (3, 2 * f, D), BF16, 0.1)), dy=put(normal(g, (T, f), BF16)),
                seg=put(torch.tensor([0, 50, 51, T], dtype=torch.int32)))


def test_captured_and_replayed():
    """Everything in one graph, the optimizer's step with its counter on the device among
    it; replays with new inputs against eager calls."""
    t = block_tensors(1)
    p = torch.randn(3000, device=DEV)
    st, step = L.adamw_state(p, bits=8), torch.zeros(1, dtype=torch.int64, device=DEV)
    grad = torch.zeros(3000, device=DEV)
    q, st2 = p.clone(), L.adamw_state(p, bits=8)

    def all_of_it():
        out = block_calls(t)
        step.add_(1)
        L.adamw_step([p], [grad], [st], step, 1e-2, seed=9)
        return out
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block_calls(t)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = all_of_it()
    for r in range(1, 5):
        new = block_tensors(10 + r)
        for k in t:
            if k != "seg":
                t[k].copy_(new[k])
        grad.copy_(torch.linspace(-1, 1, 3000, device=DEV) * r)
        graph.replay()
        torch.cuda.synchronize()
        want = block_calls(t)
        for k in want:
            assert torch.equal(out[k], want[k]), (r, k)
        L.adamw_step([q], [grad], [st2], r, 1e-2, seed=9)
        assert torch.equal(p, q) and torch.equal(st["m"].view(U8), st2["m"].view(U8)), r


def test_two_streams_at_once_and_again():
    a, b = block_tensors(2), block_tensors(3, T=311)
    want = [block_calls(a), block_calls(b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for s, t in zip(streams, (a, b)):
            with torch.cuda.stream(s):
                got.append(block_calls(t))
        torch.cuda.synchronize()
        for w, o in zip(want, got):
            for k in w:
                assert torch.equal(w[k], o[k]), k


def test_empty_calls():
    e = lambda *s, dt=BF16: torch.zeros(s, dtype=dt, device=DEV)   # noqa: E731
    q = L.quantize_rows(e(0, 32))
    assert q["q"].shape == (0, 32) and q["scale"].shape == (0, 4)
    W8 = L.quantize_weights(e(2, 16, 32), transpose=True)
    seg = torch.zeros(3, dtype=torch.int32, device=DEV)
    assert L.grouped_forward_quantized(seg, q, W8)["y"].shape == (0, 16)
    w = e(64) + 1
    n = L.residual_norm(e(0, 64), y=e(0, 64), weight=w, gate=w)
    assert n["s"].shape == n["h"].shape == (0, 64)
    d = L.residual_norm_backward(e(0, 64), ds=e(0, 64), dh=e(0, 64), y=e(0, 64), weight=w,
                                 branch_weight=w, gate=w)
    for k in ("dweight", "dbranch_weight", "dgate"):
        assert bool((d[k] == 0).all()), k
    L.adamw_step([e(0)], [e(0)], [L.adamw_state(e(0), bits=8)], 1, 1e-3)
    torch.cuda.synchronize()


def test_binding_refuses_host_tensors():
    x, w = torch.zeros(4, 64, dtype=BF16), torch.zeros(64, dtype=BF16)
    for call in (lambda: L.quantize_rows(x), lambda: L.quantize_weights(x[None]),
                 lambda: L.residual_norm(x, weight=w),
                 lambda: L.residual_norm_backward(x, ds=x),
                 lambda: L.adamw_step([x], [x], [L.adamw_state(x)], 1, 1e-3),
                 lambda: L.residual_norm(put(x), weight=w),
                 lambda: L.adamw_step([put(x)], [put(x)], [L.adamw_state(x)], 1, 1e-3)):
        with pytest.raises(ValueError):
            call()


# ---------------------------------------------------------- a run of them together

def test_training_steps_of_a_block():
    """A block of a layer as it is trained: norm, router, sort, 8-bit expert products,
    combine, the norm behind the block, and back through all of it to AdamW on the
    weights.  The gradients are those of autograd through the same 8-bit weights and rows in
    float64 (rows' and gradients' roundings pass through unchanged), and the step is
    AdamW's."""
    T, E, K, d, f = 120, 4, 2, 256, 128
    g = gen(40)
    x = normal(g, (T, d), BF16)
    wn, wb = (1 + normal(g, (d,), F32, 0.1)).to(BF16), (1 + normal(g, (d,), F32, 0.1)).to(BF16)
    gate = normal(g, (d,), BF16, 0.5)
    logits = normal(g, (T, E), F32)
    Wu, Wd = normal(g, (E, 2 * f, d), F32, 0.08), normal(g, (E, d, f), F32, 0.08)
    dy = normal(g, (T, d), BF16)
    dv = {k: put(v) for k, v in dict(x=x, wn=wn, wb=wb, gate=gate, logits=logits, dy=dy).items()}
    pu, pd = put(Wu), put(Wd)

    # forward
    h = L.residual_norm(dv["x"], weight=dv["wn"])["h"]
    gt = L.gate_topk(dv["logits"], K)
    rt = L.route_sort(gt["ids"], E, weights=gt["weights"])
    W8u, W8d = L.quantize_weights(pu, transpose=True), L.quantize_weights(pd, transpose=True)
    h8 = L.quantize_rows(h)
    seg = rt["seg_offsets"]
    up = L.grouped_forward_quantized(seg, h8, W8u, row_index=rt["row_index"], act=L.ACT_SWIGLU,
                                     save_pre=True)
    a8 = L.quantize_rows(up["y"])
    down = L.grouped_forward_quantized(seg, a8, W8d)
    y = L.combine(down["y"], rt["pos"], gt["weights"])
    out = L.residual_norm(dv["x"], y=y, branch_weight=dv["wb"], gate=dv["gate"])["s"]
    # backward
    nb = L.residual_norm_backward(out, ds=dv["dy"], y=y, branch_weight=dv["wb"], gate=dv["gate"])
    cb = L.combine_backward(nb["dy"], down["y"], rt["pos"], gt["weights"])
    da = L.grouped_forward_quantized(seg, L.quantize_rows(cb["dyp"]), L.transposed_weights(W8d))["y"]
    dz = L.act_backward(seg, da, up["pre_a"], up["pre_b"], act=L.ACT_SWIGLU, dbias=False)["dz"]
    dhp = L.grouped_forward_quantized(seg, L.quantize_rows(dz), L.transposed_weights(W8u))["y"]
    dh = L.dispatch_backward(dhp, rt["pos"])
    nx = L.residual_norm_backward(dv["x"], ds=nb["dx"], dh=dh, weight=dv["wn"])
    counts = rt["counts"].tolist()
    ones = torch.ones(T * K, device=DEV)
    pairs = torch.arange(T * K, dtype=torch.int32, device=DEV)
    plan_d = L.Plan(counts, counts, d, f, L.BF16, dw_mode=L.DW_EXACT)
    dWd = L.grouped_backward(plan_d, pairs, ones, cb["dyp"], up["y"], pd.to(BF16))
    plan_u = L.Plan(counts, counts, 2 * f, d, L.BF16, dw_mode=L.DW_EXACT)
    hp = L.dispatch(h, rt["pos"])
    dWu = L.grouped_backward(plan_u, pairs, ones, dz, hp, pu.to(BF16))

    # the same in float64, over the values that the 8-bit weights stand for
    v = {k: t.double().requires_grad_() for k, t in dict(x=x, wn=wn, wb=wb, gate=gate).items()}
    v["u"] = B.weight_values(W8u["q"].cpu(), W8u["scale"].cpu()).requires_grad_()
    v["d"] = B.weight_values(W8d["q"].cpu(), W8d["scale"].cpu()).requires_grad_()
    _, hh = B.residual_norm(v["x"], weight=v["wn"])
    ids, w = O.gate(logits, K, "softmax")
    yy = torch.zeros(T, d, dtype=torch.float64)
    for k in range(K):
        z = (v["u"][ids[:, k]] @ hh[:, :, None])[:, :, 0]
        a = O.act("swiglu", z[:, :f], z[:, f:])
        yy = yy + w[:, k:k + 1] * (v["d"][ids[:, k]] @ a[:, :, None])[:, :, 0]
    want, _ = B.residual_norm(v["x"], y=yy, branch_weight=v["wb"], gate=v["gate"])
    ref = dict(zip(v, torch.autograd.grad((want * dy.double()).sum(), list(v.values()))))

    def close(got, ref, what, steps):
        """Roundings to e4m3 (2^-4 relative at most, independent and of both signs, so
        that their sums over 64 and more terms are below 2^-4 / 4 of the result's size) and
        bf16: `steps` of them lie on the path, against the 2-norm."""
        off = float((got.detach().cpu().double() - ref.detach()).norm() / ref.detach().norm())
        assert off <= steps * 2.0 ** -4, (what, off)
    close(out, want, "stream", 2)
    close(nx["dx"], ref["x"], "dx", 4)
    close(nx["dweight"], ref["wn"], "dwn", 4)
    close(nb["dbranch_weight"], ref["wb"], "dwb", 2)
    close(nb["dgate"], ref["gate"], "dgate", 2)
    close(dWd, ref["d"], "dWd", 4)
    close(dWu, ref["u"], "dWu", 4)

    # the step, with a bf16 copy for the products of the pruned backward
    for bits in (32, 8):
        par, grads = [pu.clone(), pd.clone()], [dWu, dWd]
        sts = [L.adamw_state(t, bits) for t in par]
        copies = [torch.empty_like(t, dtype=BF16) for t in par]
        L.adamw_step(par, grads, sts, 1, 1e-3, (0.9, 0.95), 1e-8, 0.1, copies=copies, seed=1)
        for t, w0, gw, c in zip(par, (Wu, Wd), grads, copies):
            n = w0.numel()
            p1, _, _ = B.adamw(w0.view(-1), gw.cpu().view(-1), torch.zeros(n), torch.zeros(n), 1, 1e-3,
                               (0.9, 0.95), 1e-8, 0.1)
            # a first step moves each weight by lr at most: 16 u of that, 4 u of the weight
            within(t.view(-1), p1, 16 * U * 1e-3 + 5 * U * w0.view(-1).double().abs(), "step")
            assert torch.equal(c, t.to(BF16))
