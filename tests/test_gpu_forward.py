"""Forward-side operators on the GPU against the float64 oracle: every
direction, type and variant, odd sizes, masked and empty rows, captured graphs,
other streams, and a whole expert layer forward and backward.

Error bounds, with u = 2^-24 (half a float32 step) and h = half a step of the
output type (2^-8 for bf16, u for float32), are derived where they are used."""
import math

import pytest
import torch

from oracle import forward_oracle as O
from pruned_expert_backward_amd import lrmoe as L

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

DEV = torch.device("cuda:0")
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
ACTS = {"none": L.ACT_NONE, "relu": L.ACT_RELU, "silu": L.ACT_SILU, "gelu": L.ACT_GELU,
        "swiglu": L.ACT_SWIGLU}
SCORES = {"softmax": L.GATE_SOFTMAX, "sigmoid": L.GATE_SIGMOID}
BF16, F32 = torch.bfloat16, torch.float32


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def normal(g, shape, dt, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(dt)


def within(got, want, bound, what):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, what
    over = (got - want).abs() - bound
    assert torch.isfinite(got).all(), what
    assert (over <= 0).all(), f"{what}: {float(over.max()):.3e} over the bound"


# ------------------------------------------------------------------- gate

GATE = [(1, 1, 1), (1, 8, 2), (5, 16, 4), (7, 17, 3), (33, 60, 8), (64, 128, 8), (19, 97, 5),
        (9, 256, 16), (6, 256, 17), (5, 300, 8), (3, 511, 64), (4, 1024, 10), (130, 128, 1)]


def gate_bound(x, w):
    """Relative error of a weight.  Two exponentials' arguments x - m are
    rounded once, u |x - m| each, the library's expf adds 2 u; a sum of E terms
    adds at most (16 + 6) u (16 in a lane, 6 exchanges), sigmoid's 1 / (1 + e)
    3 u more, the division and the scale u each; the range of finite logits
    bounds |x - m|.  1e-37 covers the float32 subnormals."""
    fin = x[torch.isfinite(x)].double()
    span = float(fin.max() - fin.min()) if fin.numel() else 0.0
    return (2 * min(span, 200.0) + 40) * U * w.abs() + 1e-37


@pytest.mark.parametrize("T,E,K", GATE)
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("score,renorm,biased", [
    ("softmax", True, False), ("softmax", False, False), ("sigmoid", True, False),
    ("sigmoid", False, False), ("sigmoid", True, True)])
def test_gate(T, E, K, dt, score, renorm, biased):
    g = gen(T * 1000 + E)
    x = normal(g, (T, E), dt, 1.5)
    bias = normal(g, (E,), F32, 0.2) if biased else None
    ids, w = O.gate(x, K, score, bias, renorm, 1.25)
    out = L.gate_topk(x.to(DEV), K, score=SCORES[score], renorm=renorm, scale=1.25,
                      select_bias=None if bias is None else bias.to(DEV))
    assert out["ids"].dtype == torch.int32 and torch.equal(out["ids"].cpu().long(), ids)
    within(out["weights"], w, gate_bound(x, w), "weights")


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("score,biased", [("softmax", False), ("sigmoid", False),
                                          ("sigmoid", True)])
def test_gate_ties_masks_and_extremes(dt, score, biased):
    inf, nan, low = float("inf"), float("nan"), torch.finfo(dt).min
    x = torch.zeros((10, 20))
    x[0] = torch.arange(20) % 3                  # many equal logits: lower experts first
    x[1] = -inf                                  # nothing left
    x[2] = nan
    x[3, 4:] = -inf                              # fewer than K
    x[4] = low                                   # the type's lowest value is a logit like others
    x[5] = -inf
    x[5, 7] = low
    x[6, 3] = inf
    x[7] = torch.linspace(-2000, -1000, 20)      # sigmoids that underflow
    x[8, 2], x[8, 9] = nan, -inf
    x[9] = torch.linspace(-30, 30, 20)
    x = x.to(dt)
    bias = torch.zeros(20) if biased else None   # equal sigmoids stay ties
    K = 6
    for renorm in (True, False):
        ids, w = O.gate(x, K, score, bias, renorm)
        out = L.gate_topk(x.to(DEV), K, score=SCORES[score], renorm=renorm,
                          select_bias=None if bias is None else bias.to(DEV))
        assert torch.equal(out["ids"].cpu().long(), ids)
        within(out["weights"], w, 2 * 2000 * U * w.abs() + 40 * U * w.abs() + 1e-37, "weights")
        dw = normal(gen(4), (10, K), F32)
        got = L.gate_topk_backward(x.to(DEV), out["ids"], dw.to(DEV), score=SCORES[score],
                                   renorm=renorm)
        want = O.gate_grad(x, ids, dw, score, renorm)
        # a factor w (bounded as above) times differences of |dw| terms
        within(got, want, (2 * 2000 + 80) * U * 2 * dw.abs().sum(1, keepdim=True)
               + HALF[dt] * want.abs(), "dlogits")


@pytest.mark.parametrize("E,K", [(128, 8), (40, 3), (256, 16), (300, 20)])
def test_gate_near_keys(E, K):
    """Biased keys that float32 cannot order: differences of 2^-30 and less,
    equal keys, whole rows of them (more than the lanes hold), keys at the
    border of the K chosen, infinite biases."""
    g = gen(E)
    T = 12
    x = normal(g, (T, E), F32, 1.0)
    bias = normal(g, (E,), F32, 0.1)
    key = torch.sigmoid(x.double())
    # rows 0..5: x chosen so that the key of expert e is the row's common value
    # to within float32's rounding of x
    goal = 0.5 + 0.2 * torch.rand((6, 1), generator=g).double()
    want = (goal - bias.double()).clamp(0.05, 0.95)
    x[:6] = torch.log(want / (1 - want)).float()
    x[3:6, K + 2:] = -3.0            # only a few near ones
    x[6] = 0.25                      # equal logits, keys by bias alone
    x[7, ::3] = float("-inf")
    ids, w = O.gate(x, K, "sigmoid", bias, True, 1.0)
    out = L.gate_topk(x.to(DEV), K, score=L.GATE_SIGMOID, select_bias=bias.to(DEV))
    assert torch.equal(out["ids"].cpu().long(), ids)
    within(out["weights"], w, gate_bound(x, w), "weights")
    bias[:] = 0.125                  # equal biases: ties of equal logits
    x[:, 1::2] = x[:, ::2][:, :x[:, 1::2].shape[1]]
    bias[5], bias[6], bias[7] = float("inf"), float("-inf"), float("nan")
    ids, w = O.gate(x, K, "sigmoid", bias, True, 1.0)
    out = L.gate_topk(x.to(DEV), K, score=L.GATE_SIGMOID, select_bias=bias.to(DEV))
    assert torch.equal(out["ids"].cpu().long(), ids)


@pytest.mark.parametrize("E,K", [(40, 15), (40, 16), (256, 16), (64, 17), (300, 63), (300, 64),
                                 (16, 16), (128, 1)])
def test_gate_near_keys_at_the_last_slot(E, K):
    """All keys far apart but those of ranks K and K + 1, which one float32 sum
    rounds to the same number: the one a float32 step larger is chosen, though
    its expert is the higher one."""
    x = torch.zeros((1, E))                                  # sigmoid 1/2, exactly
    bias = 0.45 - 0.002 * torch.arange(E, dtype=torch.float32) * (256 / max(E, 256))
    if K < E:
        for _ in range(64):   # a step up that float32's 1/2 + bias does not see
            bias[K] = torch.nextafter(bias[K - 1], torch.tensor(1.0))
            if 0.5 + bias[K] == 0.5 + bias[K - 1]:
                break
            bias[K - 1] = torch.nextafter(bias[K - 1], torch.tensor(-1.0))
        assert 0.5 + bias[K] == 0.5 + bias[K - 1] and bias[K] > bias[K - 1]
    ids, _ = O.gate(x, K, "sigmoid", bias)
    out = L.gate_topk(x.to(DEV), K, score=L.GATE_SIGMOID, select_bias=bias.to(DEV))
    assert torch.equal(out["ids"].cpu().long(), ids)


@pytest.mark.parametrize("T,E,K", GATE)
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False),
                                          ("sigmoid", True), ("sigmoid", False)])
def test_gate_gradient(T, E, K, dt, score, renorm):
    g = gen(T * 77 + E)
    x = normal(g, (T, E), dt, 1.5)
    ids, _ = O.gate(x, K, score, None, renorm)
    ids[0, 0] = -1                       # a slot without an expert
    if T > 2:
        ids[1, :] = E + 3                # a padded row
    if T > 3 and K > 1:
        ids[2, 1] = ids[2, 0]            # the same expert twice
    dw = normal(g, (T, K), F32)
    want = O.gate_grad(x, ids, dw, score, renorm, 0.75)
    got = L.gate_topk_backward(x.to(DEV), ids.int().to(DEV), dw.to(DEV), score=SCORES[score],
                               renorm=renorm, scale=0.75)
    assert got.dtype == dt
    # p (dw - dot): p <= 1 with the weights' relative error (span <= 20), the
    # sum over K slots adds 7 u of sum |p dw| <= sum |dw|
    bound = (2 * 20 + 60) * U * 2 * dw.abs().sum(1, keepdim=True).double()
    within(got, want, bound + HALF[dt] * want.abs(), "dlogits")


def test_gate_gradient_against_differences():
    g = gen(3)
    x = normal(g, (4, 24), torch.float64)
    dw = normal(g, (4, 5), F32)
    for score in SCORES:
        for renorm in (True, False):
            ids, _ = O.gate(x, 5, score, None, renorm)

            def loss(v):
                p = torch.softmax(v, 1) if score == "softmax" else torch.sigmoid(v)
                w = p.gather(1, ids)
                w = w / w.sum(1, keepdim=True) if renorm else w
                return (w * dw.double()).sum(1)
            got = L.gate_topk_backward(x.float().to(DEV), ids.int().to(DEV), dw.to(DEV),
                                       score=SCORES[score], renorm=renorm).cpu().double()
            for e in range(24):
                d = torch.zeros_like(x)
                d[:, e] = 1e-5
                diff = (loss(x.float().double() + d) - loss(x.float().double() - d)) / 2e-5
                # central differences: third derivatives <= sum |dw|, step^2 1e-10,
                # cancellation 2^-52 / 1e-5; the kernel's own bound as above
                assert ((got[:, e] - diff).abs() <= 1e-7 + 200 * U * dw.abs().sum(1)).all()


# --------------------------------------------------------------- sort, rows

def route(g, T, K, E_all):
    return torch.stack([torch.randperm(E_all, generator=g)[:K] for _ in range(T)]).int() if T else \
        torch.zeros((0, K), dtype=torch.int32)


SORT = [(0, 2, 4, 4), (1, 1, 1, 1), (3, 2, 4, 8), (64, 8, 16, 128), (37, 5, 7, 9),
        (1024, 8, 128, 128), (1025, 8, 16, 128), (4099, 3, 256, 256), (9000, 2, 255, 300),
        (17001, 8, 3, 24)]


@pytest.mark.parametrize("T,K,E,E_all", SORT)
@pytest.mark.parametrize("weighted", [True, False])
def test_route_sort(T, K, E, E_all, weighted):
    g = gen(T + E)
    ids = route(g, T, K, E_all)
    w = torch.rand((T, K), generator=g)
    want = O.sort(ids, E, w if weighted else None)
    out = L.route_sort(ids.to(DEV), E, weights=w.to(DEV) if weighted else None)
    for k in ("counts", "seg_offsets", "row_index", "pos"):
        assert torch.equal(out[k].cpu().long(), want[k]), k
    if weighted:
        assert torch.equal(out["alpha"].cpu(), want["alpha"])
    else:
        assert "alpha" not in out
    # the counts are those of the quota planner
    if T:
        plan = L.plan_quota_device(E, ids.to(DEV).reshape(-1), ("ratio", 1, 1))
        assert torch.equal(plan["counts"], out["counts"])
        assert torch.equal(plan["seg_offsets"].int(), out["seg_offsets"])


def test_route_sort_one_expert_and_odd_ids():
    big = 2 ** 31 - 1
    ids = torch.tensor([[3, -5], [big, 3], [3, -big - 1], [-1, 4]], dtype=torch.int32)
    want, out = O.sort(ids, 4), L.route_sort(ids.to(DEV), 4)
    for k in ("counts", "seg_offsets", "row_index", "pos"):
        assert torch.equal(out[k].cpu().long(), want[k]), k
    ids = torch.full((5000, 2), 7, dtype=torch.int32)     # every slot on one expert, twice a token
    out = L.route_sort(ids.to(DEV), 8)
    assert torch.equal(out["pos"].cpu().reshape(-1), torch.arange(10000, dtype=torch.int32))
    assert out["counts"].tolist() == [0] * 7 + [10000]


def test_route_sort_millions():
    """More ids than 1024 workgroups take in one round, against torch's stable sort."""
    T, K, E = 300_001, 8, 100
    ids = torch.randint(-3, 140, (T, K), generator=gen(1), dtype=torch.int32).to(DEV)
    w = torch.rand((T, K), device=DEV)
    out = L.route_sort(ids, E, weights=w)
    flat = ids.reshape(-1).long()
    key, order = torch.sort(torch.where((flat >= 0) & (flat < E), flat, E), stable=True)
    P = int((key < E).sum())
    assert int(out["seg_offsets"][E]) == P
    assert torch.equal(out["counts"], torch.bincount(key[:P], minlength=E))
    assert torch.equal(out["row_index"][:P].long(), order[:P] // K)
    assert (out["row_index"][P:] == -1).all() and (out["alpha"][P:] == 0).all()
    assert torch.equal(out["alpha"][:P], w.reshape(-1)[order[:P]])
    assert torch.equal(out["pos"].reshape(-1)[order[:P]].long(), torch.arange(P, device=DEV))
    assert (out["pos"].reshape(-1)[order[P:]] == -1).all()


ROWS = [(1, 1, 4, 8), (3, 2, 4, 16), (5, 8, 16, 264), (33, 3, 7, 1024), (9, 9, 20, 2056),
        (20, 17, 40, 40), (257, 4, 6, 512)]


def placed(T, K, E, here):
    """Places of T x K slots over 2 E experts, those of E here; with a gap and
    places outside the rows."""
    g = gen(T * K + E)
    ids = route(g, T, K, max(2 * E, K))
    pos = O.sort(ids, E)["pos"]
    P = int((pos >= 0).sum())
    pos = pos.clone()
    if here and P:
        pos[pos == P // 2] = -7          # a row that no slot names
        pos[pos < 0] = P + 5             # places outside the rows
    return pos, P + 2


@pytest.mark.parametrize("T,K,E,D", ROWS)
@pytest.mark.parametrize("dt", [F32, BF16])
def test_dispatch(T, K, E, D, dt):
    pos, P = placed(T, K, E, True)
    x = normal(gen(D), (T, D), dt)
    xp = torch.full((P, D), 3.0, dtype=dt)
    want = O.dispatch(x, pos, xp)
    got = L.dispatch(x.to(DEV), pos.int().to(DEV), xp=xp.to(DEV))
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("T,K,E,D", ROWS)
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("residual", [True, False])
def test_combine(T, K, E, D, dt, residual):
    pos, P = placed(T, K, E, True)
    g = gen(D + T)
    yp, w = normal(g, (P, D), dt), torch.rand((T, K), generator=g)
    res = normal(g, (T, D), dt) if residual else None
    want, mag = O.combine(yp, pos, w, res)
    yp[P - 1] = float("nan")     # a row that no slot names is not read
    y = L.combine(yp.to(DEV), pos.int().to(DEV), w.to(DEV),
                  residual=None if res is None else res.to(DEV))
    # K fused multiply-adds in float32, then one rounding
    within(y, want, (K + 1) * U * mag + HALF[dt] * (want.abs() + (K + 1) * U * mag), "y")


@pytest.mark.parametrize("T,K,E,D", ROWS)
@pytest.mark.parametrize("dt,out", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
def test_dispatch_gradient(T, K, E, D, dt, out):
    pos, P = placed(T, K, E, True)
    dxp = normal(gen(D), (P, D), dt)
    want, mag = O.combine(dxp, pos)
    got = L.dispatch_backward(dxp.to(DEV), pos.int().to(DEV), dtype=out)
    assert got.dtype == out
    within(got, want, K * U * mag + HALF[out] * (want.abs() + K * U * mag), "dx")


@pytest.mark.parametrize("T,K,E,D", ROWS)
@pytest.mark.parametrize("dt", [F32, BF16])
def test_combine_gradient(T, K, E, D, dt):
    pos, P = placed(T, K, E, True)
    g = gen(D + 2 * T)
    dy, yp, w = normal(g, (T, D), dt), normal(g, (P, D), dt), torch.rand((T, K), generator=g)
    dyp0 = torch.full((P, D), 3.0, dtype=dt)
    dyp, dw, mag = O.combine_grad(dy, yp, pos, w, dyp0)
    out = L.combine_backward(dy.to(DEV), yp.to(DEV), pos.int().to(DEV), w.to(DEV),
                             out=dict(dyp=dyp0.to(DEV),
                                      dweights=torch.empty((T, K), device=DEV)))
    # one product, one rounding to storage
    within(out["dyp"], dyp, (U + HALF[dt] * (1 + U)) * dyp.abs() + 1e-38, "dyp")
    # a lane adds D / 256 terms at most, rounded up to whole pieces of 8; then
    # 6 exchanges and 4 waves
    within(out["dweights"], dw, (math.ceil(D / 2048) * 8 + 10) * U * mag + 1e-38, "dweights")


def test_combine_gradient_against_differences():
    g = gen(12)
    pos = O.sort(route(g, 6, 3, 5), 5)["pos"]
    dy, yp, w = normal(g, (6, 16), F32), normal(g, (18, 16), F32), torch.rand((6, 3), generator=g)
    out = L.combine_backward(dy.to(DEV), yp.to(DEV), pos.int().to(DEV), w.to(DEV))

    def loss(yp_, w_):
        return float((O.combine(yp_, pos, w_)[0] * dy.double()).sum())
    for at in [(0, 0), (2, 1), (5, 2)]:   # the loss is linear in each: a unit step is exact
        d = torch.zeros(6, 3, dtype=torch.float64)
        d[at] = 1.0
        diff = loss(yp, w.double() + d) - loss(yp, w.double())
        assert abs(float(out["dweights"][at]) - diff) <= 1e-5 * (1 + abs(diff))
    for at in [(0, 3), (17, 15), (9, 0)]:
        d = torch.zeros(18, 16, dtype=torch.float64)
        d[at] = 1.0
        diff = loss(yp.double() + d, w) - loss(yp, w)
        assert abs(float(out["dyp"][at]) - diff) <= 1e-5 * (1 + abs(diff))


# ------------------------------------------------------------ grouped product

def act_bound(name, z, ez, half):
    """Bound of act(z)'s error from that of z: slopes of SiLU and GELU are at
    most 1.13, the functions themselves are good to 16 u of |z| (expf and erff
    to 4 u, a few products)."""
    if name == "swiglu":
        F = z.shape[1] // 2
        a, b, ea, eb = z[:, :F], z[:, F:], ez[:, :F], ez[:, F:]
        s = O.act("silu", a)
        es = 1.13 * ea + 16 * U * a.abs()
        y, ey = s * b, es * (b.abs() + eb) + s.abs() * eb + U * (s * b).abs()
    else:
        y = O.act(name, z)
        ey = 1.13 * ez + (0 if name in ("none", "relu") else 16 * U) * z.abs()
    return y, ey


def check_linear(seg, x, W, row, bias, res, name, pre, P=None):
    dt = x.dtype
    ref = O.linear(seg, x, W, row, bias, res, name)
    P, d_out = ref["z"].shape
    F = d_out // 2 if name == "swiglu" else d_out
    out = dict(y=torch.full((P, F), 5.0, dtype=dt, device=DEV))
    if pre:
        out["pre_a"] = torch.full((P, F), 6.0, dtype=dt, device=DEV)
        if name == "swiglu":
            out["pre_b"] = torch.full((P, F), 7.0, dtype=dt, device=DEV)
    put = lambda t: None if t is None else t.to(DEV)   # noqa: E731
    L.grouped_forward(put(torch.tensor(seg, dtype=torch.int32)), put(x), put(W), put(row),
                      put(bias), put(res), ACTS[name], out=out)
    # a float32 sum of d_in + 1 terms in any order, each step off by one float32 step
    ez = (x.shape[1] + 2) * 2 * U * ref["mag"]
    y, ey = act_bound(name, ref["z"], ez, HALF[dt])
    if res is not None:
        ey = ey + U * (ref["y"].abs() + ey)
    n = seg[-1]
    within(out["y"][:n], ref["y"][:n], (ey + HALF[dt] * (ref["y"].abs() + ey))[:n] + 1e-38, "y")
    if pre:
        z = torch.cat([out["pre_a"], out["pre_b"]], 1) if name == "swiglu" else out["pre_a"]
        within(z[:n], ref["z"][:n], (ez + HALF[dt] * (ref["z"].abs() + ez))[:n] + 1e-38, "pre")
        assert (out["pre_a"][n:] == 6.0).all()
    assert (out["y"][n:] == 5.0).all()     # rows behind the last segment
    return out


# segments; most calls have few enough workgroups to do without tiles (tile
# shapes: the widest of the last ones here, below, test_gpu_forward_tiles.py)
SEGS = [[0, 1], [0, 0, 0, 1], [0, 3, 3, 20, 21], [0, 16, 33], [0, 40, 41, 41, 170],
        [0, 127, 255, 384], [0, 300], [0, 5, 600, 1100], [0, 0, 0]]
DIMS = [(8, 8), (24, 40), (64, 136), (72, 264), (264, 520)]


def linear_inputs(seg, d_in, d_out, dt, seed, spare=0, index=True, name="none"):
    g = gen(seed)
    E, P = len(seg) - 1, seg[-1] + spare
    T = max(1, P // 2) if index else P
    x = normal(g, (T, d_in), dt)
    W = normal(g, (E, d_out, d_in), dt, 0.1)
    row = torch.randint(0, T, (P,), generator=g).int() if index else None
    F = d_out // 2 if name == "swiglu" else d_out
    return x, W, row, normal(g, (E, d_out), dt), normal(g, (P, F), dt)


@pytest.mark.parametrize("seg", SEGS, ids=str)
@pytest.mark.parametrize("d_in,d_out", DIMS)
@pytest.mark.parametrize("dt", [BF16, F32])
def test_linear_shapes(seg, d_in, d_out, dt):
    x, W, row, bias, res = linear_inputs(seg, d_in, d_out, dt, len(seg) + d_in, spare=3)
    check_linear(seg, x, W, row, bias, res, "none", False)


def zipf_seg(P, E):
    w = torch.arange(1, E + 1).double() ** -0.8
    ends = (P * torch.cumsum(w, 0) / w.sum()).round().long().tolist()
    return [0] + ends[:-1] + [P]


# (segments, columns of y): each of the launch's tile shapes, by the workgroups
# that the call is expected to have
SHAPES = {
    "32x256": (zipf_seg(512, 64), 776), "32x64": (zipf_seg(300, 4), 1032),
    "64x64": (zipf_seg(1200, 4), 1032), "64x128": (zipf_seg(2500, 4), 1032),
    # 256-row tiles; 128-row ones where they fill one round; whole tiles, ends
    # of each class, and last rounds cut in four, in two and not at all
    "one round of 128": ([0, 4090], 1032), "whole and ends": ([0, 1500, 1501, 1700, 4200], 2056),
    "cut in four": ([0, 4100, 8200], 2304), "cut in two": ([0, 9990], 2304),
}


@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("name,d_in", [("none", 40), ("swiglu", 136)])
def test_linear_tile_shapes(shape, name, d_in):
    seg, F = SHAPES[shape]
    F = F // 16 * 8 if name == "swiglu" else F
    x, W, row, bias, _ = linear_inputs(seg, d_in, 2 * F if name == "swiglu" else F, BF16, 77,
                                       name=name)
    check_linear(seg, x, W, row, bias, None, name, name == "swiglu")


@pytest.mark.parametrize("name", ["gelu", "swiglu"])
@pytest.mark.parametrize("seg", [zipf_seg(900, 4), [0, 700]], ids=str)
def test_linear_float32_tiles(name, seg):
    x, W, row, bias, res = linear_inputs(seg, 100, 1224, F32, 78, name=name)
    check_linear(seg, x, W, row, bias, res, name, True)


@pytest.mark.parametrize("dt,T", [(BF16, 1_100_000), (F32, 550_000)])
def test_linear_tiles_of_rows_beyond_32_bits(dt, T):
    """Picked rows of an x beyond a buffer's 2 GiB, in tiles (300 rows, many
    columns); also an index out of range."""
    d_in, F, n = 2048, 2056, 300
    x = torch.zeros((T, d_in), dtype=dt, device=DEV)
    tail = normal(gen(6), (n, d_in), dt)
    x[T - n:] = tail.to(DEV)
    W = normal(gen(7), (1, F, d_in), dt, 0.1)
    row = torch.arange(T - n, T, dtype=torch.int32, device=DEV)
    row[5], row[250] = T, -3
    tail[5] = tail[250] = 0
    y = L.grouped_forward(torch.tensor([0, n], dtype=torch.int32, device=DEV), x, W.to(DEV),
                          row_index=row)["y"]
    ref = O.linear([0, n], tail, W)
    ez = (d_in + 2) * 2 * U * ref["mag"]
    within(y, ref["y"], ez + HALF[dt] * (ref["y"].abs() + ez), "y")


def test_linear_expert_beyond_a_buffer():
    """One expert's weights of more than 2 GiB: its last and first columns."""
    d_in, d_out, n = 32768, 32776, 130
    W = torch.zeros((1, d_out, d_in), dtype=BF16, device=DEV)
    ends = normal(gen(9), (2, 16, d_in), BF16, 0.1)
    W[0, :16], W[0, -16:] = ends[0].to(DEV), ends[1].to(DEV)
    x = normal(gen(10), (n, d_in), BF16)
    for rows in (1, n):
        seg = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
        y = L.grouped_forward(seg, x[:rows].to(DEV).contiguous(), W)["y"]
        for part, got in ((ends[0], y[:, :16]), (ends[1], y[:, -16:])):
            ref = O.linear([0, rows], x[:rows], part[None])
            ez = (d_in + 2) * 2 * U * ref["mag"]
            within(got, ref["y"], ez + HALF[BF16] * (ref["y"].abs() + ez), "y")
        assert (y[:, 16:-16] == 0).all()


def test_linear_rows_in_any_batch_company():
    """NaN rows of one expert or token touch no other row."""
    seg = zipf_seg(2500, 4)
    x, W, row, _, _ = linear_inputs(seg, 72, 1032, BF16, 79)
    x[3] = float("nan")
    W[1, 5] = float("inf")
    put = lambda t: t.to(DEV)   # noqa: E731
    s = torch.tensor(seg, dtype=torch.int32, device=DEV)
    y = L.grouped_forward(s, put(x), put(W), row_index=put(row))["y"].float().cpu()
    e = torch.bucketize(torch.arange(2500), torch.tensor(seg[1:]), right=True)
    bad_row = row == 3
    assert torch.isnan(y[bad_row]).all()
    rest = y[~bad_row]
    inf_col = torch.zeros_like(y, dtype=torch.bool)
    inf_col[e == 1, 5] = True
    assert torch.isfinite(rest[~inf_col[~bad_row]]).all()
    assert not torch.isfinite(rest[inf_col[~bad_row]]).any()


@pytest.mark.parametrize("name", list(ACTS))
@pytest.mark.parametrize("seg", [[0, 2, 9], [0, 33, 33, 150], [0, 270, 530]], ids=str)
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("bias,residual,pre", [(False, False, False), (True, True, True),
                                               (False, True, False), (True, False, True)])
def test_linear_epilogues(name, seg, dt, bias, residual, pre):
    x, W, row, b, r = linear_inputs(seg, 48, 208, dt, 5, index=False, name=name)
    check_linear(seg, x, W, None, b if bias else None, r if residual else None, name, pre)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("P", [3, 100, 600])
def test_linear_bad_rows_and_masked_values(dt, P):
    """Row indices out of range read zero rows, and NaN or infinite values in
    rows of x, of W's other experts or behind the row's end touch nothing else."""
    seg = [0, P - 1, P]
    x, W, row, bias, _ = linear_inputs(seg, 40, 72, dt, 8)
    row[0], row[P - 1] = -1, x.shape[0]
    if P > 3:
        row[P // 2] = 2 ** 31 - 1
    used = row.clone()
    used[(row < 0) | (row >= x.shape[0])] = 0
    spare = [r for r in range(x.shape[0]) if r not in set(row.tolist())]
    x[spare] = float("nan")
    check_linear(seg, x, W, row, bias, None, "silu", True)


@pytest.mark.parametrize("dt", [BF16, F32])
def test_linear_offsets_out_of_order(dt):
    """Offsets that do not ascend or pass the rows are bounded, not followed."""
    P = 40
    x, W, _, _, _ = linear_inputs([0, 10, 20, 30, P], 32, 64, dt, 9, index=False)
    for seg in ([0, 30, 10, 60, 40], [-5, 10, 10, 2 ** 31 - 1, 0], [50, 60, 70, 80, 90]):
        s = torch.tensor(seg, dtype=torch.int32, device=DEV)
        y = L.grouped_forward(s, x.to(DEV), W.to(DEV))["y"]
        dz = L.act_backward(s, y, act=L.ACT_NONE)
        torch.cuda.synchronize()
        assert y.shape == (P, 64) and dz["dbias"].shape == (4, 64)


def test_linear_many_experts():
    g = gen(31)
    n = torch.randint(0, 40, (256,), generator=g)
    n[::5] = 0
    seg = [0] + torch.cumsum(n, 0).tolist()
    x, W, row, bias, res = linear_inputs(seg, 32, 48, BF16, 32)
    check_linear(seg, x, W, row, bias, res, "gelu", False)


def test_linear_tokens_beyond_32_bits():
    """x of more than 2^32 bytes and 2^31 values: rows at its end."""
    T, d_in = 1_100_000, 2048
    x = torch.zeros((T, d_in), dtype=BF16, device=DEV)
    tail = normal(gen(1), (300, d_in), BF16)
    x[T - 300:] = tail.to(DEV)
    W = normal(gen(2), (1, 64, d_in), BF16, 0.1)
    for n in (5, 100, 300):
        row = torch.arange(T - n, T, dtype=torch.int32, device=DEV)
        seg = torch.tensor([0, n], dtype=torch.int32, device=DEV)
        y = L.grouped_forward(seg, x, W.to(DEV), row_index=row)["y"]
        ref = O.linear([0, n], tail[300 - n:], W)
        ez = (d_in + 2) * 2 * U * ref["mag"]
        within(y, ref["y"], ez + HALF[BF16] * (ref["y"].abs() + ez), "y")


def test_rows_beyond_32_bits():
    """Pair rows of more than 2^32 bytes: the places at their end."""
    P, D = 600_000, 4096
    rows = torch.zeros((P, D), dtype=BF16, device=DEV)
    pos = torch.tensor([[P - 1, 0], [P - 3, P - 2]], dtype=torch.int32, device=DEV)
    x = normal(gen(3), (2, D), BF16).to(DEV)
    L.dispatch(x, pos, xp=rows)
    for t, k in ((0, 0), (0, 1), (1, 0), (1, 1)):
        assert torch.equal(rows[pos[t, k].item()], x[t])
    w = torch.tensor([[0.5, 0.25], [1.0, 2.0]], device=DEV)
    assert torch.equal(L.combine(rows, pos, w), (x.float() * torch.tensor([[0.75], [3.0]],
                                                                          device=DEV)).to(BF16))
    dyp = torch.zeros_like(rows)
    out = L.combine_backward(x, rows, pos, w,
                             out=dict(dyp=dyp, dweights=torch.empty((2, 2), device=DEV)))
    assert torch.equal(dyp[P - 2], (2 * x[1].float()).to(BF16))
    assert torch.allclose(out["dweights"][1], x[1].float().square().sum().expand(2), rtol=1e-5)


@pytest.mark.parametrize("name", list(ACTS))
@pytest.mark.parametrize("seg", [[0, 1], [0, 0, 70, 70, 200], [0, 64, 128, 131], [0, 0]], ids=str)
@pytest.mark.parametrize("F", [8, 40, 520])
@pytest.mark.parametrize("dt,out", [(BF16, BF16), (BF16, F32), (F32, F32)])
def test_act_gradient(name, seg, F, dt, out):
    g = gen(F + len(seg))
    P = seg[-1] + 2
    dy, a, b = (normal(g, (P, F), dt, s) for s in (1.0, 2.0, 1.0))
    glu = name == "swiglu"
    ref = O.act_grad(seg, dy, a, b if glu else None, name)
    bufs = dict(dz=torch.full((P, 2 * F if glu else F), 4.0, dtype=out, device=DEV),
                dbias=torch.empty((len(seg) - 1, 2 * F if glu else F), device=DEV))
    L.act_backward(torch.tensor(seg, dtype=torch.int32, device=DEV), dy.to(DEV),
                   None if name == "none" else a.to(DEV), b.to(DEV) if glu else None,
                   act=ACTS[name], out=bufs)
    n = seg[-1]
    # slope: expf/erff to 4 u and a few products, terms up to 1 + |a|; GELU's
    # exponent -a^2/2 carries a relative u, so e^.. is off by a^2 u
    size = dy.double().abs() * (1 + a.double().abs()) * (1 + a.double() ** 2)
    e = 16 * U * (torch.cat([size * b.double().abs(), size], 1) if glu else size)
    if name in ("none", "relu"):
        e = e * 0
    dz = ref["dz"]
    within(bufs["dz"][:n], dz[:n], (e + HALF[out] * (dz.abs() + e))[:n] + 1e-38, "dz")
    assert (bufs["dz"][n:] == 4.0).all()
    # a lane adds 16 rows, 3 other waves, then the runs of 64 rows
    es = torch.stack([e[seg[i]:seg[i + 1]].sum(0) for i in range(len(seg) - 1)])
    within(bufs["dbias"], ref["dbias"], es + (19 + n // 64 + 1) * U * (ref["mag"] + es) + 1e-38,
           "dbias")


def test_act_gradient_without_bias_sum():
    dy = normal(gen(5), (70, 16), BF16).to(DEV)
    seg = torch.tensor([0, 70], dtype=torch.int32, device=DEV)
    out = L.act_backward(seg, dy, act=L.ACT_NONE, dbias=False)
    assert out["dbias"] is None and torch.equal(out["dz"], dy)


# ------------------------------------------------------------- the layer whole

def layer(x, logits, Wgu, Wd, bgu, K, res, E):
    """Forward of a gated-MLP expert layer from token rows and router logits."""
    gt = L.gate_topk(logits, K)
    rt = L.route_sort(gt["ids"], E, weights=gt["weights"])
    up = L.grouped_forward(rt["seg_offsets"], x, Wgu, row_index=rt["row_index"], bias=bgu,
                           act=L.ACT_SWIGLU, save_pre=True)
    down = L.grouped_forward(rt["seg_offsets"], up["y"], Wd)
    y = L.combine(down["y"], rt["pos"], gt["weights"], residual=res)
    return gt, rt, up, down, y


@pytest.mark.parametrize("T,E,K", [(40, 4, 2), (3, 8, 3), (400, 4, 3)])
def test_layer_forward_and_backward(T, E, K):
    """Router to residual and back, against autograd in float64: the forward
    calls' outputs are what the pruned backward reads (quotas = counts keep
    every pair)."""
    d, f = 64, 48
    g = gen(T)
    x, res = normal(g, (T, d), BF16), normal(g, (T, d), BF16)
    logits = normal(g, (T, E), F32)
    Wgu, Wd = normal(g, (E, 2 * f, d), BF16, 0.1), normal(g, (E, d, f), BF16, 0.1)
    dy = normal(g, (T, d), BF16)
    put = lambda t: t.to(DEV)   # noqa: E731
    gt, rt, up, down, y = layer(put(x), put(logits), put(Wgu), put(Wd), None, K, put(res), E)

    # float64 autograd over the same tokens
    v = {k: t.double().requires_grad_() for k, t in dict(x=x, l=logits, gu=Wgu, d=Wd).items()}
    ids, _ = O.gate(logits, K, "softmax")
    w = torch.softmax(v["l"].gather(1, ids), 1)
    want = res.double()
    for k in range(K):
        z = torch.einsum("td,tod->to", v["x"], v["gu"][ids[:, k]])
        h = O.act("swiglu", z[:, :f], z[:, f:])
        want = want + w[:, k:k + 1] * torch.einsum("tf,tof->to", h, v["d"][ids[:, k]])
    grads = dict(zip(v, torch.autograd.grad((want * dy.double()).sum(), list(v.values()))))

    def close(got, ref, what, steps):
        """bf16 roundings on the way (h, pair outputs, saved a and b, the
        handed-on gradients): each 2^-8 relative at most, against the largest
        entry; `steps` of them lie on the longest path."""
        ref = ref.detach()
        err = float((got.detach().cpu().double() - ref).abs().max())
        assert err <= steps * 2.0 ** -8 * float(ref.abs().max()), (what, err)
    assert torch.equal(gt["ids"].cpu().long(), ids)
    close(y, want, "y", 3)                       # h, pair rows, y
    counts = rt["counts"].tolist()
    plan = L.Plan(counts, counts, d, f, L.BF16, T=T, dw_mode=L.DW_EXACT)
    plan2 = L.Plan(counts, counts, 2 * f, d, L.BF16, T=T, dw_mode=L.DW_EXACT)
    out = L.glu_chain_backward(plan, plan2, rt["alpha"], put(dy), up["y"], put(Wd), up["pre_a"],
                               up["pre_b"], put(x), put(Wgu), g_row_index=rt["row_index"],
                               x_row_index=rt["row_index"])
    close(out["dW"], grads["d"], "dW down", 2)   # h (twice: its a, b and itself)
    close(out["dW2"], grads["gu"], "dW gate/up", 4)
    close(L.dispatch_backward(out["dx"], rt["pos"]), grads["x"], "dx", 4)
    cb = L.combine_backward(put(dy), down["y"], rt["pos"], gt["weights"])
    dl = L.gate_topk_backward(put(logits), gt["ids"], cb["dweights"])
    close(dl, grads["l"], "dlogits", 4)
    # the epilogue's gradient hands the same gate/up gradient on as the chain
    # does: from dh = W_d^T (alpha dy) per pair
    dh = torch.zeros((T * K, f), dtype=torch.float64)
    row = rt["row_index"].cpu().long()
    for e in range(E):
        at = slice(sum(counts[:e]), sum(counts[:e + 1]))
        dh[at] = dy[row[at]].double() @ Wd[e].double()
    dz = L.act_backward(rt["seg_offsets"], dh.float().to(BF16).to(DEV), up["pre_a"], up["pre_b"],
                        act=L.ACT_SWIGLU, dbias=False, dz_dtype=torch.float32)["dz"]
    close(dz, out["dgu_c"].cpu().double(), "dz", 2)


def test_layer_captured_and_replayed():
    """The whole forward and the gradients around it in one graph: nothing
    visits the host.  Replayed with new inputs, each replay against the eager
    calls, with eager work and waits between."""
    T, E, K, d, f = 65, 16, 4, 64, 48
    g = gen(8)
    x, logits, dy = (torch.zeros(s, dtype=t, device=DEV)
                     for s, t in (((T, d), BF16), ((T, E), F32), ((T, d), BF16)))
    Wgu, Wd = normal(g, (E, 2 * f, d), BF16, 0.1).to(DEV), normal(g, (E, d, f), BF16, 0.1).to(DEV)
    bgu = normal(g, (E, 2 * f), BF16).to(DEV)

    def work():
        gt, rt, up, down, y = layer(x, logits, Wgu, Wd, bgu, K, x, E)
        cb = L.combine_backward(dy, down["y"], rt["pos"], gt["weights"])
        dl = L.gate_topk_backward(logits, gt["ids"], cb["dweights"])
        dz = L.act_backward(rt["seg_offsets"], up["y"], up["pre_a"], up["pre_b"],
                            act=L.ACT_SWIGLU)
        return [y, cb["dyp"], dl, dz["dz"], dz["dbias"], rt["row_index"],
                L.dispatch_backward(L.dispatch(x, rt["pos"]), rt["pos"])]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    for i in range(4):
        x.copy_(normal(g, (T, d), BF16))
        logits.copy_(normal(g, (T, E), F32))
        dy.copy_(normal(g, (T, d), BF16))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        for a, b in zip(got, work()):
            assert torch.equal(a, b), i
        torch.cuda.synchronize()


def test_results_do_not_change_from_call_to_call():
    g = gen(17)
    x, W = normal(g, (700, 256), BF16).to(DEV), normal(g, (3, 512, 256), BF16, 0.1).to(DEV)
    seg = torch.tensor([0, 260, 261, 700], dtype=torch.int32, device=DEV)
    first = None
    for _ in range(3):
        up = L.grouped_forward(seg, x, W, act=L.ACT_SWIGLU, save_pre=True)
        dz = L.act_backward(seg, up["y"], up["pre_a"], up["pre_b"], act=L.ACT_SWIGLU)
        now = [up["y"], up["pre_a"], dz["dz"], dz["dbias"]]
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(first, now))


def test_two_streams_at_once():
    """Calls on two streams with their own buffers do not disturb each other."""
    g = gen(23)
    ids = [route(g, 3000, 8, 32).to(DEV) for _ in range(2)]
    x = [normal(g, (3000, 128), BF16).to(DEV) for _ in range(2)]
    W = normal(g, (32, 256, 128), BF16, 0.1).to(DEV)
    ref = []
    for i in range(2):
        rt = L.route_sort(ids[i], 32)
        ref.append((rt, L.grouped_forward(rt["seg_offsets"], x[i], W, row_index=rt["row_index"])))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                rt = L.route_sort(ids[i], 32)
                got.append((i, rt, L.grouped_forward(rt["seg_offsets"], x[i], W,
                                                     row_index=rt["row_index"])))
    torch.cuda.synchronize()
    for i, rt, out in got:
        assert torch.equal(rt["pos"], ref[i][0]["pos"])
        assert torch.equal(out["y"], ref[i][1]["y"])


def test_binding_checks_shapes_types_and_places():
    z = lambda *s, dt=BF16: torch.zeros(s, dtype=dt, device=DEV)   # noqa: E731
    i32 = torch.int32
    pos = z(4, 2, dt=i32)
    bad = [
        (ValueError, lambda: L.gate_topk(z(8), 2)),
        (L.LrmoeError, lambda: L.gate_topk(z(4, 8), 9)),
        (L.LrmoeError, lambda: L.gate_topk(z(4, 8), 2, select_bias=z(8, dt=F32))),
        (TypeError, lambda: L.gate_topk(z(4, 8, dt=torch.float16), 2)),
        (TypeError, lambda: L.gate_topk(z(4, 8), 2, score=1, select_bias=z(8))),
        (ValueError, lambda: L.gate_topk(z(8, 4).t(), 2)),
        (TypeError, lambda: L.route_sort(z(4, 2, dt=torch.int64), 3)),
        (ValueError, lambda: L.route_sort(pos, 3, weights=z(2, 4, dt=F32))),
        (ValueError, lambda: L.dispatch(z(3, 8), pos)),
        (ValueError, lambda: L.dispatch(z(4, 8), pos, xp=z(8, 16))),
        (TypeError, lambda: L.dispatch(z(4, 8), pos, xp=z(8, 8, dt=F32))),
        (L.LrmoeError, lambda: L.dispatch(z(4, 12), pos)),
        (ValueError, lambda: L.combine(z(8, 8), pos, z(4, 2, dt=F32).cpu())),
        (ValueError, lambda: L.combine(z(8, 8), pos, z(2, 4, dt=F32))),
        (TypeError, lambda: L.combine(z(8, 8), pos, z(4, 2))),
        (TypeError, lambda: L.combine(z(8, 8), pos, z(4, 2, dt=F32), residual=z(4, 8, dt=F32))),
        (ValueError, lambda: L.combine_backward(z(5, 8), z(8, 8), pos, z(4, 2, dt=F32))),
        (ValueError, lambda: L.grouped_forward(z(2, dt=i32), z(4, 8), z(2, 8, 8))),
        (ValueError, lambda: L.grouped_forward(z(3, dt=i32), z(4, 16), z(2, 8, 8))),
        (TypeError, lambda: L.grouped_forward(z(3, dt=i32), z(4, 8), z(2, 8, 8, dt=F32))),
        (ValueError, lambda: L.grouped_forward(z(3, dt=i32), z(4, 8), z(2, 8, 8), bias=z(8))),
        (ValueError, lambda: L.grouped_forward(z(3, dt=i32), z(4, 8), z(2, 16, 8),
                                               residual=z(4, 16), act=L.ACT_SWIGLU)),
        (L.LrmoeError, lambda: L.grouped_forward(z(3, dt=i32), z(4, 8), z(2, 8, 8),
                                                 act=L.ACT_SWIGLU)),
        (L.LrmoeError, lambda: L.grouped_forward(z(3, dt=i32), z(4, 8), z(2, 8, 8), act=9)),
        (L.LrmoeError, lambda: L.act_backward(z(3, dt=i32), z(4, 8), act=L.ACT_SILU)),
        (ValueError, lambda: L.act_backward(z(3, dt=i32), z(4, 8), z(4, 16), act=L.ACT_SILU)),
        (L.LrmoeError, lambda: L.act_backward(z(3, dt=i32), z(4, 8), ws=z(1, dt=torch.uint8))),
    ]
    for n, (err, call) in enumerate(bad):
        with pytest.raises(err):
            call()
            pytest.fail(f"call {n} was taken")


def test_empty_calls():
    z = lambda *s, dt=BF16: torch.zeros(s, dtype=dt, device=DEV)   # noqa: E731
    pos, w = z(0, 2, dt=torch.int32), z(0, 2, dt=F32)
    assert L.gate_topk(z(0, 8), 2)["ids"].shape == (0, 2)
    assert L.gate_topk_backward(z(0, 8), pos, w).shape == (0, 8)
    assert L.route_sort(pos, 3)["seg_offsets"].tolist() == [0, 0, 0, 0]
    assert L.dispatch(z(0, 8), pos).shape == (0, 8)
    assert L.combine(z(0, 8), pos, w).shape == (0, 8)
    none = torch.full((3, 2), -1, dtype=torch.int32, device=DEV)
    res = normal(gen(2), (3, 8), BF16).to(DEV)
    assert torch.equal(L.combine(z(0, 8), none, z(3, 2, dt=F32), residual=res), res)
    assert torch.equal(L.dispatch_backward(z(0, 8), none), z(3, 8))
    assert L.grouped_forward(z(3, dt=torch.int32), z(0, 8), z(2, 16, 8))["y"].shape == (0, 16)
    out = L.act_backward(z(3, dt=torch.int32), z(0, 8))
    assert torch.equal(out["dbias"], z(2, 8, dt=F32))
