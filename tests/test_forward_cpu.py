"""Forward-side entry points on the CPU: refusals (none of these calls reaches
a launch), workspace sizes, the binding's argument checks, and the float64
oracle against torch's autograd."""
import ctypes as C
import os

import pytest
import torch

from oracle import forward_oracle as O
from pruned_expert_backward_amd import lrmoe as L

if not os.path.exists(L.LIB_PATH):
    pytest.skip("liblrmoe.so not built (run __graft_entry__.build())", allow_module_level=True)

FAKE = 0x7F0000001000   # 16-byte aligned; validation fails before any use
NULL, INVALID, SHAPE, ALIGN, DTYPE, WORKSPACE = 1, 2, 3, 4, 5, 6


def gate(**kw):
    a = dict(T=4, E=8, K=2, dtype=L.F32, score=L.GATE_SOFTMAX, renorm=1, scale=1.0)
    a.update(kw)
    return L.Gate(*[a[k] for k in ("T", "E", "K", "dtype", "score", "renorm", "scale")])


def gate_call(fn="lrmoe_gate_topk", g=None, **over):
    names = (["logits", "bias", "ids", "weights"] if fn == "lrmoe_gate_topk"
             else ["logits", "ids", "dw", "dx"])
    a = {n: FAKE for n in names}
    if "bias" in a:
        a["bias"] = None
    a.update(over)
    g = gate() if g is None else g
    return getattr(L.lib(), fn)(C.byref(g), *[a[n] for n in names], None)


@pytest.mark.parametrize("kw,code", [
    (dict(E=0), INVALID), (dict(E=1025), INVALID), (dict(K=0), INVALID), (dict(K=9), INVALID),
    (dict(E=512, K=65), INVALID), (dict(score=2), INVALID), (dict(score=-1), INVALID),
    (dict(dtype=2), DTYPE), (dict(T=-1), SHAPE), (dict(T=2**31), SHAPE), (dict(T=2**30), SHAPE)])
@pytest.mark.parametrize("fn", ["lrmoe_gate_topk", "lrmoe_gate_topk_backward"])
def test_gate_refuses(fn, kw, code):
    assert gate_call(fn, gate(**kw)) == code


@pytest.mark.parametrize("fn,field", [("lrmoe_gate_topk", f) for f in ("logits", "ids", "weights")]
                         + [("lrmoe_gate_topk_backward", f) for f in ("logits", "ids", "dw", "dx")])
def test_gate_pointers(fn, field):
    assert gate_call(fn, **{field: None}) == NULL
    assert gate_call(fn, **{field: FAKE + 4}) == ALIGN


def test_gate_bias_needs_sigmoid():
    assert gate_call(bias=FAKE) == INVALID
    assert gate_call(g=gate(score=L.GATE_SIGMOID), bias=FAKE + 4) == ALIGN
    assert L.lib().lrmoe_gate_topk(None, FAKE, None, FAKE, FAKE, None) == NULL


def test_route_sort_refuses_and_sizes():
    f = L.lib().lrmoe_route_sort
    ok = dict(T=4, K=2, E=3, ids=FAKE, w=None, counts=FAKE, seg=FAKE, row=FAKE, pos=FAKE,
              alpha=None, ws=None, n=0)

    def call(**kw):
        return f(*{**ok, **kw}.values(), None)

    for kw, code in ((dict(E=0), INVALID), (dict(E=257), INVALID), (dict(K=0), INVALID),
                     (dict(K=65), INVALID), (dict(T=-1), SHAPE), (dict(T=2**30), SHAPE),
                     (dict(alpha=FAKE), NULL), (dict(alpha=FAKE + 8, w=FAKE), ALIGN),
                     (dict(w=FAKE + 4), ALIGN)):
        assert call(**kw) == code, kw
    for name in ("ids", "counts", "seg", "row", "pos"):
        assert call(**{name: None}) == NULL
        assert call(**{name: FAKE + 4}) == ALIGN
    # 4096 slots and fewer need no workspace; more, one row of E + 1 counts a workgroup
    assert L.route_sort_workspace_bytes(512, 8, 16) == 0
    n = L.route_sort_workspace_bytes(513, 8, 16)
    assert n == 3 * 17 * 4
    assert call(T=513, K=8, E=16, ws=None, n=n) == NULL
    assert call(T=513, K=8, E=16, ws=FAKE, n=n - 1) == WORKSPACE
    assert call(T=513, K=8, E=16, ws=FAKE + 4, n=n) == ALIGN
    with pytest.raises(L.LrmoeError):
        L.route_sort_workspace_bytes(4, 2, 0)


def test_row_movers_refuse():
    lib = L.lib()
    # dtype, T, K, D, P, pointers ...
    movers = {
        "lrmoe_dispatch": ([L.BF16, 4, 2, 16, 8], 3),
        "lrmoe_combine": ([L.BF16, 4, 2, 16, 8], 5),
        "lrmoe_combine_backward": ([L.BF16, 4, 2, 16, 8], 6),
    }
    for name, (dims, n) in movers.items():
        f = getattr(lib, name)
        ptrs = [FAKE] * n
        for i, v, code in ((0, 7, DTYPE), (1, -1, SHAPE), (1, 2**31, SHAPE), (2, 0, INVALID),
                           (2, 65, INVALID), (3, 0, SHAPE), (3, 12, ALIGN), (3, 2**20 + 8, SHAPE),
                           (4, -1, SHAPE), (4, 2**31, SHAPE)):
            d = list(dims)
            d[i] = v
            assert f(*d, *ptrs, None) == code, (name, i, v)
        for i in range(n):
            p = list(ptrs)
            p[i] = FAKE + 4
            assert f(*dims, *p, None) == ALIGN, (name, i)
            if name == "lrmoe_combine" and i == 3:   # the residual may be absent
                continue
            p[i] = None
            assert f(*dims, *p, None) == NULL, (name, i)
    f = lib.lrmoe_dispatch_backward
    assert f(L.F32, 3, 4, 2, 16, 8, FAKE, FAKE, FAKE, None) == DTYPE
    assert f(L.F32, L.BF16, 4, 2, 12, 8, FAKE, FAKE, FAKE, None) == ALIGN   # bf16 rows of 12
    assert f(L.F32, L.F32, 4, 2, 12, 8, None, FAKE, FAKE, None) == NULL
    assert f(L.F32, L.F32, 4, 2, 12, 8, FAKE, FAKE, FAKE + 8, None) == ALIGN


def fwd(**kw):
    a = dict(E=3, dtype=L.BF16, P=9, T=9, d_out=16, d_in=8, act=L.ACT_NONE)
    a.update(kw)
    return L.Forward(*[a[k] for k in ("E", "dtype", "P", "T", "d_out", "d_in", "act")])


def fwd_call(fw, **over):
    a = dict(seg=FAKE, row=None, x=FAKE, W=FAKE, bias=None, res=None, y=FAKE, pa=None, pb=None)
    a.update(over)
    return L.lib().lrmoe_grouped_forward(C.byref(fw), *a.values(), None)


BAD_FORWARD = [
    (dict(E=0), INVALID), (dict(E=257), INVALID), (dict(act=5), INVALID), (dict(act=-1), INVALID),
    (dict(dtype=9), DTYPE), (dict(P=-1), SHAPE), (dict(P=2**31), SHAPE), (dict(T=-1), SHAPE),
    (dict(d_out=12), ALIGN), (dict(d_in=12), ALIGN), (dict(d_out=0), SHAPE),
    (dict(d_in=2**20 + 8), SHAPE), (dict(act=L.ACT_SWIGLU, d_out=8), ALIGN),
    (dict(act=L.ACT_SWIGLU, d_out=17), ALIGN), (dict(dtype=L.F32, d_in=6), ALIGN)]


@pytest.mark.parametrize("kw,code", BAD_FORWARD)
def test_grouped_forward_refuses(kw, code):
    assert fwd_call(fwd(**kw)) == code


def test_grouped_forward_pointers():
    for name in ("seg", "x", "W", "y"):
        assert fwd_call(fwd(), **{name: None}) == NULL, name
    for name in ("seg", "row", "x", "W", "bias", "res", "y", "pa", "pb"):
        assert fwd_call(fwd(), **{name: FAKE + 4}) == ALIGN, name
    assert fwd_call(fwd(T=5)) == SHAPE                     # pair rows without a row index
    assert fwd_call(fwd(T=0), row=FAKE) == SHAPE           # an index into no rows
    assert fwd_call(fwd(), pa=FAKE, pb=FAKE) == INVALID    # one pre-activation only
    glu = fwd(act=L.ACT_SWIGLU)
    assert fwd_call(glu, pa=FAKE) == NULL and fwd_call(glu, pb=FAKE) == NULL
    assert L.lib().lrmoe_grouped_forward(None, *[FAKE] * 9, None) == NULL
    # no pair: nothing is read or written, nothing is launched
    empty = fwd(P=0, T=0)
    assert fwd_call(empty, x=None, W=None, y=None) == 0


@pytest.mark.parametrize("kw,code", BAD_FORWARD)
def test_act_backward_refuses(kw, code):
    f = fwd(**kw)
    assert L.lib().lrmoe_act_backward(C.byref(f), f.dtype if f.dtype < 2 else 0, FAKE, FAKE, FAKE,
                                      FAKE, FAKE, None, None, 0, None) == code
    n = C.c_size_t(0)
    assert L.lib().lrmoe_act_backward_workspace(C.byref(f), C.byref(n)) == code


def test_act_backward_pointers_and_workspace():
    f = L.lib().lrmoe_act_backward
    glu = fwd(act=L.ACT_SWIGLU, P=200, T=200)
    n = C.c_size_t(0)
    assert L.lib().lrmoe_act_backward_workspace(C.byref(glu), C.byref(n)) == 0
    assert n.value == (200 // 64 + 3) * 16 * 4   # one row of sums for each run of 64 rows
    ok = [L.BF16] + [FAKE] * 7 + [n.value, None]   # dz type, seg dy a b dz dbias ws
    for i in (1, 2, 3, 4, 5, 7):
        a = list(ok)
        a[i] = None
        assert f(C.byref(glu), *a) == NULL, i
        a[i] = FAKE + 4
        assert f(C.byref(glu), *a) == ALIGN, i
    a = list(ok)
    a[6] = FAKE + 4
    assert f(C.byref(glu), *a) == ALIGN
    a = list(ok)
    a[8] -= 1
    assert f(C.byref(glu), *a) == WORKSPACE
    a = list(ok)
    a[0] = 4
    assert f(C.byref(glu), *a) == DTYPE
    a[0] = L.BF16   # float32 pre-activations do not round to bf16
    assert f(C.byref(fwd(act=L.ACT_SWIGLU, dtype=L.F32)), *a) == DTYPE


def test_binding_refuses_cpu_tensors():
    z = torch.zeros
    i = z((2, 2), dtype=torch.int32)
    for call in (lambda: L.gate_topk(z((2, 4)), 2), lambda: L.route_sort(i, 4),
                 lambda: L.gate_topk_backward(z((2, 4)), i, z((2, 2))),
                 lambda: L.dispatch(z((2, 8)), i), lambda: L.dispatch_backward(z((4, 8)), i),
                 lambda: L.combine(z((4, 8)), i, z((2, 2))),
                 lambda: L.combine_backward(z((2, 8)), z((4, 8)), i, z((2, 2))),
                 lambda: L.grouped_forward(z(3, dtype=torch.int32), z((2, 8)), z((2, 8, 8))),
                 lambda: L.act_backward(z(3, dtype=torch.int32), z((2, 8)))):
        with pytest.raises(ValueError, match="device tensors"):
            call()


# ------------------------------------------------------- the oracle itself

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_oracle_gate_gradient_is_autograd(score, renorm):
    torch.manual_seed(1)
    x = torch.randn(5, 7, dtype=torch.float64)
    ids, w = O.gate(x, 3, score, renorm=renorm, scale=1.7)
    dw = torch.randn(5, 3, dtype=torch.float64)
    xr = x.clone().requires_grad_()
    p = torch.softmax(xr, 1) if score == "softmax" else torch.sigmoid(xr)
    wr = p.gather(1, ids)
    wr = 1.7 * (wr / wr.sum(1, keepdim=True) if renorm else wr)
    assert torch.allclose(wr.detach(), w, atol=1e-12)
    want, = torch.autograd.grad((wr * dw).sum(), xr)
    assert torch.allclose(O.gate_grad(x, ids, dw, score, renorm, 1.7), want, atol=1e-12)


def test_oracle_gate_masks():
    x = torch.tensor([[1.0, -float("inf"), float("nan"), 2.0], [float("nan")] * 4,
                      [float("inf"), 0.0, float("inf"), 0.0]])
    ids, w = O.gate(x, 3, "softmax")
    assert ids.tolist() == [[3, 0, -1], [-1, -1, -1], [0, 2, 1]]
    assert w[1].tolist() == [0, 0, 0] and w[2].tolist() == [0.5, 0.5, 0]


@pytest.mark.parametrize("name", ["none", "relu", "silu", "gelu", "swiglu"])
def test_oracle_act_gradient_is_autograd(name):
    torch.manual_seed(2)
    a = torch.randn(9, 4, dtype=torch.float64, requires_grad=True)
    b = torch.randn(9, 4, dtype=torch.float64, requires_grad=True) if name == "swiglu" else None
    dy = torch.randn(9, 4, dtype=torch.float64)
    y = O.act(name, a, b) * 1.0
    want = torch.cat(torch.autograd.grad((y * dy).sum(), [a] if b is None else [a, b]), 1)
    got = O.act_grad([0, 4, 4, 9], dy, a.detach(), None if b is None else b.detach(), name)
    assert torch.allclose(got["dz"], want, atol=1e-12)
    assert torch.equal(got["dbias"][1], torch.zeros(want.shape[1], dtype=torch.float64))
    assert torch.allclose(got["dbias"][2], want[4:].sum(0), atol=1e-12)


def test_oracle_sort_and_rows():
    ids = torch.tensor([[2, 0], [5, 2], [0, -1]])
    w = torch.arange(6.0).reshape(3, 2)
    s = O.sort(ids, 3, w)
    assert s["counts"].tolist() == [2, 0, 2] and s["seg_offsets"].tolist() == [0, 2, 2, 4]
    assert s["row_index"].tolist() == [0, 2, 0, 1, -1, -1]
    assert s["pos"].tolist() == [[2, 0], [-1, 3], [1, -1]]
    assert s["alpha"].tolist() == [1, 4, 0, 3, 0, 0]
    x = torch.arange(6.0).reshape(3, 2)
    xp = O.dispatch(x, s["pos"], torch.full((5, 2), 9.0))
    assert xp[:4].tolist() == x[[0, 2, 0, 1]].tolist() and xp[4].tolist() == [9, 9]
    y, _ = O.combine(xp, s["pos"], w, residual=x)
    assert torch.equal(y, x.double() * (1 + torch.tensor([[1.0], [3.0], [4.0]]).double()))
