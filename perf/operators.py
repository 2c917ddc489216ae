"""Timing cases of the expert layer's forward operators: the router's top-k
gate, the expert sort with its row dispatch, the weighted combine, and the
grouped expert product with its epilogue, each with its gradient.

`run` computes one pass, in elementary torch operations (own = False) or
through the library's entry points (own = True).  `exact` gives the same
results in float64."""
import math

import torch

own = False

DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------- cases

def listed():
    return [
        # the router of one decoding step over 16 sequences
        dict(name="gate-decode", op="gate", T=16, E=128, K=8, dtype="f32", score="softmax",
             renorm=True, bias=False, scale=1.0),
        # a training microbatch (4 x 8192 tokens), sigmoid router with a selection bias
        dict(name="gate-train", op="gate", T=32768, E=128, K=8, dtype="f32", score="sigmoid",
             renorm=True, bias=True, scale=1.5),
        # the same microbatch's router gradient, bf16 logits
        dict(name="gate-train-grad", op="gate_grad", T=32767, E=128, K=8, dtype="bf16",
             score="softmax", renorm=True, bias=False, scale=1.0),
        # one GPU's 16 of 128 experts, decoding 64 sequences: most pairs are elsewhere
        dict(name="sort-decode", op="sort", T=64, E=16, E_all=128, K=8, D=0, dtype="bf16"),
        # a training microbatch sorted over all experts, rows dispatched
        dict(name="sort-dispatch-train", op="sort", T=32768, E=128, E_all=128, K=8, D=2048,
             dtype="bf16"),
        # the experts' outputs back to the tokens of that microbatch, onto the residual stream
        dict(name="combine-train", op="combine", T=32768, E=128, E_all=128, K=8, D=2048,
             dtype="bf16", residual=True),
        # gradient of the combine, wider rows, an odd number of tokens
        dict(name="combine-grad", op="combine_grad", T=8191, E=16, E_all=16, K=8, D=4096,
             dtype="bf16"),
        # expert gate/up product of a decoding step: 32 pairs over one GPU's 16 experts
        dict(name="linear-decode", op="linear", P=32, T=16, E=16, d_in=2048, d_out=1536,
             dtype="bf16", act="swiglu", bias=False, residual=False, pre=False, zipf=0.5),
        # a short prompt through the wider model's gate/up product, ragged segments
        dict(name="linear-prompt", op="linear", P=1999, T=501, E=16, d_in=4096, d_out=2816,
             dtype="bf16", act="swiglu", bias=True, residual=False, pre=False, zipf=1.0),
        # one GPU's pairs of a training microbatch, gate/up product, pre-activations saved
        dict(name="linear-train", op="linear", P=32768, T=8192, E=16, d_in=2048, d_out=1536,
             dtype="bf16", act="swiglu", bias=False, residual=False, pre=True, zipf=1.2),
        # float32 storage: a down projection with bias and residual in the epilogue
        dict(name="linear-f32", op="linear", P=4097, T=4097, E=8, d_in=768, d_out=2048,
             dtype="f32", act="none", bias=True, residual=True, pre=False, zipf=1.2),
        # gradient of the gate/up epilogue of the training microbatch
        dict(name="linear-grad", op="act_grad", P=32768, E=16, d_out=1536, dtype="bf16",
             act="swiglu", zipf=1.2),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gate", "gate_grad", "sort", "combine", "combine_grad", "dispatch_grad",
                     "linear", "linear", "linear", "act_grad"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("gate", "gate_grad"):
        E = _spread(rng, 2, 256)
        K = _spread(rng, 1, min(E, 8))
        score = rng.choice(["softmax", "sigmoid"])
        # one renormalised expert has weight 1 and no gradient: nothing to compare
        return dict(op=op, T=_spread(rng, 1, 32768), E=E, K=K, dtype=dtype, score=score,
                    renorm=K > 1 and rng.random() < 0.7,
                    bias=score == "sigmoid" and op == "gate" and rng.random() < 0.5,
                    scale=round(rng.uniform(0.5, 2.5), 2))
    if op in ("linear", "act_grad"):
        E = _spread(rng, 1, 32)
        act = rng.choice(["none", "relu", "silu", "gelu", "swiglu", "swiglu"])
        d_in, F = 8 * _spread(rng, 8, 512), 8 * _spread(rng, 8, 256)
        d_out = 2 * F if act == "swiglu" else F
        most = 32768 * 2048 * 1536 // (1 if dtype == "bf16" else 8)
        P = min(_spread(rng, 1, 32768), max(1, most // (d_in * d_out)))
        E = max(1, min(E, 16 * 4096 * 2816 // (d_in * d_out)))
        if op == "act_grad":
            return dict(op=op, P=P, E=E, d_out=d_out, dtype=dtype, act=act,
                        zipf=round(rng.uniform(0, 1.6), 2))
        return dict(op=op, P=P, T=max(1, P // rng.choice([1, 2, 8])), E=E, d_in=d_in, d_out=d_out,
                    dtype=dtype, act=act, bias=rng.random() < 0.5, residual=rng.random() < 0.5,
                    pre=rng.random() < 0.5, zipf=round(rng.uniform(0, 1.6), 2))
    E_all = _spread(rng, 2, 256)
    K = _spread(rng, 1, min(E_all, 8))
    D = 8 * _spread(rng, 4, 512)
    T = min(_spread(rng, 1, 32768), max(1, 32768 * 8 * 2048 // (2 * K * D)))
    if op == "sort" and rng.random() < 0.5:
        return dict(op=op, T=_spread(rng, 1, 81920), E=max(1, E_all // rng.choice([1, 2, 8])),
                    E_all=E_all, K=K, D=0, dtype=dtype)
    c = dict(op=op, T=T, E=E_all, E_all=E_all, K=K, D=D, dtype=dtype)
    if op == "combine":   # one GPU's experts only: some pairs are elsewhere
        c.update(E=max(1, E_all // rng.choice([1, 2])), residual=rng.random() < 0.5)
    return c


# --------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, dt, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dt)


def _routing(g, T, E_all, K):
    """Expert ids [T, K] of T tokens, distinct in a row, with a skewed popularity."""
    skew = -0.5 * torch.log1p(torch.randperm(E_all, generator=g, device=DEV).float())
    noisy = skew - torch.log(-torch.log(torch.rand((T, E_all), generator=g, device=DEV)
                                        .clamp(1e-9, 1 - 1e-6)))
    return torch.topk(noisy, K, dim=1).indices.to(torch.int32)


def _positions(ids, E):
    """pos [T, K] in expert order (-1: not among experts 0..E-1) and the number of pairs."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.sort(key, stable=True).indices
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device=DEV)
    return torch.where(key < E, pos, -1).to(torch.int32).reshape(ids.shape), int((key < E).sum())


def _segments(g, P, E, zipf):
    """Device segment offsets [E + 1] of P pairs over E experts, Zipf-shared."""
    w = torch.arange(1, E + 1, device=DEV).double() ** -zipf
    w = w[torch.randperm(E, generator=g, device=DEV)]
    ends = (P * torch.cumsum(w, 0) / w.sum()).round().long()
    ends[-1] = P
    off = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), ends])
    return off.to(torch.int32)


def prepare(case, seed):
    c, g, op, dt = case, _gen(seed), case["op"], DT[case["dtype"]]
    s = dict(case=c)
    if op in ("gate", "gate_grad"):
        s["logits"] = _normal(g, (c["T"], c["E"]), dt, 1.5)
        s["bias"] = _normal(g, (c["E"],), torch.float32, 0.1) if c["bias"] else None
        if op == "gate_grad":
            s["ids"] = torch.topk(s["logits"].float(), c["K"], dim=1).indices.to(torch.int32)
            s["dw"] = _normal(g, (c["T"], c["K"]), torch.float32)
        return s
    if op in ("linear", "act_grad"):
        P, E, F = c["P"], c["E"], c["d_out"] // (2 if c["act"] == "swiglu" else 1)
        s["seg"] = _segments(g, P, E, c["zipf"])
        if op == "act_grad":
            s["dy"] = _normal(g, (P, F), dt)
            s["a"] = _normal(g, (P, F), dt)
            s["b"] = _normal(g, (P, F), dt) if c["act"] == "swiglu" else None
            return s
        s["x"] = _normal(g, (c["T"], c["d_in"]), dt)
        s["W"] = _normal(g, (E, c["d_out"], c["d_in"]), dt, 0.02)
        s["row"] = (torch.randint(0, c["T"], (P,), generator=g, device=DEV, dtype=torch.int32)
                    if c["T"] != P else None)
        s["bias"] = _normal(g, (E, c["d_out"]), dt, 0.1) if c["bias"] else None
        s["res"] = _normal(g, (P, F), dt) if c["residual"] else None
        return s
    s["ids"] = _routing(g, c["T"], c["E_all"], c["K"])
    s["w"] = torch.softmax(_normal(g, (c["T"], c["K"]), torch.float32), dim=1)
    if op == "sort":
        s["x"] = _normal(g, (c["T"], c["D"]), dt) if c["D"] else None
        return s
    s["pos"], P = _positions(s["ids"], c["E"])
    s["rows"] = _normal(g, (P, c["D"]), dt)
    if op == "combine":
        s["res"] = _normal(g, (c["T"], c["D"]), dt) if c["residual"] else None
    if op == "combine_grad":
        s["dy"] = _normal(g, (c["T"], c["D"]), dt)
    return s


# ----------------------------------------------------------- the library's calls

def _own(s):
    from pruned_expert_backward_amd import lrmoe as L
    c, op = s["case"], s["case"]["op"]
    if op in ("gate", "gate_grad"):
        score = L.GATE_SOFTMAX if c["score"] == "softmax" else L.GATE_SIGMOID
        if op == "gate":
            return L.gate_topk(s["logits"], c["K"], score=score, select_bias=s["bias"],
                               renorm=c["renorm"], scale=c["scale"])
        return L.gate_topk_backward(s["logits"], s["ids"], s["dw"], score=score,
                                    renorm=c["renorm"], scale=c["scale"])
    if op == "sort":
        out = L.route_sort(s["ids"], c["E"], weights=s["w"])
        if s["x"] is not None:
            out["xp"] = L.dispatch(s["x"], out["pos"])
        return out
    if op == "combine":
        return L.combine(s["rows"], s["pos"], s["w"], residual=s["res"])
    if op == "combine_grad":
        return L.combine_backward(s["dy"], s["rows"], s["pos"], s["w"])
    if op == "dispatch_grad":
        return L.dispatch_backward(s["rows"], s["pos"])
    act = {"none": L.ACT_NONE, "relu": L.ACT_RELU, "silu": L.ACT_SILU, "gelu": L.ACT_GELU,
           "swiglu": L.ACT_SWIGLU}[c["act"]]
    if op == "linear":
        return L.grouped_forward(s["seg"], s["x"], s["W"], row_index=s["row"], bias=s["bias"],
                                 residual=s["res"], act=act, save_pre=c["pre"])
    return L.act_backward(s["seg"], s["dy"], s["a"], s["b"], act=act)


# ------------------------------------------------------------------ plain forms

def _gate(s):
    c, x = s["case"], s["logits"].float()
    x = torch.where(torch.isnan(x), -math.inf, x)
    if c["score"] == "softmax":
        key = x
    else:   # 64 bits: the choice between two near values is a whole number
        key = 1 / (1 + torch.exp(-x.double()))
        if s["bias"] is not None:
            key = key + s["bias"].double()
        key = torch.where(x == -math.inf, -math.inf, key)
    top, ids = torch.sort(key, dim=1, descending=True, stable=True)
    top, ids = top[:, :c["K"]], ids[:, :c["K"]]
    ok = top > -math.inf
    v = torch.where(ok, torch.gather(x, 1, ids), -math.inf)
    if c["score"] == "softmax":
        m = x.amax(1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
        w = torch.exp(v - m)
        den = w.sum(1, keepdim=True) if c["renorm"] else torch.exp(x - m).sum(1, keepdim=True)
        w = w / den
    else:
        w = 1 / (1 + torch.exp(-v))
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True)
    w = torch.where(ok, c["scale"] * w, 0.0)
    return dict(ids=torch.where(ok, ids, -1).to(torch.int32), weights=w)


def _gate_grad(s):
    c, x = s["case"], s["logits"].float()
    ids, dw, scale = s["ids"].long(), s["dw"], c["scale"]
    v = torch.gather(x, 1, ids)
    dx = torch.zeros_like(x)
    if c["score"] == "softmax" and not c["renorm"]:
        p = torch.exp(x - x.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
        dot = (torch.gather(p, 1, ids) * dw).sum(1, keepdim=True)
        dx = scale * p * (dx.scatter_add(1, ids, dw) - dot)
    elif c["score"] == "softmax":
        p = torch.exp(v - v.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
        dx = dx.scatter_add(1, ids, scale * p * (dw - (p * dw).sum(1, keepdim=True)))
    else:
        sig, co = 1 / (1 + torch.exp(-v)), 1 / (1 + torch.exp(v))
        if c["renorm"]:
            r = sig / sig.sum(1, keepdim=True)
            d = scale * r * (dw - (r * dw).sum(1, keepdim=True)) * co
        else:
            d = scale * dw * sig * co
        dx = dx.scatter_add(1, ids, d)
    return dx.to(s["logits"].dtype)


def _sort(s):
    c = s["case"]
    E, K = c["E"], c["K"]
    flat = s["ids"].reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    key, order = torch.sort(key, stable=True)
    seg = torch.searchsorted(key, torch.arange(E + 1, device=key.device))
    here = key < E
    pos = torch.empty_like(order)
    pos[order] = torch.where(here, torch.arange(order.numel(), device=key.device), -1)
    out = dict(counts=seg[1:] - seg[:-1], seg_offsets=seg.to(torch.int32),
               row_index=torch.where(here, order // K, -1).to(torch.int32),
               pos=pos.to(torch.int32).reshape(s["ids"].shape),
               alpha=torch.where(here, s["w"].reshape(-1)[order], 0.0))
    if s["x"] is not None:
        out["xp"] = s["x"][order // K]
    return out


def _rows_of(s, rows):
    """rows[pos] as [T, K, D] float32, zero where a slot is not routed."""
    pos = s["pos"].long()
    return torch.where((pos >= 0)[..., None], rows[pos.clamp_min(0)].float(), 0.0)


def _combine(s):
    rows = s["rows"] if s["rows"].shape[0] else s["rows"].new_zeros((1, s["case"]["D"]))
    y = (s["w"][..., None] * _rows_of(s, rows)).sum(1)
    if s["res"] is not None:
        y = y + s["res"].float()
    return y.to(s["rows"].dtype)


def _combine_grad(s):
    dy = s["dy"].float()
    dw = (_rows_of(s, s["rows"]) * dy[:, None]).sum(2)
    at = s["pos"].reshape(-1).long()
    dyp = torch.empty_like(s["rows"])
    dyp[at] = (s["w"][..., None] * dy[:, None]).reshape(-1, dy.shape[1]).to(dyp.dtype)
    return dict(dyp=dyp, dweights=dw)


def _dispatch_grad(s):
    return _rows_of(s, s["rows"]).sum(1).to(s["rows"].dtype)


def _act(a, b, act):
    if act == "relu":
        return torch.clamp_min(a, 0)
    if act == "gelu":
        return 0.5 * a * (1 + torch.erf(a * math.sqrt(0.5)))
    if act == "silu":
        return a / (1 + torch.exp(-a))
    return a / (1 + torch.exp(-a)) * b if act == "swiglu" else a


def _linear(s):
    """The segments cut into blocks of R rows: one batched product over the
    blocks, each with its expert's weights."""
    c = s["case"]
    P, E, F = c["P"], c["E"], c["d_out"] // 2
    R = 1 << max(0, min(8, (max(1, P // E)).bit_length()))
    seg = s["seg"].long()
    first = torch.cat([seg.new_zeros(1), torch.cumsum((seg[1:] - seg[:-1] + R - 1) // R, 0)])
    block = torch.arange(P // R + E, device=seg.device)
    e = (torch.searchsorted(first, block, right=True) - 1).clamp_max(E - 1)
    u = (seg[e] + (block - first[e]) * R)[:, None] + torch.arange(R, device=seg.device)
    live = (u < seg[e + 1][:, None]) & (block < first[E])[:, None]
    row = u.clamp_max(P - 1)
    x = s["x"][row if s["row"] is None else s["row"].long()[row]].float()
    z = torch.bmm(x, s["W"].float()[e].transpose(1, 2))
    z = z[live]                        # rows in pair order
    if s["bias"] is not None:
        z = z + s["bias"].float()[torch.searchsorted(seg, torch.arange(P, device=seg.device),
                                                     right=True) - 1]
    a, b = (z[:, :F], z[:, F:]) if c["act"] == "swiglu" else (z, None)
    y = _act(a, b, c["act"])
    if s["res"] is not None:
        y = y + s["res"].float()
    dt = s["x"].dtype
    out = dict(y=y.to(dt))
    if c["pre"]:
        out["pre_a"] = a.to(dt).contiguous()
        if b is not None:
            out["pre_b"] = b.to(dt).contiguous()
    return out


def _act_grad(s):
    act, a, dy = s["case"]["act"], s["a"].float(), s["dy"].float()
    sig = 1 / (1 + torch.exp(-a))
    dsilu = sig * (1 + a * (1 - sig))
    if act == "swiglu":
        dz = torch.cat([dy * s["b"].float() * dsilu, dy * a * sig], dim=1)
    elif act == "silu":
        dz = dy * dsilu
    elif act == "gelu":
        dz = dy * (0.5 * (1 + torch.erf(a * math.sqrt(0.5)))
                   + a * torch.exp(-0.5 * a * a) * (1 / math.sqrt(2 * math.pi)))
    else:
        dz = torch.where(a > 0, dy, 0.0) if act == "relu" else dy
    # sums over whole segments in 64 bits, as a product with the segments' 0/1 rows
    seg, u = s["seg"][:, None], torch.arange(dz.shape[0], device=dz.device)
    member = ((u >= seg[:-1]) & (u < seg[1:])).double()
    return dict(dz=dz.to(s["dy"].dtype), dbias=torch.mm(member, dz.double()).float())


PLAIN = dict(gate=_gate, gate_grad=_gate_grad, sort=_sort, combine=_combine,
             combine_grad=_combine_grad, dispatch_grad=_dispatch_grad, linear=_linear,
             act_grad=_act_grad)


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------------- work

def work(case):
    c, b = case, 4 if case["dtype"] == "f32" else 2
    op = c["op"]
    if op == "gate":
        return dict(bytes=c["T"] * (c["E"] * b + c["K"] * 8), flops=c["T"] * c["E"] * 4)
    if op == "gate_grad":
        whole = c["E"] if c["score"] == "softmax" and not c["renorm"] else c["K"]
        return dict(bytes=c["T"] * ((c["E"] + whole) * b + c["K"] * 8), flops=c["T"] * whole * 8)
    if op == "act_grad":
        n = 5 if c["act"] == "swiglu" else 3 if c["act"] != "none" else 2
        F = c["d_out"] // 2 if c["act"] == "swiglu" else c["d_out"]
        return dict(bytes=n * c["P"] * F * b + c["E"] * c["d_out"] * 4, flops=c["P"] * F * 12)
    if op == "linear":
        F = c["d_out"] // 2 if c["act"] == "swiglu" else c["d_out"]
        read = min(c["T"], c["P"]) * c["d_in"] + min(c["E"], c["P"]) * c["d_out"] * c["d_in"]
        write = c["P"] * (F * (2 if c["residual"] else 1) + (c["d_out"] if c["pre"] else 0))
        return dict(bytes=(read + write) * b, flops=2 * c["P"] * c["d_out"] * c["d_in"])
    n = c["T"] * c["K"]
    if op == "sort":
        return dict(bytes=n * 20 + c["E"] * 12 + (n + c["T"]) * c["D"] * b, flops=n)
    here = n * c["E"] // c["E_all"]
    if op == "combine":
        return dict(bytes=(here + c["T"] * (2 if c["residual"] else 1)) * c["D"] * b + n * 8,
                    flops=2 * here * c["D"])
    if op == "combine_grad":
        return dict(bytes=(2 * here + c["T"]) * c["D"] * b + n * 12, flops=3 * here * c["D"])
    return dict(bytes=(here + c["T"]) * c["D"] * b + n * 4, flops=here * c["D"])


# ------------------------------------------------- the same results in 64 bits

def _exact_gate(s):
    c, x = s["case"], s["logits"].double()
    key = x if c["score"] == "softmax" else torch.sigmoid(x)
    if s["bias"] is not None:
        key = key + s["bias"].double()
    ids = torch.argsort(-key, dim=1, stable=True)[:, :c["K"]]
    prob = torch.softmax(x, 1) if c["score"] == "softmax" else torch.sigmoid(x)
    w = torch.gather(prob, 1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return dict(ids=ids.to(torch.int32), weights=c["scale"] * w)


def _exact_gate_grad(s):
    c, ids = s["case"], s["ids"].long()
    x = s["logits"].double().requires_grad_()
    prob = torch.softmax(x, 1) if c["score"] == "softmax" else torch.sigmoid(x)
    w = torch.gather(prob, 1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return torch.autograd.grad((c["scale"] * w * s["dw"].double()).sum(), x)[0]


def _exact_rows(s, fn):
    """fn over slices of tokens, its rows of [T, K, D] in float64, put together."""
    def part(at):
        pos = s["pos"][at].long()
        rows = s["rows"].new_zeros((*pos.shape, s["case"]["D"]), dtype=torch.float64)
        rows[pos >= 0] = s["rows"][pos[pos >= 0]].double()
        return fn(at, rows)
    return torch.cat([part(slice(lo, lo + 2048)) for lo in range(0, s["case"]["T"], 2048)])


def _exact_linear(s):
    c = s["case"]
    F, seg, fn = c["d_out"] // 2, s["seg"].tolist(), torch.nn.functional

    def product(e):
        at = slice(seg[e], seg[e + 1])
        x = s["x"][at] if s["row"] is None else s["x"][s["row"][at].long()]
        z = x.double() @ s["W"][e].double().t()
        return z if s["bias"] is None else z + s["bias"][e].double()
    z = torch.cat([product(e) for e in range(c["E"]) if seg[e + 1] > seg[e]])
    if c["act"] == "swiglu":
        y = fn.silu(z[:, :F]) * z[:, F:]
    else:
        y = {"none": lambda v: v, "relu": torch.relu, "silu": fn.silu, "gelu": fn.gelu}[c["act"]](z)
    out = dict(y=y if s["res"] is None else y + s["res"].double())
    if c["pre"]:
        out["pre_a"] = z[:, :F] if c["act"] == "swiglu" else z
        if c["act"] == "swiglu":
            out["pre_b"] = z[:, F:]
    return out


def _exact_act_grad(s):
    act, F = s["case"]["act"], s["a"].shape[1]
    a = s["a"].double().requires_grad_()
    b = s["b"].double().requires_grad_() if act == "swiglu" else None
    fn = torch.nn.functional
    y = {"none": lambda: a * 1, "relu": lambda: torch.relu(a), "silu": lambda: fn.silu(a),
         "gelu": lambda: fn.gelu(a), "swiglu": lambda: fn.silu(a) * b}[act]()
    dz = torch.cat(torch.autograd.grad((y * s["dy"].double()).sum(),
                                       [a] if b is None else [a, b]), dim=1)
    seg = s["seg"].tolist()
    sums = [dz[seg[e]:seg[e + 1]].sum(0) for e in range(len(seg) - 1)]
    return dict(dz=dz, dbias=torch.stack(sums))


def exact(case, seed):
    s = prepare(case, seed)
    op, w = case["op"], None
    if op == "gate":
        return _exact_gate(s)
    if op == "gate_grad":
        return _exact_gate_grad(s)
    if op == "linear":
        return _exact_linear(s)
    if op == "act_grad":
        return _exact_act_grad(s)
    if op == "sort":   # whole numbers and copies: nothing is computed
        return None
    if op == "dispatch_grad":
        return _exact_rows(s, lambda at, rows: rows.sum(1))
    w = s["w"].double()
    if op == "combine":
        def one(at, rows):
            y = (w[at, :, None] * rows).sum(1)
            return y if s["res"] is None else y + s["res"][at].double()
        return _exact_rows(s, one)
    dy, pos = s["dy"].double(), s["pos"].long()
    token = torch.empty(pos.numel(), dtype=torch.long, device=dy.device)
    token[pos.reshape(-1)] = torch.arange(pos.numel(), device=dy.device)
    dyp = w.reshape(-1)[token, None] * dy[token // case["K"]]
    return dict(dyp=dyp, dweights=_exact_rows(s, lambda at, rows: (rows * dy[at, None]).sum(2)))
