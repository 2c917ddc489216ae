"""Timing cases of the operators around the expert products of a training step
and of serving: 8-bit block-scaled quantisation and the grouped product that
reads it, the norms before and after a block with its gate and residual, and
the AdamW step over many tensors.

`run` computes one pass, in elementary torch operations (own = False) or
through the library's entry points (own = True).  `exact` gives the same
results in float64."""
import math
import random

import torch

own = False

DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
BLOCK = 128                     # values that share a scale
FP8 = torch.float8_e4m3fn
M32 = 0xFFFFFFFF


# ---------------------------------------------------------------------- cases

def listed():
    return [
        # output-gradient rows of a training microbatch, unrounded, ahead of an 8-bit product
        dict(name="quant-rows-grad", op="quant_rows", T=8191, D=4096, dtype="f32"),
        # one GPU's gate/up weights after an optimizer step, both orders (forward and gradient)
        dict(name="quant-weights", op="quant_weights", E=16, N=1536, K=2048, dtype="bf16",
             transpose=True),
        # expert gate/up product of a decoding step: 32 pairs of 16 tokens, 16 experts
        dict(name="fp8-decode", op="product", P=32, T=16, E=16, K=2048, N=1536, act="swiglu",
             bias=False, residual=False, pre=False, zipf=0.5),
        # a short prompt through the wider model's gate/up product, ragged segments
        dict(name="fp8-prompt", op="product", P=1999, T=501, E=16, K=4096, N=2816, act="swiglu",
             bias=True, residual=False, pre=False, zipf=1.0),
        # one GPU's pairs of a training microbatch, gate/up product, pre-activations saved
        dict(name="fp8-train", op="product", P=32768, T=8192, E=16, K=2048, N=1536, act="swiglu",
             bias=False, residual=False, pre=True, zipf=1.2),
        # its input gradient: rows of the output gradient with the transposed weights
        dict(name="fp8-train-dx", op="product", P=32768, T=32768, E=16, K=1536, N=2048,
             act="none", bias=False, residual=False, pre=False, zipf=1.2),
        # a shared expert: one segment, a product bound by the matrix cores
        dict(name="fp8-shared", op="product", P=8192, T=8192, E=1, K=4096, N=8192, act="none",
             bias=False, residual=True, pre=False, zipf=0.0),
        # the block's end and the next one's norm in a decoding step over 16 sequences
        dict(name="norm-decode", op="norm", T=16, D=2048, dtype="bf16", branch=True,
             branch_norm=True, gate="channel", next=True, scale=1.0),
        # the same in a training microbatch
        dict(name="norm-train", op="norm", T=32768, D=2048, dtype="bf16", branch=True,
             branch_norm=True, gate="channel", next=True, scale=1.0),
        # its gradient, an odd number of tokens, a scaled residual
        dict(name="norm-train-grad", op="norm_grad", T=32767, D=2048, dtype="bf16", branch=True,
             branch_norm=True, gate="channel", next=True, scale=0.7),
        # norm weights, biases and the router of a model: many small tensors
        dict(name="adamw-small", op="adamw", tensors=96, total=400_000, param="f32", grad="f32",
             bits=32, copy=True),
        # one GPU's experts of a layer (16 x 1536 x 2048 and 16 x 2048 x 768), 8-bit states
        dict(name="adamw-experts-8bit", op="adamw", tensors=2, total=75_497_472, param="f32",
             grad="f32", bits=8, copy=True),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quant_rows", "quant_weights", "product", "product", "product", "norm",
                     "norm_grad", "adamw", "adamw"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "quant_rows":
        D = 16 * _spread(rng, 2, 512)
        return dict(op=op, T=min(_spread(rng, 1, 32768), 32768 * 2048 // D), D=D, dtype=dtype)
    if op == "quant_weights":
        N, K = 16 * _spread(rng, 4, 256), 16 * _spread(rng, 4, 256)
        return dict(op=op, E=max(1, min(_spread(rng, 1, 32), 16 * 1536 * 2048 // (N * K))), N=N,
                    K=K, dtype=dtype, transpose=rng.random() < 0.6)
    if op == "product":
        act = rng.choice(["none", "relu", "silu", "gelu", "swiglu", "swiglu"])
        K, F = 16 * _spread(rng, 4, 256), 8 * _spread(rng, 8, 256)
        N = 2 * F if act == "swiglu" else F
        P = min(_spread(rng, 1, 32768), max(1, 32768 * 2048 * 1536 // (K * N)))
        E = max(1, min(_spread(rng, 1, 32), 16 * 4096 * 2816 // (K * N)))
        return dict(op=op, P=P, T=max(1, P // rng.choice([1, 2, 8])), E=E, K=K, N=N, act=act,
                    bias=rng.random() < 0.5, residual=rng.random() < 0.5,
                    pre=rng.random() < 0.5, zipf=round(rng.uniform(0, 1.6), 2))
    if op == "adamw":
        param = rng.choice(["f32", "f32", "bf16"])
        return dict(op=op, tensors=_spread(rng, 1, 200), total=_spread(rng, 1000, 40_000_000),
                    param=param, grad=rng.choice(["f32", "bf16"]), bits=rng.choice([32, 8]),
                    copy=param == "f32" and rng.random() < 0.5)
    D = 8 * _spread(rng, 8, 1024)
    branch = rng.random() < 0.8
    gate = rng.choice(["none", "channel", "token"]) if branch else "none"
    return dict(op=op, T=min(_spread(rng, 1, 32768), 32768 * 2048 // D), D=D, dtype=dtype,
                branch=branch, branch_norm=branch and rng.random() < 0.7, gate=gate,
                next=not branch or rng.random() < 0.8,
                scale=round(rng.uniform(0.5, 1.5), 2) if branch and rng.random() < 0.5 else 1.0)


# --------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, dt, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dt)


def _segments(g, P, E, zipf):
    """Device segment offsets [E + 1] of P pairs over E experts, Zipf-shared."""
    w = torch.arange(1, E + 1, device=DEV).double() ** -zipf
    w = w[torch.randperm(E, generator=g, device=DEV)]
    ends = (P * torch.cumsum(w, 0) / w.sum()).round().long()
    ends[-1] = P
    off = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), ends])
    return off.to(torch.int32)


def _sizes(case):
    """Sizes of the tensors of one step: the expert projections of a layer (two to
    one), or shares that range over a factor of a thousand."""
    n, total = case["tensors"], case["total"]
    if n == 2:
        return [total * 2 // 3, total - total * 2 // 3]
    rng = random.Random(total)
    w = [math.exp(rng.uniform(0, math.log(1000))) for _ in range(n)]
    return [max(1, int(total * v / sum(w))) for v in w]


STATE = {32: ("m", "v"), 8: ("m", "m_scale", "root", "root_scale")}


def _buffers(case, sizes):
    """(name, sizes, type) of what a step changes."""
    blocks = [(n + BLOCK - 1) // BLOCK for n in sizes]
    out = [("params", sizes, DT[case["param"]])]
    if case["copy"]:
        out.append(("copies", sizes, torch.bfloat16))
    if case["bits"] == 32:
        return out + [("m", sizes, torch.float32), ("v", sizes, torch.float32)]
    return out + [("m", sizes, FP8), ("m_scale", blocks, torch.uint8), ("root", sizes, FP8),
                  ("root_scale", blocks, torch.uint8)]


def _place(n):
    return (n + 15) // 16 * 16


def _views(flat, lengths):
    return [x[:n] for n, x in zip(lengths, torch.split(flat, [_place(n) for n in lengths]))]


def prepare(case, seed):
    c, g, op = case, _gen(seed), case["op"]
    s = dict(case=c)
    if op == "quant_rows":   # gradients: rows of different size, some all zero
        size = torch.exp(_normal(g, (c["T"], 1), torch.float32, 2.0)) * 1e-4
        live = torch.rand((c["T"], 1), generator=g, device=DEV) < 0.97
        s["x"] = (_normal(g, (c["T"], c["D"]), torch.float32) * size * live).to(DT[c["dtype"]])
        return s
    if op == "quant_weights":
        s["W"] = _normal(g, (c["E"], c["N"], c["K"]), DT[c["dtype"]], 0.02)
        return s
    if op == "product":
        P, E, K, N = c["P"], c["E"], c["K"], c["N"]
        F = N // 2 if c["act"] == "swiglu" else N
        s["seg"] = _segments(g, P, E, c["zipf"])
        s["x"] = _normal(g, (c["T"], K), torch.bfloat16)
        # the weights in 8 bits, laid out once
        q, byte = _quantize_weights(_normal(g, (E, N, K), torch.bfloat16, 0.02))
        s["W"] = dict(q=q, scale=byte)
        s["row"] = (torch.randint(0, c["T"], (P,), generator=g, device=DEV, dtype=torch.int32)
                    if c["T"] != P else None)
        s["bias"] = _normal(g, (E, N), torch.bfloat16, 0.1) if c["bias"] else None
        s["res"] = _normal(g, (P, F), torch.bfloat16) if c["residual"] else None
        return s
    if op == "adamw":
        s["step"], s["seed"] = 1000 + seed % 1000, seed & M32
        s["clip"] = 0.5 + 0.5 * torch.rand(1, generator=g, device=DEV)   # of a gradient norm
        sizes = _sizes(c)
        # the tensors of a kind are views of one buffer, each at a 16-byte border
        s["flat"] = {k: torch.zeros(sum(_place(n) for n in lengths), dtype=dt, device=DEV)
                     for k, lengths, dt in _buffers(c, sizes)}
        v = {k: _views(s["flat"][k], lengths) for k, lengths, _ in _buffers(c, sizes)}
        s["params"], s["grads"] = v["params"], []
        s["copies"] = v.get("copies")
        s["states"] = [dict(zip(STATE[c["bits"]], x))
                       for x in zip(*(v[name] for name in STATE[c["bits"]]))]
        for n, p, st in zip(sizes, s["params"], s["states"]):
            p.copy_(_normal(g, (n,), torch.float32, 0.02))
            spread = torch.exp(_normal(g, (n,), torch.float32))     # of the gradients' size
            grad = _normal(g, (n,), torch.float32) * spread * 1e-4
            grad[: n // 16] = 0                                     # an expert without pairs
            s["grads"].append(grad.to(DT[c["grad"]]))
            m = _normal(g, (n,), torch.float32) * spread * 3e-5
            root = spread * (torch.rand((n,), generator=g, device=DEV) + 0.5) * 1e-4
            new = (m, root * root) if c["bits"] == 32 else _quantize_flat(m) + _quantize_flat(root)
            for t, x in zip(st.values(), new):
                t.copy_(x)
        return s
    dt, T, D = DT[c["dtype"]], c["T"], c["D"]
    s["x"] = _normal(g, (T, D), dt, 2.0)
    s["y"] = _normal(g, (T, D), dt) if c["branch"] else None
    s["w"] = (1 + _normal(g, (D,), torch.float32, 0.1)).to(dt) if c["next"] else None
    s["wb"] = (1 + _normal(g, (D,), torch.float32, 0.1)).to(dt) if c["branch_norm"] else None
    s["gate"] = None
    if c["gate"] == "channel":
        s["gate"] = (0.5 + _normal(g, (D,), torch.float32, 0.1)).to(dt)
    elif c["gate"] == "token":
        s["gate"] = torch.rand((T, 1), generator=g, device=DEV)
    if op == "norm_grad":
        # what the forward pass has stored
        s["s"] = _norm(s)["s"] if c["branch"] else s["x"]
        s["ds"] = _normal(g, (T, D), dt) if c["branch"] else None
        s["dh"] = _normal(g, (T, D), dt) if c["next"] else None
    return s


# ----------------------------------------------------------- the library's calls

def _own(s):
    from pruned_expert_backward_amd import lrmoe as L
    c, op = s["case"], s["case"]["op"]
    if op == "quant_rows":
        return L.quantize_rows(s["x"])
    if op == "quant_weights":
        return L.quantize_weights(s["W"], transpose=c["transpose"])
    if op == "product":
        act = {"none": L.ACT_NONE, "relu": L.ACT_RELU, "silu": L.ACT_SILU, "gelu": L.ACT_GELU,
               "swiglu": L.ACT_SWIGLU}[c["act"]]
        return L.grouped_forward_quantized(s["seg"], L.quantize_rows(s["x"]), s["W"],
                                           row_index=s["row"], bias=s["bias"],
                                           residual=s["res"], act=act, save_pre=c["pre"])
    if op == "norm":
        return L.residual_norm(s["x"], y=s["y"], weight=s["w"], branch_weight=s["wb"],
                               gate=s["gate"], scale=c["scale"])
    if op == "norm_grad":
        return L.residual_norm_backward(s["s"], ds=s["ds"], dh=s["dh"], y=s["y"], weight=s["w"],
                                        branch_weight=s["wb"], gate=s["gate"], scale=c["scale"])
    L.adamw_step(s["params"], s["grads"], s["states"], step=s["step"], lr=LR, betas=BETAS,
                 eps=EPS, weight_decay=DECAY, copies=s["copies"], grad_scale=s["clip"],
                 seed=s["seed"])
    return s["flat"]


LR, BETAS, EPS, DECAY, NORM_EPS = 3e-4, (0.9, 0.95), 1e-8, 0.1, 1e-6


# ------------------------------------------------------------------ plain forms

def _scale_byte(top):
    """Exponent byte of a block whose largest magnitude is `top`: the smallest power
    of two with top / 2^e at most 448, as e + 127; 127 for a block of zeros."""
    bits = top.view(torch.int32)
    byte = (bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).to(torch.int32)
    return torch.where(top > 0, byte.clamp_min(1), 127)


def _pow2(byte):
    return (byte.to(torch.int32) << 23).view(torch.float32)


def _top(x, dim):
    a = x.abs()
    return torch.where(torch.isfinite(a), a, 0.0).amax(dim)


def _pad(n, m):
    return (n + m - 1) // m * m


def _quantize_rows(x):
    """q [T, D] and the scales of 1 x 128 blocks, rows of scales padded to four."""
    T, D = x.shape
    f = torch.nn.functional.pad(x.float(), (0, _pad(D, BLOCK) - D)).view(T, -1, BLOCK)
    byte = _scale_byte(_top(f, 2))
    q = (f * _pow2(254 - byte)[..., None]).view(T, -1)[:, :D].to(FP8)
    byte = torch.nn.functional.pad(byte, (0, _pad(byte.shape[1], 4) - byte.shape[1]), value=127)
    return q.contiguous(), byte.to(torch.uint8)


def _quantize_weights(W):
    """q [E, N, K] and the scales of 128 x 128 blocks, rows of scales padded to four."""
    E, N, K = W.shape
    n, k = _pad(N, BLOCK), _pad(K, BLOCK)
    f = torch.nn.functional.pad(W.float(), (0, k - K, 0, n - N))
    f = f.view(E, n // BLOCK, BLOCK, k // BLOCK, BLOCK)
    byte = _scale_byte(_top(f, (2, 4)))
    q = (f * _pow2(254 - byte)[:, :, None, :, None]).view(E, n, k)[:, :N, :K].to(FP8)
    byte = torch.nn.functional.pad(byte, (0, _pad(k // BLOCK, 4) - k // BLOCK), value=127)
    return q.contiguous(), byte.to(torch.uint8)


def _quantize_flat(x):
    """A flat tensor's e4m3 values and the scale byte of each run of 128."""
    n = x.numel()
    q, byte = _quantize_rows(torch.nn.functional.pad(x, (0, _pad(n, BLOCK) - n)).view(-1, BLOCK))
    return q.view(-1)[:n].clone(), byte[:, 0].contiguous()


def _flat_values(q, byte):
    return q.float() * _pow2(byte).repeat_interleave(BLOCK)[: q.numel()]


def _quant_weights(s):
    q, byte = _quantize_weights(s["W"])
    out = dict(q=q, scale=byte)
    if s["case"]["transpose"]:
        out["qt"], out["scale_t"] = _quantize_weights(s["W"].transpose(1, 2))
    return out


def _quant_rows(s):
    return dict(zip(("q", "scale"), _quantize_rows(s["x"])))


def _wide(q, byte, rows):
    """Values of q, whose rows' scale bytes are byte[rows]."""
    scale = _pow2(byte).repeat_interleave(BLOCK, dim=-1)[..., : q.shape[-1]]
    return q.float() * (scale if rows is None else scale[..., rows, :])


def _act(a, b, act):
    if act == "relu":
        return torch.clamp_min(a, 0)
    if act == "gelu":
        return 0.5 * a * (1 + torch.erf(a * math.sqrt(0.5)))
    if act == "silu":
        return a / (1 + torch.exp(-a))
    return a / (1 + torch.exp(-a)) * b if act == "swiglu" else a


def _product(s):
    """The segments cut into blocks of R rows: one batched product over the
    blocks, each with its expert's weights."""
    c = s["case"]
    P, E, F = c["P"], c["E"], c["N"] // 2
    x = _wide(*_quantize_rows(s["x"]), None)
    W = _wide(s["W"]["q"], s["W"]["scale"], torch.arange(c["N"], device=x.device) // BLOCK)
    R = 1 << max(0, min(8, (max(1, P // E)).bit_length()))
    seg = s["seg"].long()
    first = torch.cat([seg.new_zeros(1), torch.cumsum((seg[1:] - seg[:-1] + R - 1) // R, 0)])
    block = torch.arange(P // R + E, device=seg.device)
    e = (torch.searchsorted(first, block, right=True) - 1).clamp_max(E - 1)
    u = (seg[e] + (block - first[e]) * R)[:, None] + torch.arange(R, device=seg.device)
    live = (u < seg[e + 1][:, None]) & (block < first[E])[:, None]
    row = u.clamp_max(P - 1)
    z = torch.bmm(x[row if s["row"] is None else s["row"].long()[row]], W[e].transpose(1, 2))
    z = z[live]                        # rows in pair order
    if s["bias"] is not None:
        z = z + s["bias"].float()[torch.searchsorted(seg, torch.arange(P, device=seg.device),
                                                     right=True) - 1]
    a, b = (z[:, :F], z[:, F:]) if c["act"] == "swiglu" else (z, None)
    y = _act(a, b, c["act"])
    if s["res"] is not None:
        y = y + s["res"].float()
    out = dict(y=y.to(torch.bfloat16))
    if c["pre"]:
        out["pre_a"] = a.to(torch.bfloat16).contiguous()
        if b is not None:
            out["pre_b"] = b.to(torch.bfloat16).contiguous()
    return out


def _rstd(x):
    return 1 / torch.sqrt((x * x).mean(1, keepdim=True) + NORM_EPS)


def _norm(s):
    c, out = s["case"], {}
    x = s["x"].float()
    if s["y"] is not None:
        n = s["y"].float()
        if s["wb"] is not None:
            n = n * _rstd(n) * s["wb"].float()
        x = c["scale"] * x + (n if s["gate"] is None else s["gate"].float() * n)
        out["s"] = x.to(s["x"].dtype)
    if s["w"] is not None:
        out["h"] = (x * _rstd(x) * s["w"].float()).to(s["x"].dtype)
    return out


def _norm_grad(s):
    c, out = s["case"], {}
    dt, D = s["s"].dtype, s["case"]["D"]
    d = 0 if s["ds"] is None else s["ds"].float()
    if s["w"] is not None:
        dh, x = s["dh"].float(), s["s"].float()
        r = _rstd(x)
        n = x * r
        out["dweight"] = (dh * n).sum(0, dtype=torch.float64).float()
        dn = dh * s["w"].float()
        d = d + r * (dn - n * (dn * n).mean(1, keepdim=True))
    out["dx"] = (c["scale"] * d).to(dt)
    if s["y"] is None:
        return out
    n, w = s["y"].float(), None
    if s["wb"] is not None:
        r, w = _rstd(n), s["wb"].float()
        n = n * r
    dn = d if s["gate"] is None else s["gate"].float() * d
    if s["gate"] is not None:
        dg = d * n if w is None else d * n * w
        out["dgate"] = (dg.sum(1, keepdim=True) if c["gate"] == "token"
                        else dg.sum(0, dtype=torch.float64).float())
    if w is not None:
        out["dbranch_weight"] = (dn * n).sum(0, dtype=torch.float64).float()
        dn = dn * w
        dn = r * (dn - n * (dn * n).mean(1, keepdim=True))
    out["dy"] = dn.to(dt)
    return out


def _mix(a):
    """A 32-bit number's bits well mixed (an int or a tensor of int64)."""
    a = a ^ (a >> 16)
    a = (a * 0x6A09E667) & M32
    a = a ^ (a >> 15)
    a = (a * 0xBB67AE85) & M32
    return a ^ (a >> 16)


def _dice(s, k, n):
    """The 32 random bits of each element of tensor k in this step."""
    key = _mix((s["seed"] + s["step"] * 0x9E3779B9) & M32)
    key = _mix((key + (k + 1) * 0x3C6EF373) & M32)
    return _mix((torch.arange(n, device=DEV) + key) & M32)


def _chance(bits):
    return bits.float() * 2.0 ** -16


def _requantize(x, chance):
    """e4m3 blocks of a flat tensor, rounded up as often as the value lies beyond
    the lower neighbour."""
    n = x.numel()
    f = torch.nn.functional.pad(x, (0, _pad(n, BLOCK) - n)).view(-1, BLOCK)
    byte = _scale_byte(_top(f, 1))
    f = (f * _pow2(254 - byte)[:, None]).view(-1)[:n]
    lead = ((f.view(torch.int32) >> 23) & 255).clamp(121, 135)   # 2^-6 .. 2^8
    steps = torch.floor(f.abs() * _pow2(257 - lead) + chance)
    q = torch.copysign(steps * _pow2(lead - 3), f).to(FP8)
    return q, byte.to(torch.uint8)


def _adamw(s):
    c, (b1, b2) = s["case"], BETAS
    fix1, fix2 = 1 - b1 ** s["step"], 1 / math.sqrt(1 - b2 ** s["step"])
    for k, (p, g, st) in enumerate(zip(s["params"], s["grads"], s["states"])):
        n, g = p.numel(), g.float() * s["clip"]
        wide = c["bits"] == 32
        m = st["m"] if wide else _flat_values(st["m"], st["m_scale"])
        if wide:
            v = st["v"]
        else:
            root = _flat_values(st["root"], st["root_scale"])
            v = root * root
        m = m * b1 + g * (1 - b1)
        v = v * b2 + (g * g) * (1 - b2)
        root = torch.sqrt(v)
        new = p.float() * (1 - LR * DECAY) - (m / (root * fix2 + EPS)) * (LR / fix1)
        dice = None if wide and c["param"] == "f32" else _dice(s, k, n)
        if c["param"] == "f32":
            p.copy_(new)
            if c["copy"]:
                s["copies"][k].copy_(new.to(torch.bfloat16))
        else:
            bits = new.view(torch.int32).long() & M32
            up = _mix((dice + 0xA54FF53B) & M32) >> 16
            p.copy_((((bits + up) & 0xFFFF0000).to(torch.int32)).view(torch.float32))
        if wide:
            st["m"].copy_(m)
            st["v"].copy_(v)
        else:
            mq, mb = _requantize(m, _chance(dice >> 16))
            rq, rb = _requantize(root, _chance(dice & 0xFFFF))
            # a second moment that is not zero does not become zero
            rq = torch.where((root > 0) & (rq.float() == 0), 2.0 ** -9, rq.float()).to(FP8)
            for name, t in (("m", mq), ("m_scale", mb), ("root", rq), ("root_scale", rb)):
                st[name].copy_(t)
    return s["flat"]


PLAIN = dict(quant_rows=_quant_rows, quant_weights=_quant_weights, product=_product, norm=_norm,
             norm_grad=_norm_grad, adamw=_adamw)


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------------- work

def work(case):
    c, op = case, case["op"]
    b = 4 if c.get("dtype") == "f32" else 2
    if op == "quant_rows":
        n = c["T"] * c["D"]
        return dict(bytes=n * (b + 1) + n // BLOCK, flops=2 * n)
    if op == "quant_weights":
        n = c["E"] * c["N"] * c["K"]
        return dict(bytes=n * (b + (2 if c["transpose"] else 1)), flops=2 * n)
    if op == "product":
        F = c["N"] // 2 if c["act"] == "swiglu" else c["N"]
        read = 2 * min(c["T"], c["P"]) * c["K"] + min(c["E"], c["P"]) * c["N"] * c["K"]
        write = c["P"] * (F * (2 if c["residual"] else 1) + (c["N"] if c["pre"] else 0))
        return dict(bytes=read + 2 * write, flops=2 * c["P"] * c["N"] * c["K"])
    if op == "adamw":
        n = sum(_sizes(c))
        each = (8 if c["param"] == "f32" else 4) + (4 if c["grad"] == "f32" else 2)
        each += (16 if c["bits"] == 32 else 4) + (2 if c["copy"] else 0)
        return dict(bytes=n * each, flops=16 * n)
    n = c["T"] * c["D"]
    if op == "norm":
        return dict(bytes=n * b * (1 + 2 * c["branch"] + c["next"]), flops=10 * n)
    return dict(bytes=n * b * (2 * c["branch"] + 2 * c["next"] + 1 + c["branch"]), flops=20 * n)


# ------------------------------------------------- the same results in 64 bits

def _exact_blocks(top):
    """2^e of blocks whose largest magnitude is `top`, from the definition."""
    e = torch.ceil(torch.log2(top.clamp_min(1e-300) / 448))
    e = torch.where(top > 448 * torch.exp2(e), e + 1, e)
    e = torch.where(top <= 448 * torch.exp2(e - 1), e - 1, e)
    return torch.where(top > 0, torch.exp2(e), 1.0)


def _exact_e4m3(x):
    """The nearest e4m3 value, ties to even (x within +-448)."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 4).clamp_min(-9).double())
    return torch.round(x / step) * step


def _exact_rows(x):
    """(value of q, scale) of 1 x 128 blocks in float64."""
    parts = [x[:, i:i + BLOCK].double() for i in range(0, x.shape[1], BLOCK)]
    scales = [_exact_blocks(p.abs().amax(1, keepdim=True)) for p in parts]
    return (torch.cat([_exact_e4m3(p / z) for p, z in zip(parts, scales)], 1),
            torch.cat([z.expand_as(p) for p, z in zip(parts, scales)], 1))


def _exact_quant_weights(s):
    W = s["W"].double()
    q = torch.empty_like(W)
    for i in range(0, W.shape[1], BLOCK):
        for j in range(0, W.shape[2], BLOCK):
            part = W[:, i:i + BLOCK, j:j + BLOCK]
            q[:, i:i + BLOCK, j:j + BLOCK] = _exact_e4m3(
                part / _exact_blocks(part.abs().amax((1, 2), keepdim=True)))
    out = dict(q=q, scale=None)
    if s["case"]["transpose"]:
        out.update(qt=q.transpose(1, 2).contiguous(), scale_t=None)
    return out


def _exact_product(s):
    c, fn = s["case"], torch.nn.functional
    F, seg = c["N"] // 2, s["seg"].tolist()
    q, scale = _exact_rows(s["x"])
    x = q * scale
    byte = s["W"]["scale"].double()

    def product(e):
        at = slice(seg[e], seg[e + 1])
        rows = x[at] if s["row"] is None else x[s["row"][at].long()]
        w = torch.exp2(byte[e] - 127).repeat_interleave(BLOCK, 0)[: c["N"]]
        w = w.repeat_interleave(BLOCK, 1)[:, : c["K"]] * s["W"]["q"][e].double()
        z = rows @ w.t()
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


def _exact_rms(x, w):
    return x / torch.sqrt(x.square().mean(1, keepdim=True) + NORM_EPS) * w


def _exact_stream(s, x, y, wb, gate):
    n = y if wb is None else _exact_rms(y, wb)
    if gate is not None:
        n = n * gate
    return s["case"]["scale"] * x + n


def _exact_norm(s):
    wide = {k: None if s[k] is None else s[k].double() for k in ("x", "y", "w", "wb", "gate")}
    x, out = wide["x"], {}
    if s["y"] is not None:
        x = out["s"] = _exact_stream(s, x, wide["y"], wide["wb"], wide["gate"])
    if s["w"] is not None:
        out["h"] = _exact_rms(x, wide["w"])
    return out


def _exact_norm_grad(s):
    """Gradients of <s, ds> + <h, dh> at the stored s: through h first, then through
    the sum, whose branch is y's."""
    out = {}
    d = 0 if s["ds"] is None else s["ds"].double()
    if s["w"] is not None:
        x, w = (s[k].double().requires_grad_() for k in ("s", "w"))
        gx, out["dweight"] = torch.autograd.grad((_exact_rms(x, w) * s["dh"].double()).sum(), [x, w])
        d = d + gx
    if s["y"] is None:
        out["dx"] = s["case"]["scale"] * d
        return out
    x = torch.zeros_like(d, requires_grad=True)
    ins = {"dx": x, "dy": s["y"].double().requires_grad_()}
    if s["wb"] is not None:
        ins["dbranch_weight"] = s["wb"].double().requires_grad_()
    if s["gate"] is not None:
        ins["dgate"] = s["gate"].double().requires_grad_()
    t = _exact_stream(s, x, ins["dy"], ins.get("dbranch_weight"), ins.get("dgate"))
    out.update(zip(ins, torch.autograd.grad((t * d).sum(), list(ins.values()))))
    return out


def _exact_state(x, chance):
    """(values, None) of the 8-bit blocks, rounded up where `chance` reaches the gap."""
    n = x.numel()
    f = torch.nn.functional.pad(x, (0, -n % BLOCK)).view(-1, BLOCK)
    f = (f / _exact_blocks(f.abs().amax(1, keepdim=True))).view(-1)[:n]
    _, e = torch.frexp(f)
    step = torch.exp2((e - 4).clamp_min(-9).double())
    return torch.sign(f) * torch.floor(f.abs() / step + chance) * step


def _exact_adamw(s):
    c, t = s["case"], s["step"]
    b1, b2 = BETAS
    sizes = _sizes(c)
    flat = {k: None if k.endswith("scale") else
            torch.zeros(sum(_place(n) for n in lengths), dtype=torch.float64, device=DEV)
            for k, lengths, _ in _buffers(c, sizes)}
    out = {k: _views(x, sizes) for k, x in flat.items() if x is not None}
    for k, n in enumerate(sizes):
        p, st = s["params"][k].double(), s["states"][k]
        g = s["grads"][k].double() * s["clip"].double()
        if c["bits"] == 32:
            m, v = st["m"].double(), st["v"].double()
        else:
            m, root = (st[a].double() * torch.exp2(st[a + "_scale"].double() - 127)
                       .repeat_interleave(BLOCK)[:n] for a in ("m", "root"))
            v = root ** 2
        m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g ** 2
        mh, vh = m / (1 - b1 ** t), v / (1 - b2 ** t)
        p = p - LR * (DECAY * p + mh / (torch.sqrt(vh) + EPS))
        if c["copy"]:
            out["copies"][k].copy_(p)
        dice = _dice(s, k, n)
        if c["param"] == "bf16":
            _, e = torch.frexp(p)
            step = torch.exp2((e - 8).double())
            up = (_mix((dice + 0xA54FF53B) & M32) >> 16).double() * 2.0 ** -16
            p = torch.sign(p) * torch.floor(p.abs() / step + up) * step
        out["params"][k].copy_(p)
        if c["bits"] == 32:
            out["m"][k].copy_(m)
            out["v"][k].copy_(v)
            continue
        root = torch.sqrt(v)
        r8 = _exact_state(root, (dice & 0xFFFF).double() * 2.0 ** -16)
        out["root"][k].copy_(torch.where((root > 0) & (r8 == 0), 2.0 ** -9, r8))
        out["m"][k].copy_(_exact_state(m, (dice >> 16).double() * 2.0 ** -16))
    return flat


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant_rows":
        return dict(q=_exact_rows(s["x"])[0], scale=None)
    return dict(quant_weights=_exact_quant_weights, product=_exact_product, norm=_exact_norm,
                norm_grad=_exact_norm_grad, adamw=_exact_adamw)[op](s)
