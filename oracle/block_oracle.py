"""CPU oracle in float64 (test infrastructure only) of the operators around the
expert products: 8-bit blocks, the norms around a block with gate and residual,
and the AdamW step, written from their definitions.

Inputs are torch CPU tensors of any type; results are float64 or whole numbers."""
import math

import numpy as np
import torch

BLOCK = 128


def scale_byte(top: float) -> int:
    """e + 127 of the smallest power of two with top <= 448 * 2^e; 127 for zero."""
    if top == 0:
        return 127
    m, x = math.frexp(top)          # top = m 2^x, 1/2 <= m < 1; 448 = 7/8 2^9
    return max(1, x - 9 + (1 if m > 0.875 else 0) + 127)


def scale_row(d: int) -> int:
    blocks = (d + BLOCK - 1) // BLOCK
    return (blocks + 3) // 4 * 4


def e4m3_step(a):
    """Distance of the e4m3 values around |a|."""
    _, x = torch.frexp(a.abs())
    return torch.exp2((x - 4).clamp_min(-9).double())


def e4m3(a):
    """Nearest e4m3 value, ties to even (|a| at most 448); NaN stays."""
    step = e4m3_step(torch.nan_to_num(a))
    return torch.round(a / step) * step


def _block(x):
    """(values of the codes, byte) of one block; infinity and NaN become NaN."""
    x = x.double()
    fine = torch.isfinite(x)
    top = float(x[fine].abs().max()) if bool(fine.any()) else 0.0
    byte = scale_byte(top)
    v = e4m3(torch.where(fine, x, 0.0) * 2.0 ** (127 - byte))
    return torch.where(fine, v, math.nan), byte


def quantize_rows(x):
    """(values of q [T, D] float64, scale bytes [T, S])."""
    T, D = x.shape
    q = torch.zeros((T, D), dtype=torch.float64)
    byte = torch.full((T, scale_row(D)), 127, dtype=torch.uint8)
    for t in range(T):
        for b in range(0, D, BLOCK):
            q[t, b:b + BLOCK], byte[t, b // BLOCK] = _block(x[t, b:b + BLOCK])
    return q, byte


def quantize_weights(W):
    E, N, K = W.shape
    q = torch.zeros((E, N, K), dtype=torch.float64)
    byte = torch.full((E, (N + BLOCK - 1) // BLOCK, scale_row(K)), 127, dtype=torch.uint8)
    for e in range(E):
        for n in range(0, N, BLOCK):
            for k in range(0, K, BLOCK):
                at = (e, slice(n, n + BLOCK), slice(k, k + BLOCK))
                q[at], byte[e, n // BLOCK, k // BLOCK] = _block(W[at])
    return q, byte


def row_values(q, byte):
    """What rows in 8 bits stand for."""
    s = torch.exp2(byte.double() - 127).repeat_interleave(BLOCK, -1)[..., : q.shape[-1]]
    return q.double() * s


def weight_values(q, byte):
    N = q.shape[1]
    return row_values(q, byte.repeat_interleave(BLOCK, 1)[:, :N])


# ------------------------------------------------------------------- norms

def rms_inv(v, eps):
    return 1 / torch.sqrt(v.square().mean(1, keepdim=True) + eps)


def residual_norm(x, y=None, weight=None, branch_weight=None, gate=None, scale=1.0, eps=1e-6):
    """(s, h or None) in float64; gate [D] or [T, 1]."""
    s = x.double()
    if y is not None:
        b = y.double()
        if branch_weight is not None:
            b = b * rms_inv(b, eps) * branch_weight.double()
        s = scale * s + (b if gate is None else gate.double() * b)
    h = None if weight is None else s * rms_inv(s, eps) * weight.double()
    return s, h


def residual_norm_grad(s, ds=None, dh=None, y=None, weight=None, branch_weight=None, gate=None,
                       scale=1.0, eps=1e-6):
    """Gradients by the formulas, each with the size of the terms that it sums up
    (name + "_mag"): what bounds a float32 computation's error."""
    out, s = {}, s.double()
    d = torch.zeros_like(s) if ds is None else ds.double()
    dm = d.abs()
    if weight is not None:
        r, dh, w = rms_inv(s, eps), dh.double(), weight.double()
        n, t = s * rms_inv(s, eps), dh * w
        out["dweight"], out["dweight_mag"] = (dh * n).sum(0), (dh * n).abs().sum(0)
        d = d + r * (t - n * (t * n).mean(1, keepdim=True))
        dm = dm + r * (t.abs() + n.abs() * (t * n).abs().mean(1, keepdim=True))
    out["dx"], out["dx_mag"] = scale * d, abs(scale) * dm
    if y is None:
        return out
    z, r, w = y.double(), 1.0, 1.0
    if branch_weight is not None:
        r, w = rms_inv(z, eps), branch_weight.double()
        z = z * r
    g = 1.0 if gate is None else gate.double()
    if gate is not None:
        t, m = d * z * w, dm * (z * w).abs()
        dim = (1, True) if gate.dim() == 2 else (0, False)
        out["dgate"], out["dgate_mag"] = t.sum(*dim), m.sum(*dim)
    dg, dgm = d * g, dm * (g.abs() if gate is not None else 1.0)
    if branch_weight is None:
        out["dy"], out["dy_mag"] = dg, dgm
        return out
    out["dbranch_weight"] = (dg * z).sum(0)
    out["dbranch_weight_mag"] = (dgm * z.abs()).sum(0)
    t, m = dg * w, dgm * w.abs()
    out["dy"] = r * (t - z * (t * z).mean(1, keepdim=True))
    out["dy_mag"] = r * (m + z.abs() * (m * z.abs()).mean(1, keepdim=True))
    return out


# ------------------------------------------------------------------- AdamW

def mix(a):
    a = np.asarray(a, dtype=np.uint64)
    m = np.uint64(0xFFFFFFFF)
    a = a ^ (a >> np.uint64(16))
    a = (a * np.uint64(0x6A09E667)) & m
    a = a ^ (a >> np.uint64(15))
    a = (a * np.uint64(0xBB67AE85)) & m
    return a ^ (a >> np.uint64(16))


def dice(seed, step, k, n, first=0):
    """Random bits of elements first .. first + n - 1 of tensor k, as uint64 arrays."""
    m = 0xFFFFFFFF
    key = int(mix((seed + step * 0x9E3779B9) & m))
    key = int(mix((key + (k + 1) * 0x3C6EF373) & m))
    i = (np.arange(first, first + n, dtype=np.uint64) + np.uint64(key)) & np.uint64(m)
    return mix(i)


def second_dice(r):
    return mix((r + np.uint64(0xA54FF53B)) & np.uint64(0xFFFFFFFF)) >> np.uint64(16)


def chance(bits):
    return torch.from_numpy(bits.astype(np.float64)) * 2.0 ** -16


def blocks_of(x):
    """(scale of each element, bytes) of a flat tensor's runs of 128."""
    byte = [scale_byte(float(x[i:i + BLOCK].abs().max())) for i in range(0, x.numel(), BLOCK)]
    byte = torch.tensor(byte, dtype=torch.uint8)
    return torch.exp2(byte.double() - 127).repeat_interleave(BLOCK)[: x.numel()], byte


def adamw(p, g, m, v, step, lr, betas, eps, weight_decay, grad_scale=1.0):
    """(p, m, v) after a step, unrounded."""
    b1, b2 = betas
    p, g = p.double(), g.double() * grad_scale
    m = b1 * m.double() + (1 - b1) * g
    v = b2 * v.double() + (1 - b2) * g * g
    mh, vh = m / (1 - b1 ** step), v / (1 - b2 ** step)
    return p - lr * weight_decay * p - lr * mh / (torch.sqrt(vh) + eps), m, v
