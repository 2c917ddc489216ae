"""CPU oracle of the forward side in float64 (test infrastructure only): the
router gate, the expert sort, dispatch and combine, the grouped product with
its epilogue, and their gradients, written from their definitions with plain
loops over rows, slots and experts.

Inputs are torch CPU tensors of any type; results are float64 (or whole
numbers).  Functions that bound a result's rounding return the sum of absolute
terms beside it where their caller needs one."""
import math

import torch

NEG = -math.inf


def _clean(x):
    """Logits as the gate reads them: NaN masks, +inf is the largest float32."""
    x = x.double()
    x = torch.where(torch.isnan(x), torch.full_like(x, NEG), x)
    return x.clamp(max=torch.finfo(torch.float32).max)


def gate(logits, K, score, select_bias=None, renorm=True, scale=1.0):
    """(ids [T, K], weights [T, K]): a loop over rows and slots."""
    x = _clean(logits)
    T, E = x.shape
    ids = torch.full((T, K), -1, dtype=torch.int64)
    w = torch.zeros((T, K), dtype=torch.float64)
    for t in range(T):
        row = x[t].tolist()
        key = list(row)
        if select_bias is not None:
            key = [1 / (1 + math.exp(-v)) + float(b) if v > -700 else float(b)
                   for v, b in zip(row, select_bias.double().tolist())]
        key = [NEG if v == NEG or k != k else k for v, k in zip(row, key)]
        order = sorted((e for e in range(E) if key[e] > NEG), key=lambda e: (-key[e], e))[:K]
        for k, e in enumerate(order):
            ids[t, k] = e
        if order:
            w[t, :len(order)] = scale * _weights(x[t], order, score, renorm)
    return ids, w


def _weights(row, chosen, score, renorm):
    v = row[chosen]
    if score == "softmax":
        return torch.softmax(v, 0) if renorm else torch.softmax(row, 0)[chosen]
    if renorm:   # ratios of sigmoids, without their underflow
        return torch.softmax(torch.nn.functional.logsigmoid(v), 0)
    return torch.sigmoid(v)


def gate_grad(logits, ids, dw, score, renorm=True, scale=1.0):
    """dlogits by the chain rule of the weights, slot by slot."""
    x = _clean(logits)
    T, E = x.shape
    dx = torch.zeros((T, E), dtype=torch.float64)
    for t in range(T):
        on = [k for k in range(ids.shape[1]) if 0 <= int(ids[t, k]) < E]
        sel = [int(ids[t, k]) for k in on]
        if not on:
            continue
        d, v = dw[t, on].double(), x[t, sel]
        if score == "softmax" and not renorm:
            p = torch.softmax(x[t], 0)
            dx[t] -= scale * p * (p[sel] * d).sum()
            g = scale * p[sel] * d
        elif score == "softmax":
            p = torch.softmax(v, 0)
            g = scale * p * (d - (p * d).sum())
        elif renorm:
            r = torch.softmax(torch.nn.functional.logsigmoid(v), 0)
            g = scale * r * (d - (r * d).sum()) * torch.sigmoid(-v)
        else:
            g = scale * d * torch.sigmoid(v) * torch.sigmoid(-v)
        for e, one in zip(sel, g):
            dx[t, e] += one
    return dx


def sort(ids, E, weights=None):
    T, K = ids.shape
    flat = ids.reshape(-1).tolist()
    n = T * K
    order = [i for e in range(E) for i in range(n) if flat[i] == e] if E <= 8 else \
        sorted((i for i in range(n) if 0 <= flat[i] < E), key=lambda i: (flat[i], i))
    counts = [0] * E
    for i in order:
        counts[flat[i]] += 1
    seg = [0]
    for c in counts:
        seg.append(seg[-1] + c)
    row = torch.full((n,), -1, dtype=torch.int64)
    pos = torch.full((n,), -1, dtype=torch.int64)
    alpha = torch.zeros(n, dtype=torch.float32)
    for p, i in enumerate(order):
        row[p] = i // K
        pos[i] = p
        if weights is not None:
            alpha[p] = weights.reshape(-1)[i]
    return dict(counts=torch.tensor(counts), seg_offsets=torch.tensor(seg), row_index=row,
                pos=pos.reshape(T, K), alpha=alpha)


def _places(pos, P):
    T, K = pos.shape
    return [(t, k, int(pos[t, k])) for t in range(T) for k in range(K) if 0 <= int(pos[t, k]) < P]


def dispatch(x, pos, xp):
    out = xp.clone()
    for t, k, p in _places(pos, xp.shape[0]):
        out[p] = x[t]
    return out


def combine(yp, pos, weights=None, residual=None):
    """(y, sum of absolute terms), float64."""
    T, D = pos.shape[0], yp.shape[1]
    y = torch.zeros((T, D), dtype=torch.float64) if residual is None else residual.double().clone()
    mag = y.abs()
    for t, k, p in _places(pos, yp.shape[0]):
        v = yp[p].double() * (1.0 if weights is None else weights[t, k].double())
        y[t] += v
        mag[t] += v.abs()
    return y, mag


def combine_grad(dy, yp, pos, weights, dyp0):
    """(dyp over dyp0, dweights, sum of |products| behind each dweight)."""
    dyp = dyp0.double().clone()
    dw = torch.zeros(pos.shape, dtype=torch.float64)
    mag = torch.zeros(pos.shape, dtype=torch.float64)
    for t, k, p in _places(pos, yp.shape[0]):
        prod = dy[t].double() * yp[p].double()
        dyp[p] = weights[t, k].double() * dy[t].double()
        dw[t, k], mag[t, k] = prod.sum(), prod.abs().sum()
    return dyp, dw, mag


def act(name, a, b=None):
    if name == "relu":
        return a.clamp(min=0)
    if name == "silu":
        return a * torch.sigmoid(a)
    if name == "gelu":
        return 0.5 * a * (1 + torch.erf(a / math.sqrt(2)))
    if name == "swiglu":
        return a * torch.sigmoid(a) * b
    return a


def act_slope(name, a):
    if name == "relu":
        return (a > 0).double()
    if name in ("silu", "swiglu"):
        s = torch.sigmoid(a)
        return s * (1 + a * (1 - s))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(a / math.sqrt(2))) \
            + a * torch.exp(-0.5 * a * a) / math.sqrt(2 * math.pi)
    return torch.ones_like(a)


def linear(seg, x, W, row_index=None, bias=None, residual=None, name="none"):
    """dict(y, z, mag): z before the activation, mag = sum |x w| + |bias|, for
    the rows of the segments (others are zero)."""
    E, d_out, d_in = W.shape
    P = x.shape[0] if row_index is None else row_index.numel()
    z = torch.zeros((P, d_out), dtype=torch.float64)
    mag = torch.zeros((P, d_out), dtype=torch.float64)
    for e in range(E):
        rows = [u if row_index is None else int(row_index[u])
                for u in range(int(seg[e]), int(seg[e + 1]))]
        if not rows:
            continue
        v = torch.stack([x[r].double() if 0 <= r < x.shape[0]
                         else torch.zeros(d_in, dtype=torch.float64) for r in rows])
        at = slice(int(seg[e]), int(seg[e + 1]))
        z[at] = v @ W[e].double().t()
        mag[at] = v.abs() @ W[e].double().abs().t()
        if bias is not None:
            z[at] += bias[e].double()
            mag[at] += bias[e].double().abs()
    if name == "swiglu":
        F = d_out // 2
        y = act(name, z[:, :F], z[:, F:])
    else:
        y = act(name, z)
    if residual is not None:
        y = y + residual.double()
    return dict(y=y, z=z, mag=mag)


def act_grad(seg, dy, a, b, name):
    """dict(dz, dbias, mag): mag = sum |dz| behind each dbias."""
    g, a = dy.double(), a.double()
    if name == "swiglu":
        dz = torch.cat([g * b.double() * act_slope(name, a), g * a * torch.sigmoid(a)], 1)
    else:
        dz = g * act_slope(name, a)
    E = len(seg) - 1
    db = torch.stack([dz[int(seg[e]):int(seg[e + 1])].sum(0) for e in range(E)])
    mag = torch.stack([dz[int(seg[e]):int(seg[e + 1])].abs().sum(0) for e in range(E)])
    return dict(dz=dz, dbias=db, mag=mag)
