"""What 8-bit AdamW states do over many steps, beside float32 ones: the first moment's
mean is kept, the second moment's is a little high, and elements far below their block's
largest are held at the smallest code.  The recurrence on the CPU by the oracle's
definitions, and the kernel's on the GPU.

The bound on the second moment's mean.  A step rounds root = sqrt(w), w = b2 u + (1 -
b2) g^2, to one of the two codes around it, whose distance d is at most root / 8 while
the code is a normal one (at least 2^-6 of the scale), with E[code] = root.  So
E[code^2] = w + f (1 - f) d^2, f the place between the codes, and
  w <= E[u'] <= w (1 + 1 / 256).
Over steps E[u] = r E[v] with 1 <= r <= (1 - b2) (1 + e) / (1 - b2 (1 + e)), e = 1 / 256:
at b2 = 0.95 at most 1.0846.  A mean of n elements is off by its standard error, taken from
the elements themselves; six of those are allowed."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B

B2 = 0.95
MOST = (1 - B2) * (1 + 1 / 256) / (1 - B2 * (1 + 1 / 256))


def rounded(x, u, root):
    """Values of the codes of x at the chances u."""
    s, _ = B.blocks_of(x)
    a = x.abs() / s
    step = B.e4m3_step(a)
    q = torch.floor(a / step + u) * step
    if root:
        q = torch.where((x > 0) & (q == 0), 2.0 ** -9, q)
    return torch.sign(x) * q * s


def mean_within(d, lo, hi):
    """The mean of d's elements lies between lo and hi, but for six standard errors."""
    d = d.double()
    se = float(d.std()) / d.numel() ** 0.5
    assert lo - 6 * se <= float(d.mean()) <= hi + 6 * se, (float(d.mean()), lo, hi, se)


def compare(m8, v8, m32, v32):
    mean_within(m8 - m32, 0.0, 0.0)
    mean_within(v8 - v32, 0.0, (MOST - 1) * float(v32.mean()))


def test_rounding_keeps_the_mean_and_adds_its_variance():
    """Over all 65536 chances: E[code] = x, E[code^2] = x^2 + f (1 - f) d^2."""
    u = torch.arange(65536, dtype=torch.float64) * 2.0 ** -16
    for x, d in ((13.3, 1.0), (8.0, 1.0), (0.7, 2.0 ** -4), (2.0 ** -7 * 1.3, 2.0 ** -9)):
        top = 448.0
        s, _ = B.blocks_of(torch.tensor([top, x]).double())
        assert float(s[0]) == 1.0
        c = torch.floor(x / d + u) * d
        f = x / d - np.floor(x / d)
        assert float(B.e4m3_step(torch.tensor(x).double())) == d
        assert abs(float(c.mean()) - x) <= d * 2.0 ** -16
        assert abs(float((c * c).mean()) - (x * x + f * (1 - f) * d * d)) <= 40 * d * 2.0 ** -16


def test_recurrence_of_the_moments():
    """100 steps of 8-bit and unrounded states on the same gradients."""
    n, b1 = 128 * 48, 0.9
    g = torch.Generator().manual_seed(11)
    size = torch.exp(torch.randn(n, generator=g, dtype=torch.float64))
    m8 = v8 = m = v = torch.zeros(n, dtype=torch.float64)
    for t in range(1, 101):
        d = torch.randn(n, generator=g, dtype=torch.float64) * size
        dice = B.dice(3, t, 0, n)
        m, v = b1 * m + (1 - b1) * d, B2 * v + (1 - B2) * d * d
        m8 = rounded(b1 * m8 + (1 - b1) * d, B.chance(dice >> 16), False)
        v8 = rounded(torch.sqrt(B2 * v8 + (1 - B2) * d * d), B.chance(dice & 0xFFFF), True) ** 2
    compare(m8 / size, v8 / size ** 2, m / size, v / size ** 2)


def test_recurrence_of_elements_far_below_their_blocks_largest():
    """The largest is 1, so the scale is 2^-8 and the smallest code stands for 2^-17.
    2^-14 is 8 of those: steps of a seventh of the root at most once it has gone down by one,
    so with e = 1 / 196 the mean is 1.11 times the moment at most; a step's noise, of
    relative variance 4 f (1 - f) / 64 <= 1 / 64 in u, adds up to 1 / 64 / (1 - b2^2) = 0.16,
    a standard error of 0.4 / sqrt(63) = 0.05 and six of them 0.3: together below 0.5.
    2^-21 is a sixteenth of the smallest code, which it is held at."""
    n = 128
    size = torch.full((n,), 2.0 ** -14, dtype=torch.float64)
    size[0], size[64:] = 1.0, 2.0 ** -21
    v8 = torch.zeros(n, dtype=torch.float64)
    for t in range(1, 201):
        v8 = rounded(torch.sqrt(B2 * v8 + (1 - B2) * size ** 2),
                     B.chance(B.dice(5, t, 0, n) & 0xFFFF), True) ** 2
    s = float(B.blocks_of(torch.sqrt(v8))[0][0])
    assert bool((v8[64:] == (2.0 ** -9 * s) ** 2).all()) and float(v8[64]) > 4 * 2.0 ** -42
    assert abs(float(v8[1:64].mean()) * 2.0 ** 28 - 1) < 0.5


# ----------------------------------------------------------------------- kernel

gpu = pytest.mark.gpu


def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def values(st):
    return [B.row_values(st[k].cpu().view(1, -1), st[k + "_scale"].cpu().view(1, -1))[0]
            for k in ("m", "root")]


@gpu
@pytest.mark.parametrize("gdt", [torch.float32, torch.bfloat16])
def test_kernel_states_over_many_steps(gdt):
    """100 steps with 8-bit and with float32 states on the same gradients."""
    need_gpu()
    from pruned_expert_backward_amd import lrmoe as L
    n = 128 * 256
    g = torch.Generator().manual_seed(12)
    size = torch.exp(torch.randn(n, generator=g))
    p8, p32 = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    s8, s32 = L.adamw_state(p8, bits=8), L.adamw_state(p32)
    for t in range(1, 101):
        d = (torch.randn(n, generator=g) * size).to(gdt).cuda()
        L.adamw_step([p8, p32], [d, d], [s8, s32], t, 1e-3, (0.9, B2), weight_decay=0.0, seed=5)
    m8, r8 = values(s8)
    z = size.double()
    compare(m8 / z, r8 ** 2 / z ** 2, s32["m"].cpu().double() / z, s32["v"].cpu().double() / z ** 2)
