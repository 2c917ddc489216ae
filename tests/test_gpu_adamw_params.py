"""Parameters after an AdamW step on the GPU, with their signs: bfloat16 ones of both
signs and through zero, and those behind element 2^32."""
import pytest
import torch

from oracle import block_oracle as B
from pruned_expert_backward_amd import lrmoe as L

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)


def stochastic_bf16(p, ep, u, got):
    """got is p rounded to bfloat16 away from zero where the chance u reaches the gap, with
    p's sign; p is known to ep."""
    gap = lambda a: torch.exp2((torch.frexp(a)[1] - 8).double())   # noqa: E731
    step = gap(p)
    t = p.abs() / step
    want = torch.sign(p) * (torch.floor(t) + ((t - torch.floor(t) + u) >= 1)) * step
    got = got.cpu().double()
    near = (t + u - torch.round(t + u)).abs() <= ep / step + 2.0 ** -15
    # where p is too near to tell: a neighbour of some p' with |p' - p| <= ep, so that
    # |got - p| <= |got - p'| + |p' - p| <= gap(|p| + ep) + ep; and on p's side of zero unless
    # p is within ep of it.  (Where the update takes nearly all of a parameter of 1e-2, the
    # rest of 1e-7 has gaps of 1e-9 and ep is 2^-24 of 1e-2 and more: 15 gaps.)
    side = (torch.sign(got) == torch.sign(p)) | (p.abs() <= ep) | (got == 0)
    ok = (got == want) | near & ((got - p).abs() <= gap(p.abs() + ep) + ep) & side
    assert bool(ok.all()), f"{int((~ok).sum())} of {ok.numel()}"
    assert float(near.double().mean()) < 0.01


@pytest.mark.parametrize("gdt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bits", [32, 8])
def test_bf16_parameters_keep_their_sign(gdt, bits):
    """Positive and negative parameters, and some that the step takes through zero.

    The update's error as in the test of all lengths: m to 4 u of its terms (u = 2^-24), the
    root to 4.5 u, the reciprocal, quotient and products 11.5 u more, p's own product 4 u."""
    g = torch.Generator().manual_seed(13)
    n, lr, betas, eps, wd, t, seed = 20000, 1e-2, (0.9, 0.95), 1e-8, 0.1, 1, 77
    p = torch.randn(n, generator=g) * torch.exp(torch.randn(n, generator=g))
    p[::3] *= 1e-2                        # as small as the step
    p = p.to(torch.bfloat16)
    d = (torch.randn(n, generator=g) * 0.01).to(gdt)
    q, st = p.cuda(), L.adamw_state(p.cuda(), bits)
    L.adamw_step([q], [d.cuda()], [st], t, lr, betas, eps, wd, seed=seed)
    zero = torch.zeros(n)
    want, m, v = B.adamw(p, d, zero, zero, t, lr, betas, eps, wd)
    assert int((torch.sign(want) != torch.sign(p.double())).sum()) > 100
    assert int((want < 0).sum()) > 1000
    U = 2.0 ** -24
    upd = lr / (1 - betas[0]) / (torch.sqrt(v / (1 - betas[1])) + eps)
    ep = upd * 20 * U * m.abs() + 4 * U * p.double().abs()
    stochastic_bf16(want, ep, B.chance(B.second_dice(B.dice(seed, t, 0, n))), q)


def test_parameters_beyond_32_bits():
    """The parameters behind element 2^32, which have a gradient, and those before."""
    tail, lr, betas, eps, seed = 3000, 1e-2, (0.9, 0.95), 1e-8, 7
    n = 2 ** 32 + tail
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    d = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(14)
    start = torch.randn(tail, generator=g).to(torch.bfloat16)
    p[-tail:] = start.cuda()
    grad = torch.randn(tail, generator=g).to(torch.bfloat16)
    d[-tail:] = grad.cuda()
    st = L.adamw_state(p, bits=8)
    L.adamw_step([p], [d], [st], 1, lr, betas, eps, 0.0, seed=seed)
    zero = torch.zeros(tail)
    want, m, v = B.adamw(start, grad, zero, zero, 1, lr, betas, eps, 0.0)
    U = 2.0 ** -24
    upd = lr / (1 - betas[0]) / (torch.sqrt(v / (1 - betas[1])) + eps)
    ep = upd * 20 * U * m.abs() + 4 * U * start.double().abs()
    # the hash takes the index mod 2^32
    stochastic_bf16(want, ep, B.chance(B.second_dice(B.dice(seed, 1, 0, tail))), p[-tail:])
    assert int(p[:-tail].view(torch.int16).count_nonzero()) == 0
    del p, d, st
    torch.cuda.empty_cache()
