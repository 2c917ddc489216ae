"""The Python examples of the README, run in the order in which they stand there:
on the CPU through the binding's checks, on the GPU with their results."""
import os
import re

import pytest
import torch

from oracle import block_oracle as B
from pruned_expert_backward_amd import lrmoe as L

if not os.path.exists(L.LIB_PATH):
    pytest.skip("liblrmoe.so not built (run __graft_entry__.build())", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16, F32 = torch.bfloat16, torch.float32
T, E, K, D, F = 24, 4, 8, 128, 64


def examples():
    """The code blocks from the forward side's on."""
    with open(os.path.join(ROOT, "README.md"), encoding="utf-8") as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    at = next(i for i, b in enumerate(blocks) if "gate_topk(" in b)
    assert len(blocks) >= at + 2
    return blocks[at:]


def inputs(dev):
    """What the examples take as given, by their names.  Eight slots need eight experts:
    the first E of them are this rank's."""
    g = torch.Generator().manual_seed(3)
    r = lambda *s, dt=BF16, std=1.0: (torch.randn(s, generator=g) * std).to(dt).to(dev)  # noqa: E731
    P = T * K
    return dict(lrmoe=L, torch=torch, E=2 * E, logits=r(T, 2 * E, dt=F32), x=r(T, D),
                W_gate_up=r(2 * E, 2 * F, D, std=0.1), W_down=r(2 * E, D, F, std=0.1),
                dx_pairs=r(P, D), dy=r(T, D), dz=r(P, 2 * F), ds=r(T, D), dh_next=r(T, D),
                w_in=1 + r(D, std=0.1), w_out=1 + r(D, std=0.1), w_next=1 + r(D, std=0.1),
                branch_gate=r(D), W=r(E, F, D, dt=F32), dW=r(E, F, D, dt=F32),
                W_bf16=torch.zeros(E, F, D, dtype=BF16, device=dev))


def run(names):
    for block in examples():
        exec(compile(block, "README.md", "exec"), names)
    return names


def test_examples_pass_the_bindings_checks(monkeypatch):
    monkeypatch.setattr(L, "_device", lambda t: t.device)
    calls = []
    monkeypatch.setattr(L, "_call", lambda fn, dev, *args: calls.append(fn))
    run(inputs("cpu"))
    assert calls[-1] == "lrmoe_adamw_step" and "lrmoe_residual_norm_backward" in calls


@pytest.mark.gpu
def test_examples_results():
    """The stream behind the block is x + gate * rms(MoE output) * weight, x once, and
    its norm and gradients are those of the formulas.  The roundings that differ from
    float64 here are the stored y's, s's and h's own: half a bfloat16 step of each, taken as
    2^-7 of the terms' sizes."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    n = run(inputs("cuda"))
    c = {k: v.cpu() for k, v in n.items() if isinstance(v, torch.Tensor)}
    moe = L.combine(n["down"]["y"], n["route"]["pos"], n["gate"]["weights"]).cpu()
    s, h = B.residual_norm(c["x"], y=moe, weight=c["w_next"], branch_weight=c["w_out"],
                           gate=c["branch_gate"])
    for name, want, size in (("s", s, c["x"].double().abs() + (s - c["x"].double()).abs()),
                             ("h", h, h.abs())):
        off = (n["out"][name].cpu().double() - want).abs()
        assert bool((off <= 2 ** -7 * size + 2 ** -20).all()), name
    ref = B.residual_norm_grad(n["out"]["s"].cpu(), c["ds"], c["dh_next"], y=moe, weight=c["w_next"],
                               branch_weight=c["w_out"], gate=c["branch_gate"])
    for k, got in n["grads"].items():
        off = (got.cpu().double() - ref[k]).abs()
        assert bool((off <= 2 ** -7 * ref[k + "_mag"] + 2 ** -20).all()), k
