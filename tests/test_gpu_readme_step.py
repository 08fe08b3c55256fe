"""The README's example of norm, dropout and loss runs as it is written (needs a GB300)."""
import os
import re

import pytest
import torch

import rank_linear_gb300 as rl

pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
DEV = "cuda:0"


def test_the_example():
    text = open(README, encoding="utf-8").read()
    code, = [c for c in re.findall(r"```python\n(.*?)```", text, re.S) if "rms_norm" in c]
    r = lambda *s: torch.randn(*s, device=DEV).bfloat16()
    leaves = dict(branch=r(2, 60, 256).requires_grad_(), A=(r(16, 256) / 16).requires_grad_(),
                  B=(r(320, 16) / 10).requires_grad_(), w=torch.ones(256, device=DEV).requires_grad_())
    targets = torch.randint(-1, 1000, (2, 60), device=DEV)
    names = dict(rl=rl, step=3, stream=r(2, 60, 256), W8=rl.quantize_w_fp8(r(320, 256) / 16),
                 head=r(1000, 320) / 16, targets=targets, **leaves)
    exec(code, names)
    rl.device_status()
    assert torch.isfinite(names["loss"]) and names["each"].shape == (2, 60)
    assert torch.all(names["each"][targets < 0] == 0)
    for t in leaves.values():
        assert t.grad.shape == t.shape and torch.isfinite(t.grad.float()).all()
