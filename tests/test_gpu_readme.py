"""The Python example of the README runs as it is written (needs a GB300)."""
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
    code, = [c for c in re.findall(r"```python\n(.*?)```", text, re.S) if "rotary_frequencies" in c]
    r = lambda *s: torch.randn(*s, device=DEV).bfloat16()
    q, k, v = r(2, 100, 8, 128).requires_grad_(), r(2, 100, 2, 128).requires_grad_(), r(2, 100, 2, 128)
    adapters = [r(16, 64).requires_grad_(), r(64, 16).requires_grad_()]
    for p in adapters:
        p.grad = torch.randn_like(p)
    names = dict(rl=rl, q=q, k=k, v=v, adapters=adapters,
                 positions=torch.arange(100, device=DEV).expand(2, 100),
                 doc_ids=torch.zeros(2, 100, dtype=torch.int32, device=DEV), q1=r(2, 8, 128),
                 k_cache=r(2, 50, 2, 128), v_cache=r(2, 50, 2, 128),
                 lengths=torch.tensor([50, 7], dtype=torch.int32, device=DEV))
    exec(code, names)
    rl.device_status()
    names["o"].float().sum().backward()
    assert names["o"].shape == (2, 100, 8, 128) and names["o1"].shape == (2, 8, 128)
    assert q.grad.shape == q.shape and float(names["norm"]) > 1.0
