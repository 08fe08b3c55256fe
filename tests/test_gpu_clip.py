"""Global gradient norm and clipping on the GPU against 64 bits (needs a GB300).

Norm: at most 33 squares are summed in fp32 (33 * 2^-24 of the sum, half of it
in the root) and the result is rounded to fp32: 2^-19.  Clipped values: the
factor has the norm's error and two roundings, 2^-18, and bf16 outputs one
rounding more, 2^-8 (half of the smallest subnormal at the least).
"""
import math

import numpy as np
import pytest
import torch

import rank_linear_gb300 as rl

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
SMALLEST = {BF: 2.0 ** -133, F32: 2.0 ** -149}


def draw(shapes, dtypes, seed=0, gain=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [(torch.randn(s, generator=g, device=DEV) * gain).to(d) for s, d in zip(shapes, dtypes)]


def exact(grads, norm_type):
    x = [t.double().cpu().numpy().ravel() for t in grads]
    if norm_type == 2.0:
        return math.sqrt(sum(float((v * v).sum()) for v in x))
    return max([float(np.abs(v).max()) for v in x if v.size] + [0.0])


def check(grads, max_norm, norm_type=2.0, out=None):
    was = [t.clone() for t in grads]
    plan = rl.GradClip(grads, out=out)
    want = exact(was, norm_type)
    alone = plan.norm(norm_type=norm_type)
    assert all(torch.equal(a, b) for a, b in zip(grads, was)), "norm() changed the gradients"
    norm = plan.clip(max_norm, norm_type=norm_type)
    torch.cuda.synchronize()
    assert norm.item() == alone.item()
    assert abs(norm.item() - want) <= 2.0 ** -19 * want
    by = min(1.0, max_norm / (want + 1e-6))
    for g, w, o in zip(grads, was, plan.out):
        ref = w.double().cpu().numpy() * by
        err = np.abs(o.double().cpu().numpy() - ref)
        rel = 2.0 ** -18 + (2.0 ** -8 if g.dtype == BF else 0.0)
        assert np.all(err <= rel * np.abs(ref) + SMALLEST[g.dtype])
        if out is not None:
            assert torch.equal(g, w)
        elif norm.item() < max_norm * 0.99:
            assert torch.equal(g, w)
    return plan, norm


@pytest.mark.parametrize("norm_type", [2.0, math.inf])
@pytest.mark.parametrize("max_norm", [0.0, 0.5, 1e9])
@pytest.mark.parametrize("dtypes", [(BF,), (F32,), (BF, F32, F32)])
@pytest.mark.parametrize("inplace", [True, False])
def test_types_and_norms(dtypes, max_norm, norm_type, inplace):
    shapes = [(16, 4096), (1000, 16), (7, 333), (1,), (0,), (3, 5)]
    d = [dtypes[i % len(dtypes)] for i in range(len(shapes))]
    g = draw(shapes, d)
    check(g, max_norm, norm_type, None if inplace else [torch.full_like(t, math.nan) for t in g])


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 255, 2047, 2048, 2049, 4097, 8191, 8193, 1000003])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_sizes(n, dtype):
    check(draw([(n,)], [dtype], n), 0.25)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("a,b", [(0, 0), (1, 1), (1, 0), (0, 3), (5, 2), (7, 7)])
def test_addresses_off_a_vector(dtype, a, b):
    n = 30001
    src = draw([(n + 8,)], [dtype], 1)[0]
    dst = torch.full((n + 8,), 9.0, dtype=dtype, device=DEV)
    check([src[a:a + n], src[:0]], 0.1, out=[dst[b:b + n], dst[:0]])
    assert (dst[:b] == 9).all() and (dst[b + n:] == 9).all()


def test_many_tensors_of_many_sizes():
    shapes = [(i % 37 + 1, (i * i) % 211 + 1) for i in range(900)]
    check(draw(shapes, [BF if i % 3 else F32 for i in range(900)]), 1.0)


def test_large():
    check(draw([(128, 27648), (27648, 128), (40, 1 << 20)], [BF, F32, BF]), 1.0)


@pytest.mark.parametrize("gain", [1e-30, 1e-38, 1e-42, 1e17, 1e30])
def test_squares_out_of_fp32_range(gain):
    """Squares that fp32 cannot hold still give the norm."""
    g = draw([(4097,), (130,)], [F32, BF], gain=gain)
    plan = rl.GradClip(g)
    want = exact(g, 2.0)
    assert abs(plan.norm().item() - want) <= 2.0 ** -19 * want + 2.0 ** -149
    # small beside large within one tensor
    h = draw([(5000,)], [F32])[0]
    h[::7] *= gain
    want = exact([h], 2.0)
    assert abs(rl.GradClip([h]).norm().item() - want) <= 2.0 ** -19 * want


@pytest.mark.parametrize("norm_type", [2.0, math.inf])
def test_not_finite(norm_type):
    g = draw([(100,), (3000,)], [BF, F32])
    g[1][1234] = math.inf
    plan = rl.GradClip(g, out=[torch.empty_like(t) for t in g])
    assert plan.clip(1.0, norm_type=norm_type).item() == math.inf
    assert (plan.out[0] == 0).all() and torch.isnan(plan.out[1][1234])
    g[0][3] = math.nan
    assert math.isnan(plan.clip(1.0, norm_type=norm_type).item())
    assert torch.isnan(plan.out[0]).all()
    g[0][3], g[1][1234] = 0.0, 0.0
    want = exact(g, norm_type)
    assert abs(plan.clip(1.0, norm_type=norm_type).item() - want) <= 2.0 ** -19 * want


def test_zero_and_none():
    g = [torch.zeros(1000, dtype=BF, device=DEV), torch.zeros(0, device=DEV)]
    plan, norm = check(g, 1.0)
    assert norm.item() == 0.0
    assert rl.GradClip([]).norm().item() == 0.0
    assert rl.GradClip([]).clip(1.0).item() == 0.0


def test_same_bits_each_time_and_new_values():
    g = draw([(300000,), (77777,)], [BF, F32])
    plan = rl.GradClip(g, out=[torch.empty_like(t) for t in g])
    first = plan.clip(1.0).clone()
    outs = [t.clone() for t in plan.out]
    for _ in range(5):
        assert torch.equal(plan.clip(1.0), first)
        assert all(torch.equal(a, b) for a, b in zip(outs, plan.out))
    g[0].mul_(2.0)  # the plan reads what the tensors hold now
    want = exact(g, 2.0)
    assert abs(plan.clip(1.0).item() - want) <= 2.0 ** -19 * want


def test_on_another_stream():
    g = draw([(100000,)], [BF])
    want = exact(g, 2.0)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    norm = torch.empty((), device=DEV)
    rl.GradClip(g).clip(1.0, norm=norm, stream=s)
    s.synchronize()
    assert abs(norm.item() - want) <= 2.0 ** -19 * want


def test_refusals():
    g = torch.zeros(8, 8, dtype=BF, device=DEV)
    with pytest.raises(ValueError):
        rl.GradClip([g.t()[1:]])
    with pytest.raises(ValueError):
        rl.GradClip([g], out=[])
    with pytest.raises(ValueError):
        rl.GradClip([g], out=[g.float()])
    with pytest.raises(ValueError):
        rl.GradClip([g.cpu()])
    with pytest.raises(TypeError):
        rl.GradClip([g.half()])
    with pytest.raises(ValueError):
        rl.GradClip([g]).norm(norm_type=1.0)
    with pytest.raises(rl._lib.LoraError):
        rl.GradClip([g]).clip(-1.0)
    with pytest.raises(rl._lib.LoraError):
        rl.GradClip([g]).clip(math.nan)
