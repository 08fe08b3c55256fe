"""Rotary positions on the GPU against complex rotation in 64 bits (needs a GB300).

Per element: the cosine and sine are off by at most 2^-21 (the angle rounded
to 24 bits of half a turn, 2^-23 of a turn's radians, and two ulp of the
functions), products and the sum by 3 * 2^-24, so 2^-20 m (|x| + |y|); a bf16
output is rounded once more, 2^-8 of itself.
"""
import math

import numpy as np
import pytest
import torch

import rank_linear_gb300 as rl

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def turned(x, pos, freqs, interleaved, sign=1.0):
    """(value, |x| + |y| of its pair) in 64 bits; x [..., heads, dim], pos [...]."""
    x = x.double().cpu().numpy()
    r = freqs.rot
    a = pos.double().cpu().numpy()[..., None, None] * np.array(freqs.radians)
    z = x[..., 0:r:2] + 1j * x[..., 1:r:2] if interleaved else x[..., :r // 2] + 1j * x[..., r // 2:r]
    w = z * np.exp(1j * sign * a) * freqs.magnitude
    mag = (np.abs(z.real) + np.abs(z.imag)) * abs(freqs.magnitude)
    out, size = x.copy(), np.zeros_like(x)
    if interleaved:
        out[..., 0:r:2], out[..., 1:r:2] = w.real, w.imag
        size[..., 0:r:2] = size[..., 1:r:2] = mag
    else:
        out[..., :r // 2], out[..., r // 2:r] = w.real, w.imag
        size[..., :r // 2] = size[..., r // 2:r] = mag
    return out, size


def near(got, ref, size):
    bf = got.dtype == torch.bfloat16
    g = got.detach().double().cpu().numpy()
    bound = 2.0 ** -20 * size + (2.0 ** -8 * np.abs(ref) if bf else 0.0)
    assert np.all(np.abs(g - ref) <= bound + 1e-30), np.abs(g - ref).max()


def draw(shape, dtype, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


SCALINGS = [None, {"kind": "linear", "factor": 4.0}, {"kind": "base", "factor": 8.0},
            {"kind": "bands", "factor": 8.0, "original": 8192, "low": 1.0, "high": 4.0},
            {"kind": "ramp", "factor": 16.0, "original": 4096, "fast": 32.0, "slow": 1.0}]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(128, 128), (128, 64), (64, 64), (80, 80), (96, 32), (64, 2),
                                     (40, 24), (7, 6), (2, 2), (256, 256)])
def test_head_layouts(dim, rot, interleaved, dtype):
    f = rl.rotary_frequencies(rot, base=10000.0, device=DEV)
    q, k = draw((2, 37, 5, dim), dtype, 1), draw((2, 37, 2, dim), dtype, 2)
    pos = torch.randint(0, 100000, (2, 37), device=DEV)
    a, b = rl.rotary_forward(q, k, pos, f, interleaved=interleaved)
    near(a, *turned(q, pos, f, interleaved))
    near(b, *turned(k, pos, f, interleaved))
    a, b = rl.rotary_backward(q, k, pos, f, interleaved=interleaved)
    near(a, *turned(q, pos, f, interleaved, -1.0))
    near(b, *turned(k, pos, f, interleaved, -1.0))


@pytest.mark.parametrize("scaling", SCALINGS)
@pytest.mark.parametrize("top", [1, 5000, 2 ** 20, 2 ** 31 - 1, 2 ** 40])
def test_positions_and_scalings(scaling, top):
    f = rl.rotary_frequencies(64, base=500000.0, scaling=scaling, device=DEV)
    q = draw((50, 3, 64), torch.float32, 3)
    # numpy's own pos * w is exact to 2^-53 of the angle: compare where that is below the bound
    pos = torch.randint(-top, top + 1, (50,), device=DEV)
    a, none = rl.rotary_forward(q, None, pos, f)
    assert none is None
    ref, size = turned(q, pos, f, False)
    slack = top * 2.0 ** -52 * size
    err = np.abs(a.double().cpu().numpy() - ref)
    assert np.all(err <= 2.0 ** -20 * size + slack + 1e-30)
    if top < 2 ** 31:
        b, _ = rl.rotary_forward(q, None, pos.int(), f)
        assert torch.equal(a, b)


def test_scalings_follow_their_formulas():
    w = rl.rotary_frequencies(64, base=10000.0, device=DEV).radians
    assert w == [10000.0 ** (-2 * i / 64) for i in range(32)]
    f = rl.rotary_frequencies(64, base=10000.0, scaling=SCALINGS[2], device=DEV).radians
    assert f[0] == 1.0 and math.isclose(f[-1] * 8.0, w[-1], rel_tol=1e-12)
    f = rl.rotary_frequencies(64, base=10000.0, scaling=SCALINGS[3], device=DEV).radians
    for x, y in zip(w, f):
        turns = 8192 * x / (2 * math.pi)
        assert y == x if turns >= 4 else math.isclose(y, x / 8) if turns <= 1 else x / 8 < y < x
    r = rl.rotary_frequencies(64, base=10000.0, scaling=SCALINGS[4], device=DEV)
    assert r.radians[0] == w[0] and math.isclose(r.radians[-1], w[-1] / 16)
    assert math.isclose(r.magnitude, 0.1 * math.log(16) + 1)


@pytest.mark.parametrize("tokens", [1, 2, 31, 4097])
def test_token_counts_and_broadcast_positions(tokens):
    f = rl.rotary_frequencies(128, device=DEV)
    q, k = draw((3, tokens, 8, 128), torch.bfloat16, 1), draw((3, tokens, 2, 128), torch.bfloat16, 2)
    pos = torch.arange(tokens, device=DEV)
    a, b = rl.rotary_forward(q, k, pos, f)
    near(a, *turned(q, pos.expand(3, -1), f, False))
    near(b, *turned(k, pos.expand(3, -1), f, False))


@pytest.mark.parametrize("dim", [128, 60])
@pytest.mark.parametrize("interleaved", [False, True])
def test_views_in_place_and_out(dim, interleaved):
    """q and k inside one q|k|v tensor: turned in place, v untouched."""
    f = rl.rotary_frequencies(32, device=DEV)
    x = draw((2, 19, 12, dim), torch.bfloat16, 4)
    pos = torch.arange(19, device=DEV) + 100
    was = x.clone()
    q, k = x[:, :, :8], x[:, :, 8:10]
    sep = rl.rotary_forward(q, k, pos, f, interleaved=interleaved)
    assert torch.equal(x, was)
    out = rl.rotary_forward(q, k, pos, f, interleaved=interleaved, q_out=q, k_out=k)
    assert out[0] is q and torch.equal(q, sep[0]) and torch.equal(k, sep[1])
    assert torch.equal(x[:, :, 10:], was[:, :, 10:])
    near(q, *turned(was[:, :, :8], pos.expand(2, -1), f, interleaved))


@pytest.mark.parametrize("shift", [1, 3])
def test_addresses_off_a_vector(shift):
    f = rl.rotary_frequencies(64, device=DEV)
    flat = draw((5 * 4 * 64 + 8,), torch.bfloat16, 5)
    q = flat[shift:shift + 5 * 4 * 64].view(5, 4, 64)
    pos = torch.arange(5, device=DEV)
    a, _ = rl.rotary_forward(q, None, pos, f)
    near(a, *turned(q, pos, f, False))


def test_autograd_and_differences():
    f = rl.rotary_frequencies(32, scaling=SCALINGS[4], device=DEV)
    q, k = draw((2, 9, 4, 48), torch.float32, 1), draw((2, 9, 2, 48), torch.float32, 2)
    pos = torch.randint(0, 10000, (2, 9), device=DEV)
    q.requires_grad_()
    k.requires_grad_()
    gq, gk = draw(q.shape, torch.float32, 3), draw(k.shape, torch.float32, 4)
    a, b = rl.rotary(q, k, pos, f, interleaved=True)
    torch.autograd.backward((a, b), (gq, gk))
    near(q.grad, *turned(gq, pos, f, True, -1.0))
    near(k.grad, *turned(gk, pos, f, True, -1.0))
    # the operator is linear: a difference over a whole step is its derivative
    u = draw(q.shape, torch.float32, 5)
    up, _ = turned(q.detach() + u, pos, f, True)
    down, _ = turned(q.detach(), pos, f, True)
    want = float(((up - down) * gq.double().cpu().numpy()).sum())
    got = float((q.grad.double() * u.double()).sum())
    size = float((gq.abs().sum(-1, keepdim=True) * u.abs()).sum()) * f.magnitude
    assert abs(got - want) <= 2.0 ** -19 * size


def test_nothing_and_another_stream():
    f = rl.rotary_frequencies(64, device=DEV)
    e = torch.empty(2, 0, 4, 64, dtype=torch.bfloat16, device=DEV)
    a, b = rl.rotary_forward(e, None, torch.empty(2, 0, dtype=torch.int64, device=DEV), f)
    assert a.shape == e.shape and b is None
    q = draw((70, 4, 64), torch.bfloat16, 1)
    pos = torch.arange(70, device=DEV)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    a, _ = rl.rotary_forward(q, None, pos, f, stream=s)
    s.synchronize()
    near(a, *turned(q, pos, f, False))


@pytest.mark.parametrize("kw,error", [
    (dict(positions=torch.zeros(3)), TypeError),
    (dict(positions=torch.zeros(4, dtype=torch.int64)), ValueError),
    (dict(k=torch.zeros(3, 2, 32, dtype=torch.bfloat16)), ValueError),
    (dict(k=torch.zeros(3, 2, 64)), TypeError),
    (dict(q=None, k=None), ValueError),
    (dict(rot=128), rl._lib.LoraError),
])
def test_refusals(kw, error):
    f = rl.rotary_frequencies(kw.pop("rot", 64), device=DEV)
    a = dict(q=torch.zeros(3, 4, 64, dtype=torch.bfloat16), k=None,
             positions=torch.zeros(3, dtype=torch.int64))
    a.update(kw)
    a = {n: None if t is None else t.to(DEV) for n, t in a.items()}
    with pytest.raises(error):
        rl.rotary_forward(a["q"], a["k"], a["positions"], f)


@pytest.mark.parametrize("kw", [dict(rot=3), dict(rot=0), dict(base=-1.0),
                                dict(scaling={"kind": "what"}), dict(scaling={"kind": "linear"}),
                                dict(scaling={"kind": "linear", "factor": 0.0}),
                                dict(scaling={"kind": "bands", "factor": 2.0, "original": 8, "low": 2.0,
                                              "high": 1.0})])
def test_frequency_refusals(kw):
    with pytest.raises(ValueError):
        rl.rotary_frequencies(kw.pop("rot", 64), device=DEV, **kw)


@pytest.mark.parametrize("top", [2 ** 20, 2 ** 31, 2 ** 36, 2 ** 40, 2 ** 41])
def test_far_positions_against_whole_numbers(top):
    """The angle's fraction of a turn from exact arithmetic: no allowance for the position."""
    from fractions import Fraction
    from test_rotary_turns_cpu import over_two_pi
    c = over_two_pi()
    f = rl.rotary_frequencies(64, base=500000.0, device=DEV)
    q = draw((40, 2, 64), torch.float32, 3)
    pos = torch.randint(top // 2, top, (40,), device=DEV)
    pos[::2] *= -1
    got = rl.rotary_forward(q, None, pos, f)[0].double().cpu().numpy()
    turn = np.array([[float(p * Fraction(w) * c % 1) for w in f.radians] for p in pos.tolist()])
    x = q.double().cpu().numpy()
    z = (x[..., :32] + 1j * x[..., 32:]) * np.exp(2j * np.pi * turn)[:, None]
    size = np.abs(x[..., :32]) + np.abs(x[..., 32:])
    assert np.all(np.abs(got[..., :32] - z.real) <= 2.0 ** -20 * size)
    assert np.all(np.abs(got[..., 32:] - z.imag) <= 2.0 ** -20 * size)
