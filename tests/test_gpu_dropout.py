"""Dropout against its 64-bit definition (needs a GB300).

A kept element is x times the fp32 number nearest 2^32 / (2^32 - T) (off by 2^-24),
the product rounded to fp32 (2^-24) and to the type (2^-8 in bf16): relative
errors of at most 2^-8 + 2^-22 and 2^-22.  Dropped elements are 0 exactly.
"""
import numpy as np
import pytest
import torch

import rank_linear_gb300 as rl
from oracle import norm as on
from rank_linear_gb300 import _lib

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
REL = {torch.bfloat16: 2.0 ** -8 + 2.0 ** -22, torch.float32: 2.0 ** -22}
SEED = 0xFEDCBA9876543210


def check(x, y, p, seed, offset):
    x64 = x.double().cpu().numpy().reshape(-1, x.shape[-1])
    want = on.dropout(x64, p, seed % 2 ** 64, offset)
    got = y.double().cpu().numpy().reshape(want.shape)
    assert np.array_equal(got == 0, (want == 0) | (got == 0) & (np.abs(want) < 1e-38))
    assert np.all(np.abs(got - want) <= REL[x.dtype] * np.abs(want))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 3), (7, 8), (3, 9), (5, 1001), (300, 64), (2, 20000),
                                       (1000, 1), (129, 520)])
@pytest.mark.parametrize("p", [0.0, 0.3, 0.999])
def test_against_definition(rows, cols, p, dtype):
    g = torch.Generator(device=DEV).manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=g, device=DEV).to(dtype)
    y = rl.dropout_forward(x, p, SEED, 9)
    check(x, y, p, SEED if p else 0, 9)
    # the backward is the same mask and factor
    assert torch.equal(rl.dropout_backward(x, p, SEED, 9), y)


def test_strides_alignment_and_place():
    g = torch.Generator(device=DEV).manual_seed(1)
    base = torch.randn(40, 200, generator=g, device=DEV).bfloat16()
    for x in (base[:, :64], base[:, 1:66], base[::2, 8:72], base[3:4, 5:6], base[:1].expand(6, 200)):
        y = rl.dropout_forward(x, 0.4, 3, 1)
        check(x, y, 0.4, 3, 1)
        assert torch.equal(y, rl.dropout_forward(x.contiguous(), 0.4, 3, 1))
    x = base.clone()
    want = rl.dropout_forward(x, 0.25, 8)
    assert rl.dropout_forward(x, 0.25, 8, out=x) is x and torch.equal(x, want)
    part = torch.full((40, 210), 7.0, device=DEV, dtype=torch.bfloat16)
    rl.dropout_forward(base, 0.25, 8, out=part[:, :200])
    assert torch.equal(part[:, :200], want) and torch.all(part[:, 200:] == 7.0)
    with pytest.raises(ValueError):
        rl.dropout_forward(base.view(2, 20, 200)[:, :7], 0.1, 1)
    with pytest.raises(ValueError):
        rl.dropout_forward(base.t(), 0.1, 1)
    with pytest.raises(_lib.LoraError):
        rl.dropout_forward(base, 0.1, 1, out=base[:1].expand(40, 200))


def test_dropped_values_do_not_show():
    x = torch.tensor([[np.inf, np.nan, -np.inf, 1.0] * 50], device=DEV)
    y = rl.dropout_forward(x, 0.5, 4, 2).cpu().numpy()
    keep = on.words(1, 200, 4, 2) >= 2 ** 31
    assert np.all(y[~keep] == 0) and np.array_equal(np.isnan(y[keep]), np.isnan(x.cpu().numpy()[keep]))


def test_rows_beyond_32_bits_of_elements():
    """2^31 + elements: offsets pass 32 bits; rows from the start, the middle and the end."""
    rows, cols = 2 ** 18 + 3, 2 ** 13
    x = torch.ones(rows, cols, device=DEV, dtype=torch.bfloat16)
    y = rl.dropout_forward(x, 0.5, 21, 3)
    for r in (0, 1, 2 ** 17, 2 ** 18 - 1, 2 ** 18 + 2):
        want = on.dropout(np.ones((1, cols)), 0.5, 21, 3, first_row=r)
        assert np.array_equal(y[r].double().cpu().numpy(), want[0])


def test_many_items():
    """Rows past 32 bits: the counter's third word."""
    rows = 2 ** 32 + 5
    x = torch.ones(rows, 1, device=DEV, dtype=torch.bfloat16)
    rl.dropout_forward(x, 0.5, 21, 3, out=x)
    for r in (0, 2 ** 31 - 1, 2 ** 31, 2 ** 32 - 1, 2 ** 32, 2 ** 32 + 4):
        assert x[r, 0].item() == on.dropout(np.ones((1, 1)), 0.5, 21, 3, first_row=r)[0, 0]


def test_gradient_and_seed_tensor():
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randn(4, 50, 33, generator=g, device=DEV).requires_grad_()
    words = torch.tensor([12345, 6], device=DEV)
    y = rl.dropout(x, 0.3, words, 2)
    check(x.detach(), y.detach(), 0.3, 12345, 8)
    words.fill_(1)  # the backward's mask is the forward's all the same
    dy = torch.randn(y.shape, generator=g, device=DEV)
    y.backward(dy)
    check(dy, x.grad, 0.3, 12345, 8)
    with pytest.raises(ValueError):
        rl.dropout(x, 0.3, torch.tensor([1, 2]))
    with pytest.raises(ValueError):
        rl.dropout(x, 0.3, 1, 2 ** 32)
    with pytest.raises(ValueError):
        rl.dropout(x, 0.3, 2 ** 64)
    with pytest.raises(_lib.LoraError):
        rl.dropout(x, 1.0, 1)


def test_captured_graph_takes_new_seeds():
    x = torch.ones(64, 256, device=DEV)
    words = torch.tensor([5, 0], device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        rl.dropout_forward(x, 0.5, words)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = rl.dropout_forward(x, 0.5, words, 1)
    for seed, offset in ((5, 0), (6, 4)):
        words.copy_(torch.tensor([seed, offset]))
        graph.replay()
        assert torch.equal(y, rl.dropout_forward(x, 0.5, seed, offset + 1))


def test_other_stream_and_nothing():
    x = torch.randn(100, 64, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = rl.dropout_forward(x, 0.5, 1, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, rl.dropout_forward(x, 0.5, 1))
    assert rl.dropout_forward(x[:0], 0.5, 1).shape == (0, 64)
    assert rl.dropout_forward(x[:, :0], 0.5, 1).shape == (100, 0)
    with pytest.raises(TypeError):
        rl.dropout_forward(x.double(), 0.5, 1)


@pytest.mark.parametrize("cols", [192, 193, 255, 1001, 2033, 2034, 2046, 4099])
@pytest.mark.parametrize("lead", [0, 1, 7])
def test_rows_off_the_16_byte_boundaries(cols, lead):
    """bf16 rows whose x and y lie alike past a boundary (aligned pieces, masks shifted), and
    differently (element by element); strides that move the boundary from row to row or not."""
    g = torch.Generator(device=DEV).manual_seed(cols)
    for pad in (0, 1, 8 - cols % 8):
        step = cols + pad
        room = torch.randn(11 * step + lead + 1, generator=g, device=DEV).bfloat16()
        x = room[lead:].as_strided((11, cols), (step, 1))
        want = rl.dropout_forward(x.float().contiguous(), 0.4, SEED, 5).bfloat16()
        check(x, want, 0.4, SEED, 5)
        for off in (lead, lead + 1):
            out = torch.full_like(room, 7.0)
            y = out[off:].as_strided((11, cols), (step, 1)) if off + 10 * step + cols <= out.numel() else None
            if y is None:
                continue
            rl.dropout_forward(x, 0.4, SEED, 5, out=y)
            check(x, y, 0.4, SEED, 5)
            y.fill_(7.0)
            assert torch.all(out == 7.0)  # nothing beside the rows was written
        words = torch.tensor([77, 3], device=DEV)
        assert torch.equal(rl.dropout_forward(x, 0.1, words, 1), rl.dropout_forward(x.contiguous(), 0.1, 77, 4))
        bad = x.clone()
        bad[:, ::5] = float("nan")
        y = rl.dropout_forward(bad, 0.5, 3)
        keep = rl.dropout_forward(torch.ones_like(bad), 0.5, 3) != 0
        assert torch.all(y[~keep] == 0) and torch.equal(y.isnan(), bad.isnan() & keep)
        rl.dropout_forward(x, 0.4, SEED, 5, out=x)  # in place
        check_again = torch.where(want == 0, 0.0, x.float())
        assert torch.equal(check_again, x.float())
