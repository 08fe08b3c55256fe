"""Tensors of several devices do not reach the norm, dropout and loss kernels (with
stand-ins that have no memory), and what their argument blocks hold, on the CPU."""
import importlib

import pytest
import torch

from test_block_devices_cpu import HERE, THERE, Standin
from test_block_ops_abi_cpu import setup_module  # noqa: F401  (builds the library)

# (the package's names of these are the functions in them)
norm = importlib.import_module("rank_linear_gb300.norm")
dropout = importlib.import_module("rank_linear_gb300.dropout")
loss = importlib.import_module("rank_linear_gb300.loss")


class Tensor(Standin):
    def is_contiguous(self):
        return self.like.is_contiguous()

    def numel(self):
        return self.like.numel()


def norm_block(at=None, strides=None):
    t = lambda n, *s, dtype=torch.bfloat16: Tensor(*s, dtype=dtype, device=THERE if n == at else HERE)
    x = t("x", 6, 5, 64)
    if strides:
        x.like = torch.empty(6, 9, 64, dtype=torch.bfloat16, device="meta")[:, :5]
    return norm._make(x, t("weight", 64, dtype=torch.float32), 1e-5,
                      {"x": x, "residual": t("residual", 6, 5, 64), "h": t("h", 6, 5, 64), "y": t("y", 6, 5, 64)})


def test_norm_block():
    sh, dtype = norm_block()
    assert (sh.outer, sh.inner, sh.dim, sh.weight_fp32, dtype) == (30, 1, 64, 1, 0)
    sh, _ = norm_block(strides=True)  # x's two strides make the split of all
    assert (sh.outer, sh.inner) == (6, 5)
    assert tuple(sh.x) == (576, 64) and tuple(sh.y) == (320, 64)


@pytest.mark.parametrize("name", ["weight", "residual", "h", "y"])
def test_norm_devices(name):
    with pytest.raises(ValueError, match="cuda:1"):
        norm_block(name)


def test_norm_rstd_and_types():
    x = Tensor(6, 64)
    with pytest.raises(ValueError):
        norm._row_floats(Tensor(6, dtype=torch.float32, device=THERE), "rstd", x)
    with pytest.raises(ValueError):
        norm._row_floats(Tensor(7, dtype=torch.float32), "rstd", x)
    with pytest.raises(TypeError):
        norm._make(x, Tensor(64), 0.0, {"x": x, "y": Tensor(6, 64, dtype=torch.float32)})
    with pytest.raises(TypeError):
        norm._make(x, Tensor(64, dtype=torch.float16), 0.0, {"x": x})


def test_dropout_devices_and_seeds():
    assert dropout._make(Tensor(6, 64), Tensor(6, 64))[0] == (6, 64, 64, 64)
    with pytest.raises(ValueError, match="cuda:1"):
        dropout._make(Tensor(6, 64), Tensor(6, 64, device=THERE))
    assert dropout._drop_block(0.0, 1, 0, HERE) is None
    b = dropout._drop_block(0.5, -1, 7, HERE)
    assert (b.p, b.seed, b.offset, b.state) == (0.5, 2 ** 64 - 1, 7, None)
    for seed, offset in ((2 ** 64, 0), (-2 ** 63 - 1, 0), (1, -1), (1, 2 ** 32)):
        with pytest.raises(ValueError):
            dropout._drop_block(0.5, seed, offset, HERE)


@pytest.mark.parametrize("name", [None, "W", "targets", "weights", "dX", "losses"])
def test_loss_devices(name):
    t = lambda n, *s, dtype=torch.bfloat16: Tensor(*s, dtype=dtype, device=THERE if n == name else HERE)
    make = lambda: loss._make(t("X", 4, 3, 64), t("W", 100, 64), t("targets", 4, 3, dtype=torch.int32),
                              t("weights", 4, 3, dtype=torch.float32), 0.0, True, t("dX", 4, 3, 64),
                              t("losses", 4, 3, dtype=torch.float32))
    if name is None:
        sh, need = make()
        assert (sh.rows, sh.vocab, sh.dim, sh.target_bits, sh.mean, sh.x, sh.w, sh.dx) == \
            (12, 100, 64, 32, 1, 64, 64, 64) and need > 0
    else:
        with pytest.raises(ValueError, match="cuda:1"):
            make()


def test_collapsed_strides():
    c = dropout._collapsed
    assert c((3, 4), (4, 1)) == 1 and c((3, 4), (8, 2)) == 2 and c((3, 4), (9, 2)) is None
    assert c((), ()) == 0 and c((1, 1), (7, 9)) == 0 and c((1, 4), (99, 5)) == 5
    assert c((3, 4), (0, 0)) == 0 and c((3, 1), (5, 77)) == 5
