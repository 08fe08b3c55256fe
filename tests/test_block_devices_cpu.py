"""Tensors of several devices do not reach the kernels between the layers: the
argument blocks are formed from shapes, strides, types and devices alone, so that
stand-ins without memory show it on the CPU."""
import importlib

import pytest
import torch

import rank_linear_gb300 as rl
from test_block_ops_abi_cpu import setup_module  # noqa: F401  (builds the library)

# (the package's names of these are the functions in them)
attention = importlib.import_module("rank_linear_gb300.attention")
rotary = importlib.import_module("rank_linear_gb300.rotary")
HERE, THERE = torch.device("cuda", 0), torch.device("cuda", 1)


class Standin:
    """What an argument block is made from, of a tensor that is not there."""
    is_cuda = True

    def __init__(self, *shape, dtype=torch.bfloat16, device=HERE):
        self.like = torch.empty(shape, dtype=dtype, device="meta")
        self.shape, self.dtype, self.device = self.like.shape, dtype, device

    def stride(self, *a):
        return self.like.stride(*a)

    def dim(self):
        return self.like.dim()

    def unsqueeze(self, at):
        x = Standin(1, device=self.device)
        x.like = self.like.unsqueeze(at)
        x.shape = x.like.shape
        return x


def attention_block(**at):
    q = Standin(2, 5, 4, 64)
    big = lambda n, h: Standin(2, 5, h, 64, device=at.get(n, HERE))
    word = lambda n, *s, dtype=torch.int32: Standin(*s, dtype=dtype, device=at.get(n, HERE))
    return attention._make_shape(q, big("k", 2), big("v", 2), None, True, 0.0,
                                 word("slopes", 4, dtype=torch.float32), word("q_docs", 2, 5),
                                 word("k_docs", 2, 5), word("prefix", 2),
                                 {n: big(n, 4) for n in ("o", "d_o", "dq")},
                                 {n: big(n, 2) for n in ("dk", "dv")})


def test_one_device():
    assert attention_block().q_heads == 4


@pytest.mark.parametrize("name", ["k", "v", "o", "d_o", "dq", "dk", "dv", "slopes", "q_docs", "k_docs", "prefix"])
def test_attention(name):
    with pytest.raises(ValueError, match="cuda:1"):
        attention_block(**{name: THERE})


@pytest.mark.parametrize("name", ["k", "v", "o", "lengths", "slopes"])
def test_token(name):
    on = lambda n: THERE if n == name else HERE
    with pytest.raises(ValueError, match="cuda:1"):
        attention._make_token(Standin(2, 4, 64), Standin(2, 9, 2, 64, device=on("k")),
                              Standin(2, 9, 2, 64, device=on("v")),
                              Standin(2, dtype=torch.int32, device=on("lengths")), None, 0.0,
                              Standin(4, dtype=torch.float32, device=on("slopes")),
                              Standin(2, 4, 64, device=on("o")))


@pytest.mark.parametrize("name", [None, "k", "positions", "q_out", "k_out", "freqs"])
def test_rotary(name):
    on = lambda n: THERE if n == name else HERE

    class Freqs:
        rot, magnitude, device = 64, 1.0, on("freqs")

    make = lambda: rotary._make_shape(Standin(2, 5, 4, 64), Standin(2, 5, 2, 64, device=on("k")),
                                      Standin(2, 5, dtype=torch.int64, device=on("positions")), Freqs, False,
                                      False, Standin(2, 5, 4, 64, device=on("q_out")),
                                      Standin(2, 5, 2, 64, device=on("k_out")))
    if name is None:
        assert make()[0].q_heads == 4
    else:
        with pytest.raises(ValueError, match="device|cuda:1"):
            make()


def test_log_sum_exp_of_the_backward():
    t = lambda h: torch.zeros(1, 3, h, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="lse"):
        rl.attention_backward(t(4), t(4), t(2), t(2), t(4), torch.zeros(1, 4, 3, device="meta"))


def test_given_workspaces():
    like = torch.zeros(4)
    assert attention._scratch(16, like, like) is like
    for bad in (torch.zeros(4, device="meta"), torch.zeros(1).expand(64), torch.zeros(8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            attention._scratch(16, like, bad)


def test_the_current_device(monkeypatch):
    """A launch goes to the current device: it has to be the tensors'."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        rotary._stream_on(HERE, None)


def test_documents_of_one_side_are_refused():
    """The queries' alone or the keys' alone say nothing; the keys' were left out."""
    t = lambda h: torch.zeros(1, 3, h, 64, dtype=torch.bfloat16)
    d = torch.zeros(1, 3, dtype=torch.int32)
    for bad in ((None, d), (d, None), (d,), (d, d, d), []):
        with pytest.raises(ValueError, match="documents"):
            rl.attention_forward(t(4), t(2), t(2), documents=bad)
        with pytest.raises(ValueError, match="documents"):
            rl.attention_backward(t(4), t(4), t(2), t(2), t(4), torch.zeros(1, 4, 3), documents=bad)
    assert attention._doc_pair((None, None), t(4), t(2)) == (None, None)
