"""Calls from several host threads at once on one kernel whose launches differ in shared memory
(needs a GB300)."""
import ctypes
import threading

import pytest
import torch

import rank_linear_gb300 as rl
from rank_linear_gb300 import _lib

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
CALLS = 4000


def at_once(make, *sizes):
    """Two threads a size, each with tensors and a stream of its own, call the library over and over
    with as little of Python in between as there can be: no call fails, and the last results have the
    bits of a call alone."""
    jobs = [make(s) for s in sizes for _ in range(2)]
    alone = []
    for entry, args, out, _ in jobs:
        assert entry(*args, None) == _lib.LORA_OK, _lib.lib().lora_last_error().decode()
        torch.cuda.synchronize()
        alone.append([t.clone() for t in out])
    gate, failed = threading.Barrier(len(jobs)), []

    def work(entry, args):
        torch.cuda.set_device(DEV)
        stream = torch.cuda.Stream()
        handle = ctypes.c_void_p(stream.cuda_stream)
        gate.wait(60)
        for _ in range(CALLS):
            if entry(*args, handle):
                failed.append(_lib.lib().lora_last_error().decode())
                break
        stream.synchronize()
    threads = [threading.Thread(target=work, args=job[:2]) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for (_, _, out, _), want in zip(jobs, alone):
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    rl.device_status()


def rand(*shape, dtype=torch.bfloat16):
    g = torch.Generator(device=DEV).manual_seed(sum(shape))
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def address(t):
    return ctypes.c_void_p(t.data_ptr())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("backward", [False, True])
def test_norms_of_two_widths(backward, dtype):
    """Rings of blocks of at most 256 threads, over rows of 4096 and 2048 elements."""
    code = 0 if dtype == torch.bfloat16 else 1

    def make(dim):
        x, res, w, y, h = (rand(*s, dtype=dtype) for s in ((310, dim), (310, dim), (dim,), (310, dim), (310, dim)))
        rstd = torch.rand(310, device=DEV)
        names = ("x", "residual", "h", "y", "dy", "dh", "dx", "dresidual")
        sh = _lib.NormShape(outer=310, inner=1, dim=dim, eps=1e-6, **{n: (dim, 0) for n in names})
        at = [address(t) for t in (x, res, w, h, y, rstd)]
        keep = (sh, x, res, w, h, y, rstd)
        if backward:  # (y: the gradient that comes out)
            return _lib.lib().lora_norm_bwd, (ctypes.byref(sh), at[0], at[1], at[2], at[5], at[3], None, code, at[4],
                                              None, None, None, 0), (y,), keep
        return _lib.lib().lora_norm_fwd, (ctypes.byref(sh), at[0], at[1], at[2], None, code, at[3], at[4], at[5],
                                          None, None), (y, h, rstd), keep
    at_once(make, 4096, 2048)


def test_layers_of_two_ranks():
    """The low-rank passes of rank 8 and 256 take 104 KB of shared memory and 134 or more."""
    def make(rank):
        X, W, A, B, Y = rand(256, 512), rand(512, 512), rand(rank, 512), rand(512, rank), rand(256, 512)
        saved = torch.empty(_lib.lib().lora_linear_saved_bytes(256, rank, 0), dtype=torch.uint8, device=DEV)
        n = _lib.lib().lora_linear_workspace_bytes(256, 512, 512, rank, 0)
        ws = torch.empty(n, dtype=torch.uint8, device=DEV)
        return _lib.lib().lora_linear_fwd, (*(address(t) for t in (X, W, A, B)), 16.0, rank, 256, 512, 512, 0,
                                            *(address(t) for t in (Y, saved, ws)), n), (Y,), (X, W, A, B, saved, ws)
    at_once(make, 8, 256)
