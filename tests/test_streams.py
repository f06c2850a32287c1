"""The helpers that allocate (fwd, bwd, decode, fp8_quantize, fwd_fp8) on a stream other than the
current one: their outputs and workspaces lie in no memory that work queued on the current stream
still uses, and results that are dropped wait for the work that reads them."""
import math

import pytest
import torch

import io_aware_exact_07_gb300 as fa

pytestmark = pytest.mark.gpu
DEV = "cuda"
B, H, N, D = 2, 2, 256, 128


def inputs(sign):
    """q, k, v, dO; q of 4 rows; O and lse; the quantised tensors: all there before any call."""
    g = torch.Generator().manual_seed(3)
    x = [sign * torch.randn((B, H, N, D), generator=g).to(torch.bfloat16).to(DEV) for _ in range(4)]
    out = dict(x=x, q4=x[0][:, :, :4].contiguous(), o=fa.fwd(*x[:3], causal=True),
               z=fa.fp8_quantize(*x[:3]))
    torch.cuda.synchronize()
    return out


def fwd(y, **kw):
    return fa.fwd(*y["x"][:3], causal=True, **kw)


def bwd(y, **kw):
    return fa.bwd(*y["x"][:3], y["o"][0], y["x"][3], y["o"][1], causal=True, **kw)


def decode(y, **kw):
    return fa.decode(y["q4"], *y["x"][1:3], num_ctas=40, **kw)


def fp8_quantize(y, **kw):
    return tuple(fa.fp8_quantize(*y["x"][:3], **kw).values())


def fwd_fp8(y, **kw):
    return fa.fwd_fp8(y["z"], 1.0 / math.sqrt(D), causal=True, **kw)


CALLS = [fwd, bwd, decode, fp8_quantize, fwd_fp8]


@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("call", CALLS)
def test_memory_is_neither_taken_too_early_nor_given_back(call, as_handle):
    x, other = inputs(1), inputs(-1)
    want = [t.clone() for t in call(x)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    stream = side.cuda_stream if as_handle else side
    torch.cuda.empty_cache()
    for _ in range(2):
        # blocks of every size up to the largest output's are dropped while writes to them wait
        # behind a long kernel on the current stream
        torch.cuda._sleep(200_000_000)
        late = [torch.empty(n, dtype=torch.uint8, device=DEV).fill_(77)
                for n in (512, 4096, 65536, 1 << 18, 1 << 19, 1 << 20) for _ in range(6)]
        del late
        got = call(x, stream=stream)
        torch.cuda.synchronize()
        assert fa.fa_device_status() == fa.FA_OK
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    # results dropped while a copy of them waits; the same call would write over them
    got = call(x, stream=stream)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(200_000_000)
    copies = [t.clone() for t in got]
    del got
    for _ in range(2):
        call(other, stream=stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(copies, want))


@pytest.mark.parametrize("handle", [0, 1, 2])  # the default stream, and CUDA's two handles for it
@pytest.mark.parametrize("call", CALLS)
def test_default_streams_by_their_handles(call, handle):
    x = inputs(1)
    want = call(x)
    torch.cuda.synchronize()
    got = call(x, stream=handle)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
