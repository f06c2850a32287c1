"""Batches whose units hold query tiles without any key tile, several of them to a CTA: no more rows
than one query tile, or sequences without keys. Every head comes out as it does in a small batch."""
import pytest
import torch

import io_aware_exact_07_gb300 as fa

pytestmark = pytest.mark.gpu


def draw(B, H, N, d):
    g = torch.Generator(device="cuda").manual_seed(N)
    return [torch.randn((B, H, N, d), generator=g, device="cuda").to(torch.bfloat16)
            for _ in range(4)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [1, 2, 100, 128, 129])
def test_forward_and_backward(N, d):
    x = draw(60, 16, N, d)
    o, lse = fa.fwd(*x[:3])
    grads = fa.bwd(*x[:3], o, x[3], lse)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_OK
    for b in (0, 31, 59):
        y = [t[b:b + 1].contiguous() for t in x]
        o1, lse1 = fa.fwd(*y[:3])
        assert torch.equal(o1, o[b:b + 1]) and torch.equal(lse1, lse[b:b + 1])
        for g, g1 in zip(grads, fa.bwd(*y[:3], o1, y[3], lse1)):
            assert torch.equal(g1, g[b:b + 1])


@pytest.mark.parametrize("N", [1, 100, 129])
def test_fp8_forward(N):
    x = draw(60, 16, N, 128)
    o, lse = fa.fwd_fp8(fa.fp8_quantize(*x[:3]), 0.088)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_OK
    for b in (0, 31, 59):
        o1, lse1 = fa.fwd_fp8(fa.fp8_quantize(*(t[b:b + 1].contiguous() for t in x[:3])), 0.088)
        assert torch.equal(o1, o[b:b + 1]) and torch.equal(lse1, lse[b:b + 1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,Nk", [(300, 300), (100, 700)])
@pytest.mark.parametrize("bias", [False, True])
def test_most_sequences_without_keys(Nq, Nk, d, bias):
    B, H = 80, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    q, do = (torch.randn((B, H, Nq, d), generator=g, device="cuda").to(torch.bfloat16)
             for _ in range(2))
    k, v = (torch.randn((B, H, Nk, d), generator=g, device="cuda").to(torch.bfloat16)
            for _ in range(2))
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    lens[5], lens[44] = Nk, 70
    kw = {}
    if bias:
        kw["rel_bias"] = fa.rel_bias(torch.randn((8, H), device="cuda"), fa.rel_buckets(8, 16))
    o, lse = fa.fwd(q, k, v, seqlens_k=lens, **kw)
    grads = fa.bwd(q, k, v, o, do, lse, seqlens_k=lens, **kw)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_OK
    none = lens == 0
    assert o[none].eq(0).all() and lse[none].eq(float("-inf")).all()
    assert all(t[none].eq(0).all() for t in grads[:3])
    for b in (5, 44):
        y = [t[b:b + 1].contiguous() for t in (q, k, v, do)]
        n = lens[b:b + 1].clone()
        o1, lse1 = fa.fwd(*y[:3], seqlens_k=n, **kw)
        assert torch.equal(o1, o[b:b + 1]) and torch.equal(lse1, lse[b:b + 1])
        for t, t1 in zip(grads, fa.bwd(*y[:3], o1, y[3], lse1, seqlens_k=n, **kw)[:3]):
            assert torch.equal(t1, t[b:b + 1])
