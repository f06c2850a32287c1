"""Attention with keys of another length and a bias by relative position where counting could go wrong:
lengths out of range, more batch rows than are put in order, workspaces that hold anything, caches
of more than 2^31 elements."""
import math

import pytest
import torch

import io_aware_exact_07_gb300 as fa
from test_cross import check
from _cross import plain, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
def test_lengths_out_of_range_count_as_the_nearest_in_range(d):
    g = torch.Generator(device="cuda").manual_seed(d)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    q, k, v, do = r(4, 2, 70, d), r(4, 2, 200, d), r(4, 2, 200, d), r(4, 2, 70, d)
    rel = fa.rel_bias(torch.randn((32, 2), generator=g, device="cuda"), fa.rel_buckets())

    def run(lens):
        kw = dict(seqlens_k=torch.tensor(lens, dtype=torch.int32, device="cuda"), rel_bias=rel)
        o, lse = fa.fwd(q, k, v, **kw)
        step = fa.decode(q[:, :, :1].contiguous(), k, v, **kw)
        return (o, lse) + tuple(fa.bwd(q, k, v, o, do, lse, **kw)) + tuple(step)
    for a, b in zip(run([-5, 201, 2 ** 31 - 1, -2 ** 31]), run([0, 200, 200, 0])):
        assert torch.equal(a, b)


@pytest.mark.parametrize("rule", [None, (8, 30, True)])
def test_more_batch_rows_than_are_put_in_order(rule):
    check(300, 1, 1, 9, 150, 64, lens=[(7 * b) % 151 for b in range(300)], rule=rule, seed=70)


# the kernels' lists and parts lie in the workspace: of few key tiles cut into pieces, of the list of
# key tiles, of the gradient of a table, of steps of both kernels
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,Nk", [(1500, 150), (200, 700)])
def test_what_the_workspace_holds_does_not_matter(Nq, Nk, d):
    B, H, Hkv = 2, 4, 2
    g = torch.Generator(device="cuda").manual_seed(d)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    q, k, v, do = r(B, H, Nq, d), r(B, Hkv, Nk, d), r(B, Hkv, Nk, d), r(B, H, Nq, d)
    buckets = fa.rel_buckets(32, 128, True)
    rel = fa.rel_bias(torch.randn((32, H), generator=g, device="cuda"), buckets)
    kw = dict(seqlens_k=torch.tensor([Nk, 130], dtype=torch.int32, device="cuda"), rel_bias=rel)
    o, lse = fa.fwd(q, k, v, **kw)
    n = fa.fa_bwd_cross_workspace_size(B, H, Nq, Nk, d, rel_grad=True, rel_left=buckets.left,
                                       rel_right=buckets.right)
    guard = 4096
    got = []
    for fill in (0, 0xFF, 0x7F):
        ws = torch.full((n + guard,), fill, dtype=torch.uint8, device="cuda")
        ws[n:] = 0x5A
        got.append(fa.bwd(q, k, v, o, do, lse, workspace=ws[:n], **kw))
        assert ws[n:].eq(0x5A).all()
    for a, b, c in zip(*got):
        assert torch.equal(a, b) and torch.equal(a, c)
    for rows in (1, 8):
        qs = q[:, :, :rows].contiguous()
        n = fa.fa_decode_rel_workspace_size(B, H, Hkv, rows, Nk, d, 5)
        got = []
        for fill in (0, 0xFF, 0x7F):
            ws = torch.full((n + guard,), fill, dtype=torch.uint8, device="cuda")
            ws[n:] = 0x5A
            os, ls = torch.empty_like(qs), torch.empty((B, H, rows), device="cuda")
            st = fa.fa_decode_rel(qs, k, v, os, ls, B, H, Hkv, rows, Nk, d, 1 / math.sqrt(d),
                                  rel.lines, buckets.left, buckets.right, True, -1,
                                  kw["seqlens_k"], 5, ws, n)
            assert st == fa.FA_OK and ws[n:].eq(0x5A).all()
            got.append((os, ls))
        for a, b, c in zip(*got):
            assert torch.equal(a, b) and torch.equal(a, c)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_OK


def _enough(gb):
    if torch.cuda.mem_get_info()[0] < gb * 1e9:
        pytest.skip("not enough memory")


def test_keys_of_more_than_2_31_elements():
    """Forward and backward over 1100 heads of 31000 keys: the last head lies behind 2^31 elements."""
    _enough(40)
    B, H, Nq, Nk, d = 55, 20, 5, 31000, 64
    assert B * H * Nk * d > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16)
    q, k, v, do = r(B, H, Nq, d), r(B, H, Nk, d), r(B, H, Nk, d), r(B, H, Nq, d)
    lens = [Nk - 11 * b for b in range(B)]
    kw = dict(seqlens_k=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    o, lse = fa.fwd(q, k, v, **kw)
    grads = fa.bwd(q, k, v, o, do, lse, **kw)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_OK
    for b, h in ((0, 0), (B - 1, H - 1)):
        one = lambda x: x[b:b + 1, h:h + 1].cpu()
        want, tol = plain(one(q), one(k), one(v), one(do), lens=lens[b:b + 1])
        within("o", one(o), want["o"], tol["o"])
        for n, x in zip(("dq", "dk", "dv"), grads):
            within(n, one(x), want[n], tol[n])


@pytest.mark.parametrize("G", [1, 24])
def test_a_cache_of_more_than_2_31_elements(G):
    """A step over 16 heads of 1100000 keys, by either kernel (1 and 24 rows per K/V head)."""
    _enough(30)
    Hkv, Nk, d = 16, 1100000, 128
    assert Hkv * Nk * d > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16)
    q, k, v = r(1, Hkv * G, 1, d), r(1, Hkv, Nk, d), r(1, Hkv, Nk, d)
    table = torch.randn((32, Hkv * G), generator=g, device="cuda")
    b = fa.rel_buckets(32, 128, False)
    o, lse = fa.decode(q, k, v, causal=True, rel_bias=fa.rel_bias(table, b))
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_OK
    away = torch.arange(1 - Nk, 1, device="cuda").clamp(-b.left, b.right) + b.left
    for h in (0, Hkv * G - 1):
        kh, vh = k[0, h // G].double(), v[0, h // G].double()
        s = kh @ q[0, h, 0].double() / math.sqrt(d) + table[:, h].double()[b.map.long()[away]]
        p = s.softmax(0)
        want = p @ vh
        # weights and output rounded to bf16, half a step each
        bound = 2.0 ** -8 * (p @ vh.abs() + want.abs()) + 2.0 ** -18
        assert ((o[0, h, 0].double() - want).abs() - bound * (1 + 2.0 ** -9)).max() <= 0
        assert abs(lse[0, h, 0].double() - s.logsumexp(0)) <= 5e-4


@pytest.mark.parametrize("d", [64, 128])
def test_hidden_keys_of_any_size(d):
    """Keys that the causal mask hides from some rows or all, with scores whose weights overflow."""
    g = torch.Generator().manual_seed(d)
    r = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)
    q, k, v, do = r(2, 2, 100, d), r(2, 2, 300, d), r(2, 2, 300, d), r(2, 2, 100, d)
    k[:, :, 200:] *= 4096
    v[:, :, 200:] *= 4096
    gpu = [t.cuda() for t in (q, k, v, do)]
    kw = dict(causal=True, q_offset=100)
    o, lse = fa.fwd(*gpu[:3], **kw)
    grads = fa.bwd(*gpu[:3], o, gpu[3], lse, **kw)
    torch.cuda.synchronize()
    want, tol = plain(q, k, v, do, **kw)
    within("o", o, want["o"], tol["o"])
    for n, x in zip(("dq", "dk", "dv"), grads):
        within(n, x, want[n], tol[n])
