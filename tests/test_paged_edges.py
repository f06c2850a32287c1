"""Paged caches at the edges of what the calls take, on the GPU against the fp64 oracle."""
import numpy as np
import pytest
import torch

import io_aware_exact_07_gb300 as fa
import oracle
from _paged import Batch, check_attn

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -8  # half a step of bf16, relative to the value


def sync():
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_OK


def attn(b, x, **kw):
    return fa.paged_attn(x.q, x.k, x.v, x.table, x.kv, cu_seqlens_q=x.cu, **x.sc, **kw)


# ------------------------------------------------------------------ scales by key tile

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq,kv", [
    ([40] * 60, [300, 380, 257] * 20),               # pieces of 3 tiles, cut by the runs' ends
    ([33] * 40, [600, 130, 890, 100] * 10),          # 5, 2, 7 and 1 tiles
    ([200] * 9, [1100, 640, 333] * 3),               # rounds of whole units
])
def test_scales_that_differ_from_tile_to_tile(nq, kv, d):
    # every 128 keys the scales of K and of V change by up to 2^6 and 2^12, so that a tile that
    # took another one's would be far off. Within a tile they are alike, so that the f16 tiles
    # are exact; P's rounding to f16 adds 2^-32 of the row's largest weight times value scale,
    # once a key.
    b = Batch(nq, kv, 32, 2, d, True, G=2, seed=51)
    g = torch.Generator().manual_seed(51)
    for i, L in enumerate(kv):
        for n, lo, hi in (("k", -6, 1), ("v", -10, 3)):
            e = torch.randint(lo, hi, (-(-L // 128), 1, 1), generator=g).repeat_interleave(128, 0)
            b.rows[n][i] = (b.rows[n][i].float() * torch.exp2(e[:L].float())).to(torch.bfloat16)
    x = b.fill().on(DEV)
    o_ref, lse_ref, o_abs = b.oracle(True)
    tol = 1.05 * U * (o_abs + np.abs(o_ref)) + max(kv) * 2.0 ** -32 * 448 * 2.0 ** -4
    assert int(b.scale["v"][b.scale["v"] != 133].max()) - 127 <= -4  # |V| < 28 = 448 * 2^-4
    for _ in range(5):
        o, lse = attn(b, x, causal=True, max_q=max(nq))
        sync()
        assert np.all(np.abs(o.double().cpu().numpy() - o_ref) <= tol)
        assert np.abs(lse.double().cpu().numpy() - lse_ref).max() <= 2e-4


# ------------------------------------------------------------------ the longest sequences

class Longest:
    """One sequence of 2^31 - 272 positions, the most that a table of whole pages can hold, over
    four pages named many times: its first three pages hold values of -1, all others of +1. The
    exact result follows from how often each page is named."""
    page, entries = 144, 14913079

    def __init__(self, d, e4m3, G, seed):
        g = torch.Generator().manual_seed(seed)
        self.L = self.page * self.entries
        assert self.L == 2 ** 31 - 272
        self.table = torch.randint(1, 4, (1, self.entries), generator=g, dtype=torch.int32)
        self.table[0, :3] = 0
        self.q = torch.randn((1, G, d), generator=g).to(torch.bfloat16)
        rows = torch.randn((4 * self.page, 1, d), generator=g).to(torch.bfloat16)
        vals = torch.ones((4, self.page, 1, d), dtype=torch.bfloat16)
        vals[0] = -1
        self.cache = fa.paged_cache(4, self.page, 1, d, e4m3=e4m3, device=DEV)
        fill = torch.arange(4, dtype=torch.int32, device=DEV)[None]
        n = torch.tensor([4 * self.page], dtype=torch.int32, device=DEV)
        fa.paged_write(rows.to(DEV), vals.reshape(rows.shape).to(DEV), page_table=fill, kv_lens=n,
                       **self.cache)
        k, _ = fa.paged_read(page_table=fill, kv_lens=n, N=4 * self.page, **self.cache)
        self.kv = torch.tensor([self.L], dtype=torch.int32, device=DEV)
        s = self.q[0].double() @ k[0, 0].double().cpu().T / np.sqrt(d)       # [G, 4 pages' rows]
        times = torch.bincount(self.table[0].long(), minlength=4).double().repeat_interleave(self.page)
        w = times * s.exp()
        sign = torch.ones(4 * self.page, dtype=torch.float64)
        sign[:self.page] = -1
        self.lse, self.o = w.sum(1).log(), (w * sign).sum(1) / w.sum(1)

    def check(self, steps):
        """Sums of `steps` terms in fp32, each addition off by at most 2^-23 of the sum (the tensor
        cores may cut where others round): O, of values of magnitude 1, and lse."""
        o, lse = fa.paged_attn(self.q.to(DEV), page_table=self.table.to(DEV), kv_lens=self.kv, max_q=1,
                               causal=True, **self.cache)
        sync()
        tol = steps * 2.0 ** -23 + 2 * U
        assert (o[0].double().cpu() - self.o[:, None]).abs().max().item() <= 2 * tol < 0.5
        assert (lse[0].double().cpu() - self.lse).abs().max().item() <= tol


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("G", [4, 16, 24])
def test_longest_sequence_with_few_rows(G, d, e4m3):
    # each warp of a CTA (8 of them at least) adds 16 keys at a time
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    Longest(d, e4m3, G, 61).check(2 ** 31 // 16 // 8 // sms + 1)


@pytest.mark.parametrize("e4m3", [False, True])
def test_new_row_at_the_last_position(e4m3):
    z = Longest(64, e4m3, 1, 62)
    new = torch.full((1, 1, 64), 0.5, dtype=torch.bfloat16, device=DEV)
    fa.paged_write(new, -new, page_table=z.table.to(DEV), kv_lens=z.kv, **z.cache)
    k, v = fa.paged_read(page_table=z.table[:, -1:].to(DEV), N=z.page,
                         kv_lens=torch.tensor([z.page], dtype=torch.int32, device=DEV), **z.cache)
    sync()
    assert (k[0, 0, -1] == 0.5).all() and (v[0, 0, -1] == -0.5).all() and (v[0, 0, :-1] == 1).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("e4m3", [False, True])
def test_longest_sequence_with_many_rows(d, e4m3):
    # a CTA's two warpgroups take key tiles of 128 in turn, in 8 products of 16 keys each
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    Longest(d, e4m3, 32, 63).check(2 ** 31 // 16 // 2 // sms + 8)


# ------------------------------------------------------------------ NaN

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("nq,kv,Hkv", [
    ([1, 1], [300, 170], 2),         # whole heads
    ([3, 1], [9000, 12345], 2),      # heads cut between CTAs
    ([60, 33], [300, 170], 2),       # whole query tiles
    ([300], [9001], 1),              # cut ones
])
def test_a_nan_in_a_query_is_a_nan_in_its_row(nq, kv, Hkv, d, e4m3):
    b = Batch(nq, kv, 32, Hkv, d, e4m3, G=2, seed=71)
    ref = b.oracle(True)
    hit = torch.zeros(b.q.shape[:2], dtype=torch.bool)
    for t, h, c in ((0, 1, 5), (b.T - 1, 0, d - 1), (b.T // 2, b.H - 1, 0)):
        b.q[t, h, c] = float("nan")
        hit[t, h] = True
    x = b.fill().on(DEV)
    o, lse = attn(b, x, causal=True, max_q=max(nq))
    sync()
    o, lse = o.cpu(), lse.cpu()
    assert torch.isnan(o[hit]).all() and torch.isnan(lse[hit]).all()
    keep = ~hit.numpy()
    check_attn(o[~hit], lse[~hit], tuple(r[keep] for r in ref))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("nq,kv", [([1, 1], [300, 170]), ([1, 1], [20001, 170]),
                                   ([60, 33], [300, 170]), ([60, 33], [9001, 170])])
def test_a_nan_in_a_key_is_a_nan_in_the_rows_that_see_it(nq, kv, e4m3):
    b = Batch(nq, kv, 16, 1, 64, e4m3, G=2, seed=72)
    ref = b.oracle(True)
    b.rows["k"][0][5, 0, 3] = float("nan")
    x = b.fill().on(DEV)
    o, lse = attn(b, x, causal=True, max_q=max(nq))
    sync()
    assert torch.isnan(o[:nq[0]]).all() and torch.isnan(lse[:nq[0]]).all()
    check_attn(o[nq[0]:], lse[nq[0]:], tuple(r[nq[0]:] for r in ref))


# ------------------------------------------------------------------ the ends of the range of scales

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("order", ["small first", "large first", "mixed"])
@pytest.mark.parametrize("nq,kv", [([1, 1], [600, 90]), ([4, 3], [600, 90]), ([8, 5], [600, 90]),
                                   ([2, 1], [20001, 90]), ([60, 33], [600, 90])])
def test_values_of_both_ends_of_the_range_of_scales(nq, kv, order, d):
    # V's rows have the smallest scale, 2^-117, and the largest, 2^6 (or any between): the softmax
    # sum counts all keys alike, also those whose weight times value scale is 2^-126 of the largest
    # or less, as scores of up to 4 sqrt(d) make it. P's rounding to f16 adds 2^-32 of the row's
    # largest weight times value scale, once a key, and f16 tiles 2^-25 of the scale. Scores are
    # four times those of check_attn, and their fp32 errors: 8e-4, 20 % of 2^-8.
    b = Batch(nq, kv, 16, 2, d, True, G=2, seed=81)
    g = torch.Generator().manual_seed(81)
    for i, L in enumerate(kv):
        b.rows["k"][i] *= 4
        e = torch.full((L, 1, 1), -116.0)
        if order == "mixed":
            e = torch.randint(-116, 14, (L, 1, 1), generator=g).float()
        elif order == "small first":
            e[L * 3 // 4::37] = 13
        else:
            e[:L // 4:37] = 13
        v = b.rows["v"][i].double().clamp(-3.4, 3.4) * torch.exp2(e.double())
        b.rows["v"][i] = v.to(torch.bfloat16)
    x = b.fill().on(DEV)
    scales = oracle.quantize_rows(b.rows["v"][0].double().numpy())[1].astype(int) - 127
    assert scales.min() == -117 and scales.max() >= 5
    o, lse = attn(b, x, causal=True, max_q=max(nq))
    sync()
    o_ref, lse_ref, o_abs = b.oracle(True)
    tol = 1.2 * U * (o_abs + np.abs(o_ref)) + 448 * 2.0 ** 7 * (max(kv) * 2.0 ** -32 + 2.0 ** -25)
    assert np.abs(lse.double().cpu().numpy() - lse_ref).max() <= 8e-4
    assert np.all(np.abs(o.double().cpu().numpy() - o_ref) <= tol)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,B", [(1, 200), (16, 200), (24, 200), (4, 3)])
def test_smallest_values_under_large_sums(G, B, d):
    # a head's first 384 keys have a score of 0, the others one of 5.5 (7.9 in log2 units, just less
    # than moves the maximum); all its values are 1.5 * 2^-112, so O is that
    n, page = 30000, 16
    c = fa.paged_cache(n // page, page, 1, d, e4m3=True, device=DEV)
    k = torch.full((n, 1, d), 0.6875 * 64 / d)
    k[:384] = 0
    v = torch.full((n, 1, d), 1.5 * 2.0 ** -112)
    table = torch.arange(n // page, dtype=torch.int32, device=DEV).expand(B, -1).contiguous()
    kv = torch.full((B,), n, dtype=torch.int32, device=DEV)
    fa.paged_write(k.to(torch.bfloat16).to(DEV), v.to(torch.bfloat16).to(DEV), page_table=table[:1],
                   kv_lens=kv[:1], **c)
    q = torch.ones(B, G, d, dtype=torch.bfloat16, device=DEV)
    o, lse = fa.paged_attn(q, page_table=table, kv_lens=kv, max_q=1, scale=0.125, **c)
    sync()
    exact = float(v[0, 0, 0])
    # O is off by its rounding, 2^-8 of it, P's weights by 2^-11, and 30000 additions in fp32 by less
    # than 2^-9
    assert (o.double() / exact - 1).abs().max().item() <= 2.0 ** -8 + 2.0 ** -9 + 2.0 ** -10
    lse_ref = np.log(384 + (n - 384) * np.exp(5.5))
    assert (lse.double() - lse_ref).abs().max().item() <= 2e-4 + 2.0 ** -9


# ------------------------------------------------------------------ memory on another stream

def handles(stream):
    return stream, stream.cuda_stream


@pytest.mark.parametrize("as_handle", [0, 1])
def test_memory_that_the_current_stream_still_uses_is_not_taken(as_handle):
    # a tensor of the results' size is dropped while a write to it waits behind a long kernel
    b = Batch([1, 30], [700, 300], 16, 2, 64, G=2, seed=91)
    x = b.fill().on(DEV)
    side = torch.cuda.Stream()
    call = dict(stream=handles(side)[as_handle])
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    for _ in range(2):
        torch.cuda._sleep(200_000_000)
        late = [torch.empty(t.shape, dtype=t.dtype, device=DEV).fill_(9) for t in
                (x.q, torch.empty(x.q.shape[:2]), torch.empty(2, 2, 700, 64, dtype=torch.bfloat16),
                 torch.empty(2, 2, 700, 64, dtype=torch.bfloat16),
                 torch.empty(fa.fa_paged_workspace_size(4, 2, 64, 30, 704), dtype=torch.uint8))]
        del late
        o, lse = attn(b, x, causal=True, max_q=30, **call)
        k, v = fa.paged_read(x.k, x.v, x.table, x.kv, 700, **call)
        sync()
        check_attn(o, lse, b.oracle(True))
        for n, got in (("k", k), ("v", v)):
            assert np.array_equal(got[0].double().cpu().numpy(), np.moveaxis(b.stored(n, 0), 0, 1))


@pytest.mark.parametrize("as_handle", [0, 1])
def test_results_dropped_while_the_current_stream_reads_them(as_handle):
    b = Batch([1, 30], [700, 300], 16, 2, 64, G=2, seed=92)
    x = b.fill().on(DEV)
    side = torch.cuda.Stream()
    call = dict(stream=handles(side)[as_handle])
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    o, lse = attn(b, x, causal=True, max_q=30, **call)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(200_000_000)
    got = o.clone(), lse.clone()
    del o, lse
    for _ in range(3):  # would write over them, had their memory been handed out again
        fa.paged_attn(-x.q, x.k, x.v, x.table, x.kv, cu_seqlens_q=x.cu, max_q=30, **call)
    sync()
    check_attn(*got, b.oracle(True))


@pytest.mark.parametrize("handle", [0, 1, 2])  # the default stream, and CUDA's two handles for it
def test_default_streams_by_their_handles(handle):
    b = Batch([1, 30], [700, 300], 16, 2, 64, G=2, seed=93)
    x = b.fill().on(DEV)
    torch.cuda.synchronize()
    o, lse = attn(b, x, causal=True, max_q=30, stream=handle)
    k, _ = fa.paged_read(x.k, x.v, x.table, x.kv, 700, stream=handle)
    sync()
    check_attn(o, lse, b.oracle(True))
    assert np.array_equal(k[0].double().cpu().numpy(), np.moveaxis(b.stored("k", 0), 0, 1))


# ------------------------------------------------------------------ reported from the device

@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("cu,kv,stored", [
    # offsets, lengths; the new tokens (of 6) of each sequence that enter its last positions
    ([0, 3, 6], [200, 130], ((0, 3), (3, 6))),      # nothing wrong
    ([0, 3, 1000], [200, 130], ((0, 3), None)),
    ([0, 3, 7], [200, 130], ((0, 3), None)),
    ([0, -2, 6], [200, 130], (None, None)),
    ([-1, 3, 6], [200, 130], (None, (3, 6))),
    ([0, 6, 1000], [200, 130], ((0, 6), None)),     # no token leads to the second sequence ...
    ([0, 6, 5], [200, 130], ((0, 5), None)),
    ([0, 6, 6], [200, -1], ((0, 6), None)),
    ([0, 0, 6], [10 ** 6, 130], (None, (0, 6))),    # ... or to the first
    ([0, 3, 6], [200, 10 ** 6], ((0, 3), None)),
    ([0, 3, 6], [-5, 130], (None, (3, 6))),
])
def test_what_a_write_reports_and_stores(cu, kv, stored, e4m3):
    b = Batch([3, 3], [200, 130], 16, 2, 64, e4m3, G=2, seed=101)
    old = {n: b.fill().pages[n].clone() for n in "kv"}
    old_scale = {n: b.scale[n].clone() if e4m3 else None for n in "kv"}
    x = b.on(DEV)
    new = {n: (b.new[n].float() * 0.25 + 8).to(torch.bfloat16) for n in "kv"}
    for i, rows in enumerate(stored):
        if rows is None:
            continue
        n_seq = cu[i + 1] - cu[i] if cu[i + 1] > cu[i] else 0
        for t in range(*rows):
            pos = kv[i] - n_seq + t - cu[i]
            at, row = oracle.paged_positions(b.table.numpy(), 16, i, np.array([pos]))
            for n in "kv":
                y = new[n][t]
                if e4m3:
                    codes, sc = oracle.quantize_rows(y.double().numpy())
                    old_scale[n][at, :, row] = torch.from_numpy(sc)[None]
                    y = torch.from_numpy(codes)
                old[n][at, :, row] = y[None]
    as_int = lambda z: torch.tensor(z, dtype=torch.int32, device=DEV)
    fa.paged_write(new["k"].to(DEV), new["v"].to(DEV), x.k, x.v, x.table, as_int(kv),
                   cu_seqlens_q=as_int(cu), **x.sc)
    torch.cuda.synchronize()
    wrong = (cu, kv) != ([0, 3, 6], [200, 130])
    assert fa.fa_device_status(clear=True) == (fa.FA_ERR_INVALID_ARG if wrong else fa.FA_OK)
    for n, got in (("k", x.k), ("v", x.v)):
        assert torch.equal(got.cpu(), old[n])
        assert not e4m3 or torch.equal(x.sc[n + "_scale"].cpu(), old_scale[n])


@pytest.mark.parametrize("e4m3", [False, True])
def test_rows_that_two_sequences_write(e4m3):
    # the second half of every sequence's page is shared by pairs: what each unit of such a row
    # holds comes from one of the two, all other rows are as written
    B, Hkv, d, page, n = 64, 4, 128, 16, 16
    g = torch.Generator().manual_seed(111)
    new = torch.randn((B * n, Hkv, d), generator=g).to(torch.bfloat16)
    table = torch.stack([torch.arange(B, dtype=torch.int32), torch.arange(B, dtype=torch.int32) // 2 + B], 1)
    c = fa.paged_cache(B + B // 2, page, Hkv, d, e4m3=e4m3, device=DEV)
    kv = torch.full((B,), 24, dtype=torch.int32, device=DEV)  # positions 8 .. 23
    fa.paged_write(new.to(DEV), -new.to(DEV), page_table=table.to(DEV), kv_lens=kv, **c)
    sync()
    for name, x in (("k", new), ("v", -new)):
        got = c[name + "_pages"].cpu()
        want = x.reshape(B, n, Hkv, d).transpose(1, 2)  # [B, Hkv, tokens, d]
        if e4m3:
            want, sc = (torch.from_numpy(t) for t in oracle.quantize_rows(want.double().numpy()))
            got_sc = c[name + "_scale"].cpu()
            assert torch.equal(got_sc[:B, :, 8:], sc[:, :, :8])
            pair = sc[:, :, 8:].reshape(B // 2, 2, Hkv, 8)
            assert ((got_sc[B:, :, :8] == pair[:, 0]) | (got_sc[B:, :, :8] == pair[:, 1])).all()
        assert torch.equal(got[:B, :, 8:], want[:, :, :8])
        pair = want[:, :, 8:].reshape(B // 2, 2, Hkv, 8, d // 8, 8)
        units = got[B:, :, :8].reshape(B // 2, Hkv, 8, d // 8, 8)
        assert ((units == pair[:, 0]).all(-1) | (units == pair[:, 1]).all(-1)).all()


# ------------------------------------------------------------------ outputs over q

def test_outputs_over_a_part_of_q_are_refused():
    b = Batch([1, 2], [20, 5], 16, 2, 64, G=2, seed=131)
    x = b.fill().on(DEV)
    n = x.q.numel()
    flat = torch.empty(4 * n, dtype=torch.bfloat16, device=DEV)
    q = flat[n:2 * n].view(x.q.shape).copy_(x.q)
    lse = torch.empty(x.q.shape[:2], device=DEV)
    call = dict(page_table=x.table, kv_lens=x.kv, cu_seqlens_q=x.cu, max_q=2, causal=True)
    for at in (n // 2, n - 8, n, n + 8, 2 * n - 8):
        with pytest.raises(ValueError):
            fa.paged_attn(q, x.k, x.v, out=(flat[at:at + n].view(q.shape), lse), **call)
    with pytest.raises(ValueError):
        over = flat[n:n + 2 * lse.numel()].view(torch.float32).view(lse.shape)
        fa.paged_attn(q, x.k, x.v, out=(torch.empty_like(q), over), **call)
    for at in (0, 2 * n):   # next to it
        out = flat[at:at + n].view(q.shape), lse
        fa.paged_attn(q, x.k, x.v, out=out, **call)
        sync()
        check_attn(*out, b.oracle(True))


# ------------------------------------------------------------------ the C mirrors

@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("nq", [[1, 2], [40, 9]])
def test_calls_with_caller_owned_buffers(nq, e4m3):
    # fa_paged_write, _attn and _read as the C entry points take their arguments
    b = Batch(nq, [700, 130], 16, 2, 64, e4m3, G=2, seed=121)
    x = b.fill(upto=[L - n for L, n in zip(b.kv, nq)]).on(DEV)
    P, Hkv, page, d = x.k.shape
    scales = (x.sc["k_scale"], x.sc["v_scale"])
    cache = (int(e4m3), P, page)
    rest = (Hkv, d, *x.k.stride()[:3], x.table, x.table.stride(0), x.table.shape[1], x.kv)
    assert fa.fa_paged_write(x.k_new, x.v_new, x.k, x.v, *scales, *cache, *rest, x.cu, 2, b.T,
                             max(nq), Hkv * d, Hkv * d) == fa.FA_OK
    o, lse = torch.empty_like(x.q), torch.empty(x.q.shape[:2], device=DEV)
    size = fa.fa_paged_workspace_size(b.H, Hkv, d, max(nq), x.table.shape[1] * page)
    ws = torch.empty(max(size, 1), dtype=torch.uint8, device=DEV)
    assert fa.fa_paged_attn(x.q, x.k, x.v, *scales, o, lse, *cache, b.H, *rest, x.cu, 2, b.T,
                            max(nq), b.H * d, d ** -0.5, True, -1, ws, size) == fa.FA_OK
    k, v = (torch.empty((2, Hkv, 700, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    assert fa.fa_paged_read(x.k, x.v, *scales, *cache, *rest, 2, 700, k, v) == fa.FA_OK
    sync()
    check_attn(o, lse, b.oracle(True))
    for n, got in (("k", k), ("v", v)):
        assert np.array_equal(got[0].double().cpu().numpy(), np.moveaxis(b.stored(n, 0), 0, 1))


@pytest.mark.parametrize("as_handle", [0, 1])
def test_a_forked_stream_inside_a_capture(as_handle):
    # outputs and workspace come from the graph's memory, also on a stream that joined its capture
    b = Batch([1, 30], [700, 300], 16, 2, 64, G=2, seed=94)
    x = b.fill().on(DEV)
    side = torch.cuda.Stream()
    call = dict(stream=handles(side)[as_handle])
    attn(b, x, causal=True, max_q=30)
    torch.cuda.synchronize()
    q = x.q.clone()
    x.q.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        o, lse = attn(b, x, causal=True, max_q=30, **call)
        k, _ = fa.paged_read(x.k, x.v, x.table, x.kv, 700, **call)
        torch.cuda.current_stream().wait_stream(side)
    x.q.copy_(q)
    for _ in range(3):
        fa.paged_attn(-q, x.k, x.v, x.table, x.kv, cu_seqlens_q=x.cu, max_q=30)
        g.replay()
        sync()
        check_attn(o, lse, b.oracle(True))
        assert np.array_equal(k[0].double().cpu().numpy(), np.moveaxis(b.stored("k", 0), 0, 1))
