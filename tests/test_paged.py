"""Paged caches on the GPU against the fp64 oracle: writing (bit for bit, quantised or not),
reading back, attention of single tokens and chunks, what the calls report from the device,
and the three together as a server uses them."""
import numpy as np
import pytest
import torch

import io_aware_exact_07_gb300 as fa
import oracle
from _paged import Batch, check_attn

pytestmark = pytest.mark.gpu
DEV = "cuda"


def sync():
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_OK


def attn(b, x, **kw):
    return fa.paged_attn(x.q, x.k, x.v, x.table, x.kv, cu_seqlens_q=x.cu, **x.sc, **kw)


def run(b, causal=True, window_left=-1, max_q=None):
    x = b.fill().on(DEV)
    rows = int(b.cu[-1])  # those of the sequences: the others are not written
    o, lse = attn(b, x, causal=causal, window_left=window_left, max_q=max_q or max(b.nq))
    sync()
    check_attn(o, lse, b.oracle(causal, window_left), rows)
    o2, lse2 = attn(b, x, causal=causal, window_left=window_left, max_q=max_q or max(b.nq))
    sync()
    assert torch.equal(o[:rows], o2[:rows]) and torch.equal(lse[:rows], lse2[:rows])
    return x, o, lse


# ------------------------------------------------------------------ write and read

@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("layout", ["head", "row", "pair"])
@pytest.mark.parametrize("nq,kv,page,Hkv,d", [
    ([1], [1], 16, 1, 64),
    ([1, 1, 1], [1, 17, 300], 16, 3, 128),
    ([5, 0, 40], [5, 0, 100], 48, 5, 64),      # odd heads, a page size that is no power of two
    ([130, 7], [130, 515], 256, 8, 128),
    ([3, 2], [2, 1], 32, 2, 64),               # more tokens than positions
])
def test_write_and_read_back(nq, kv, page, Hkv, d, layout, e4m3):
    b = Batch(nq, kv, page, Hkv, d, e4m3, layout=layout, seed=page + d, extra_rows=3, table_pad=2)
    old = [max(L - n, 0) for n, L in zip(nq, kv)]
    x = b.fill(upto=old).on(DEV)
    fa.paged_write(x.k_new, x.v_new, x.k, x.v, x.table, x.kv, cu_seqlens_q=x.cu, **x.sc)
    sync()
    b.fill()  # what the pages have to hold now, the untouched rows among them
    for n, got in (("k", x.k), ("v", x.v)):
        assert torch.equal(got.cpu(), b.pages[n])
        if e4m3:
            assert torch.equal(x.sc[n + "_scale"].cpu(), b.scale[n])
    N = max(kv) + 5
    for N in (N, max(1, max(kv) // 2)):
        out = fa.paged_read(x.k, x.v, x.table, x.kv, N, **x.sc)
        sync()
        for n, got in zip("kv", out):
            ref = np.zeros((b.B, Hkv, N, d))
            for i, L in enumerate(kv):
                ref[i, :, :min(L, N)] = np.moveaxis(b.stored(n, i)[:N], 0, 1)
            assert np.array_equal(got.double().cpu().numpy(), ref)


@pytest.mark.parametrize("d", [64, 128])
def test_quantiser_edges(d):
    g = torch.Generator().manual_seed(d)
    T, Hkv = 300, 2
    x = torch.randn((T, Hkv, d), generator=g)
    x *= torch.exp2(torch.randint(-140, 30, (T, Hkv, 1), generator=g).float())  # all magnitudes
    x = x.to(torch.bfloat16)
    x[0], x[1, 0, 5], x[2, 1, d - 1], x[3, 0, 0] = 0, float("inf"), float("nan"), -float("inf")
    x[4] = 0
    x[4, :, 7] = 448.0           # the row's largest magnitude on the border of a scale
    x[5] = x[4] * -2
    x[6] = -0.0
    x[7], x[8] = torch.finfo(torch.bfloat16).max, torch.finfo(torch.bfloat16).tiny
    # every halfway case of the format, and its neighbours, next to a 256 that sets E = 0
    mags = torch.from_numpy(oracle.e4m3_decode(np.arange(0x78, dtype=np.uint8)))
    half = ((mags[1:] + mags[:-1]) / 2).to(torch.bfloat16)
    for i in range(0, half.numel(), d - 1):
        part = half[i:i + d - 1]
        x[20 + i // (d - 1), 0, :part.numel()] = part
        x[20 + i // (d - 1), 0, part.numel():] = 0
        x[20 + i // (d - 1), 0, d - 1] = 256.0
    c = fa.paged_cache(-(-T // 16), 16, Hkv, d, e4m3=True)
    table = torch.arange(-(-T // 16), dtype=torch.int32, device=DEV)[None]
    kv = torch.tensor([T], dtype=torch.int32, device=DEV)
    fa.paged_write(x.to(DEV), -x.to(DEV), page_table=table, kv_lens=kv, **c)
    k, v = fa.paged_read(page_table=table, kv_lens=kv, N=T, **c)
    sync()
    for n, sign, back in (("k", 1, k), ("v", -1, v)):
        codes, s = oracle.quantize_rows(sign * x.double().numpy())
        got = c[n + "_pages"].transpose(1, 2).reshape(-1, Hkv, d)[:T].cpu().numpy()
        gs = c[n + "_scale"].transpose(1, 2).reshape(-1, Hkv)[:T].cpu().numpy()
        assert np.array_equal(gs, s) and np.array_equal(got, codes)
        ref = np.moveaxis(oracle.dequantize_rows(codes, s), 0, 1)[None]
        assert np.array_equal(back.double().cpu().numpy(), ref, equal_nan=True)


def test_rows_of_a_fused_projection():
    # q, k and v as slices of one [T, (H + 2 Hkv) d] tensor: token stride wider than the rows
    b = Batch([3, 4], [40, 9], 16, 2, 64, G=3, seed=8)
    x = b.fill(upto=[37, 5]).on(DEV)
    qkv = torch.cat([x.q, x.k_new, x.v_new], 1).contiguous()
    H = b.H
    fa.paged_write(qkv[:, H:H + 2], qkv[:, H + 2:], x.k, x.v, x.table, x.kv, cu_seqlens_q=x.cu)
    o, lse = fa.paged_attn(qkv[:, :H], x.k, x.v, x.table, x.kv, cu_seqlens_q=x.cu, max_q=4,
                           causal=True)
    sync()
    check_attn(o, lse, b.oracle(True))


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,Hkv,kv,page", [
    (1, 1, [1], 16),
    (1, 3, [1, 15, 16, 17, 127, 128, 129], 16),
    (4, 8, [1, 1000, 255, 77], 64),
    (8, 2, [4096, 300], 128),
    (7, 1, [513, 2050, 100], 48),
    (16, 1, [700, 16], 256),
    (17, 1, [700, 130], 32),       # more rows than a 16-row tile
    (128, 1, [300, 129], 64),      # a full query tile of heads
])
def test_single_tokens(G, Hkv, kv, page, d, e4m3):
    run(Batch([1] * len(kv), kv, page, Hkv, d, e4m3, G=G, seed=G + d))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("causal,wl", [(True, -1), (False, -1), (True, 100), (False, 37),
                                       (True, 0)])
@pytest.mark.parametrize("nq,kv,G,Hkv,page,d", [
    ([4, 2, 3, 4], [500, 2, 130, 4], 4, 2, 16, 128),        # up to 16 rows per K/V head
    ([5, 5], [1000, 5], 4, 2, 32, 64),                       # 20 rows
    ([130, 1, 64], [130, 700, 500], 3, 2, 48, 64),           # rows that do not fill a tile
    ([200, 0, 33, 1], [777, 40, 33, 1], 5, 1, 64, 128),
    ([128, 256], [128, 1300], 1, 2, 128, 128),
])
def test_chunks(nq, kv, G, Hkv, page, d, causal, wl, e4m3):
    run(Batch(nq, kv, page, Hkv, d, e4m3, G=G, seed=sum(kv) + d), causal, wl)


@pytest.mark.parametrize("d,e4m3", [(64, False), (128, False), (128, True)])
def test_long_sequences_cut_between_many_blocks(d, e4m3):
    run(Batch([1], [20001], 64, 1, d, e4m3, G=8, seed=1))
    run(Batch([3, 1], [9000, 12345], 16, 2, d, e4m3, G=2, seed=2))
    run(Batch([300], [9001], 64, 1, d, e4m3, G=2, seed=3))


def test_many_short_sequences():
    g = np.random.RandomState(5)
    kv = [int(n) for n in g.randint(0, 70, 700)]
    run(Batch([1] * 700, kv, 16, 2, 64, G=2, seed=5))
    nq = [int(g.randint(0, n + 1)) for n in kv]
    run(Batch(nq, kv, 16, 1, 128, True, G=3, seed=6))


@pytest.mark.parametrize("nq", [[1, 1, 1, 1], [40, 3, 9, 20]])
@pytest.mark.parametrize("e4m3", [False, True])
def test_rows_without_keys(nq, e4m3):
    # empty caches, and sequences with more new tokens than positions
    b = Batch(nq, [0, 2, 0, 30], 16, 2, 64, e4m3, G=2, seed=9)
    for causal in (True, False):
        x, o, lse = run(b, causal)
    if nq[0] > 1:
        assert torch.isneginf(lse[:40]).all() and (o[:40] == 0).all()


@pytest.mark.parametrize("nq,max_q", [([1, 1], 1), ([70, 3], 70)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("e4m3", [False, True])
def test_what_lies_behind_a_sequence_does_not_matter(nq, max_q, d, e4m3):
    # NaN (scale byte 255 in a quantised cache) in every row of the pool that no position of a sequence below its length takes,
    # within the last pages too
    b = Batch(nq, [130, 75], 64, 2, d, e4m3, G=2, seed=10, garbage=float("nan"), extra_rows=5)
    x = b.fill().on(DEV)
    o = torch.full((b.T, b.H, d), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((b.T, b.H), 7.0, device=DEV)
    attn(b, x, causal=True, max_q=max_q, out=(o, lse))
    sync()
    check_attn(o, lse, b.oracle(True), rows=int(b.cu[-1]))
    assert (o[b.cu[-1]:] == 7).all() and (lse[b.cu[-1]:] == 7).all()


@pytest.mark.parametrize("layout", ["row", "pair"])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("nq", [[1, 1], [150, 20]])
def test_orders_of_the_pages_in_memory(layout, e4m3, nq):
    run(Batch(nq, [200, 1050], 32, 3, 128, e4m3, G=2, seed=11, layout=layout, table_pad=1))


def test_extreme_scores():
    # scores of +-2^9 and more: the running maximum moves by hundreds between keys, and the
    # last key of one head outweighs all others
    b = Batch([1, 9], [600, 333], 16, 2, 64, G=2, seed=12)
    for n in range(2):
        b.rows["k"][n] *= 64
    b.rows["k"][0][-1] = 0
    b.rows["k"][1][200] *= 8
    x = b.fill().on(DEV)
    o, lse = attn(b, x, causal=True, max_q=9)
    o1, lse1 = fa.paged_attn(x.q[:1], x.k, x.v, x.table[:1], x.kv[:1], causal=True, max_q=1)
    sync()
    # scores up to 2^13 in fp32: off by d 2^-24 scale sum |q k| < 64 * 2^-24 * 2^13 = 2^-5
    o_ref, lse_ref, o_abs = b.oracle(True)
    for got, gl, rows in ((o, lse, slice(0, 10)), (o1, lse1, slice(0, 1))):
        tol = (np.exp(2.0 ** -4) - 1 + 2.0 ** -7) * (o_abs[rows] + np.abs(o_ref[rows]))
        assert np.all(np.abs(got.double().cpu().numpy() - o_ref[rows]) <= tol)
        assert np.abs(gl.double().cpu().numpy() - lse_ref[rows]).max() <= 2.0 ** -5


def test_pool_larger_than_32_bit_offsets():
    # pages at the far end of a pool of 2^32 + elements (bf16 and e4m3), K and V one pool each
    for e4m3 in (False, True):
        b = Batch([1, 40], [300, 100], 64, 2, 128, e4m3, G=2, seed=13)
        far = (1 << 32) // (64 * 2 * 128) + 7
        x = b.fill().on(DEV)
        c = fa.paged_cache(far + b.P, 64, 2, 128, e4m3=e4m3)
        for n, small in (("k", x.k), ("v", x.v)):
            c[n + "_pages"][far:] = small
            if e4m3:
                c[n + "_scale"][far:] = x.sc[n + "_scale"]
        table = torch.where(x.table >= 0, x.table + far, x.table)
        fa.paged_write(x.k_new, x.v_new, page_table=table, kv_lens=x.kv, cu_seqlens_q=x.cu, **c)
        k, v = fa.paged_read(page_table=table, kv_lens=x.kv, N=300, **c)
        o, lse = fa.paged_attn(x.q, page_table=table, kv_lens=x.kv, cu_seqlens_q=x.cu, max_q=40,
                               causal=True, **c)
        o1, lse1 = fa.paged_attn(x.q[:1], page_table=table[:1], kv_lens=x.kv[:1], max_q=1, **c)
        sync()
        ref = b.oracle(True)
        check_attn(o, lse, ref)
        check_attn(o1, lse1, tuple(r[:1] for r in ref))
        assert np.array_equal(k[0].double().cpu().numpy(), np.moveaxis(b.stored("k", 0), 0, 1))
        assert np.array_equal(v[1, :, :100].double().cpu().numpy(),
                              np.moveaxis(b.stored("v", 1), 0, 1))
        del c, k, v
        torch.cuda.empty_cache()


# ------------------------------------------------------------------ reported from the device

def reported():
    torch.cuda.synchronize()
    return fa.fa_device_status(clear=True)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("nq", [[1, 1, 1], [40, 2, 33]])
def test_pages_out_of_range_are_reported_and_not_touched(nq, e4m3):
    b = Batch(nq, [200, 130, 300], 16, 2, 64, e4m3, G=2, seed=14)
    x = b.fill().on(DEV)
    before = x.k.clone(), x.v.clone()
    good, _ = attn(b, x, causal=True, max_q=max(nq))
    for page in (-1, b.P, 1 << 30, -(1 << 31)):
        bad = x.table.clone()
        bad[1, 130 // 16] = page       # the page of the sequence's last positions
        o, lse = fa.paged_attn(x.q, x.k, x.v, bad, x.kv, cu_seqlens_q=x.cu, max_q=max(nq),
                               causal=True, **x.sc)
        assert reported() == fa.FA_ERR_INVALID_ARG
        c = b.cu
        for i in (0, 2):               # the other sequences are as they were
            assert torch.equal(o[c[i]:c[i + 1]], good[c[i]:c[i + 1]])
        assert torch.isfinite(o.float()).all() and torch.isfinite(lse).all()
        fa.paged_write(x.k_new, x.v_new, x.k, x.v, bad, x.kv, cu_seqlens_q=x.cu, **x.sc)
        assert reported() == fa.FA_ERR_INVALID_ARG
        assert torch.equal(x.k, before[0]) and torch.equal(x.v, before[1])
        k, _ = fa.paged_read(x.k, x.v, bad, x.kv, 300, **x.sc)
        assert reported() == fa.FA_ERR_INVALID_ARG
        assert (k[1, :, 128:130] == 0).all() and (k[1, :, 127] != 0).any()


@pytest.mark.parametrize("bad", [dict(kv=[200, -1]), dict(kv=[200, 10 ** 6]), dict(cu=[0, 5, 3]),
                                 dict(cu=[0, -2, 6]), dict(cu=[0, 3, 1000]), dict(max_q=2)])
def test_lengths_and_offsets_out_of_range_are_reported(bad):
    b = Batch([3, 3], [200, 130], 16, 2, 64, G=2, seed=15)
    x = b.fill().on(DEV)
    before = x.k.clone()
    kv = torch.tensor(bad.get("kv", b.kv), dtype=torch.int32, device=DEV)
    cu = torch.tensor(bad.get("cu", list(b.cu)), dtype=torch.int32, device=DEV)
    for max_q in ((bad["max_q"],) if "max_q" in bad else (6, 64)):
        fa.paged_attn(x.q, x.k, x.v, x.table, kv, cu_seqlens_q=cu, max_q=max_q, causal=True)
        assert reported() == fa.FA_ERR_INVALID_ARG
    if "max_q" not in bad:
        zero = torch.zeros_like(x.k_new)
        fa.paged_write(zero, zero, x.k, x.v, x.table, kv, cu_seqlens_q=cu)
        assert reported() in (fa.FA_ERR_INVALID_ARG, fa.FA_OK)  # tokens of no sequence: nothing read
        if "kv" in bad:
            keep = x.table[1].long().clamp(min=0)
            assert torch.equal(x.k[keep], before[keep])  # the second sequence is as it was


# ------------------------------------------------------------------ streams, graphs, together

def test_a_captured_step_is_replayed_with_other_lengths():
    # a server's step, write and attention, captured once; lengths, tokens and tables change
    for e4m3 in (False, True):
        b = Batch([1, 1, 1], [900, 40, 333], 16, 2, 128, e4m3, G=4, seed=16)
        x = b.fill(upto=[L - 1 for L in b.kv]).on(DEV)
        kv = x.kv.clone()
        o = torch.empty((3, 8, 128), dtype=torch.bfloat16, device=DEV)
        lse = torch.empty((3, 8), device=DEV)

        def step():
            fa.paged_write(x.k_new, x.v_new, x.k, x.v, x.table, kv, **x.sc)
            fa.paged_attn(x.q, x.k, x.v, x.table, kv, max_q=1, causal=True, out=(o, lse), **x.sc)
        step()
        sync()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        for lens in (b.kv, [17, 40, 1], b.kv):
            c = Batch([1, 1, 1], lens, 16, 2, 128, e4m3, G=4, seed=16)
            c.q = b.q
            c.rows = {n: [r[:L].clone() for r, L in zip(b.rows[n], lens)] for n in "kv"}
            kv.copy_(torch.tensor(lens, dtype=torch.int32))
            for n, new in (("k", x.k_new), ("v", x.v_new)):
                new.copy_(torch.stack([r[L - 1] for r, L in zip(b.rows[n], lens)]))
            g.replay()
            sync()
            check_attn(o, lse, c.oracle(True))


def test_two_graphs_and_an_eager_call_share_a_workspace():
    lib = fa.load()
    b = Batch([1, 2], [3000, 100], 16, 2, 64, G=4, seed=17)
    c = Batch([60, 5], [2000, 70], 16, 2, 64, G=4, seed=18)
    xs = [y.fill().on(DEV) for y in (b, c)]
    need = max(fa.fa_paged_workspace_size(8, 2, 64, n, 1 << 20) for n in (2, 60))
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    outs = [(torch.empty_like(x.q), torch.empty(x.q.shape[:2], device=DEV)) for x in xs]

    def call(y, x, out, n):
        P, Hkv, page, d = x.k.shape
        st = lib.fa_paged_attn(x.q.data_ptr(), x.k.data_ptr(), x.v.data_ptr(), None, None,
                               out[0].data_ptr(), out[1].data_ptr(), 0, P, page, y.H, Hkv, d,
                               *x.k.stride()[:3], x.table.data_ptr(), x.table.stride(0),
                               x.table.shape[1], x.kv.data_ptr(), x.cu.data_ptr(), y.B, y.T, n,
                               y.H * d, 0.125, 1, -1, ws.data_ptr(), ws.numel(),
                               torch.cuda.current_stream().cuda_stream)
        assert st == fa.FA_OK
    calls = [lambda: call(b, xs[0], outs[0], 2), lambda: call(c, xs[1], outs[1], 60)]
    for f in calls:
        f()
    torch.cuda.synchronize()
    graphs = []
    for f in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            f()
    for _ in range(3):
        ws.random_(0, 256)
        for o, lse in outs:
            o.fill_(9)
            lse.fill_(9)
        graphs[0].replay()
        calls[1]()
        graphs[1].replay()
        graphs[0].replay()
        sync()
        for y, (o, lse) in zip((b, c), outs):
            check_attn(o, lse, y.oracle(True))


def test_on_another_stream():
    b = Batch([1, 30], [2500, 700], 64, 2, 128, G=2, seed=19)
    x = b.fill(upto=[2499, 670]).on(DEV)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        fa.paged_write(x.k_new, x.v_new, x.k, x.v, x.table, x.kv, cu_seqlens_q=x.cu, stream=stream)
        o, lse = attn(b, x, causal=True, max_q=30, stream=stream)
        k, v = fa.paged_read(x.k, x.v, x.table, x.kv, 2500, stream=stream)
        side.synchronize()
        assert fa.fa_device_status(side) == fa.FA_OK
        check_attn(o, lse, b.oracle(True))
        assert np.array_equal(k[0].double().cpu().numpy(), np.moveaxis(b.stored("k", 0), 0, 1))


def test_two_calls_at_once():
    b = Batch([1, 2], [30000, 100], 16, 2, 64, G=4, seed=20)
    c = Batch([600, 5], [2000, 70], 16, 2, 64, G=4, seed=21)
    xs = [y.fill().on(DEV) for y in (b, c)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    outs = []
    for _ in range(4):
        for y, x, s in zip((b, c), xs, streams):
            outs.append((y, attn(y, x, causal=True, max_q=max(y.nq), stream=s)))
    sync()
    for y in (b, c):
        ref = y.oracle(True)
        for z, (o, lse) in outs:
            if z is y:
                check_attn(o, lse, ref)


@pytest.mark.parametrize("e4m3", [False, True])
def test_prefill_then_steps_then_read_back(e4m3):
    # a server's run: two prompts enter in chunks, then tokens one by one; every output equals
    # attention over all that was written, and the cache read back feeds decode
    d, Hkv, G, page = 128, 2, 4, 16
    total = [301, 150]
    b = Batch(total, total, page, Hkv, d, e4m3, G=G, seed=22)
    whole = b.oracle(True)
    x = b.on(DEV)
    done = [0, 0]
    for take in ([128, 100], [128, 45], [40, 0], [1, 1], [1, 1], [1, 1], [2, 2]):
        cu = np.concatenate([[0], np.cumsum(take)])
        rows = np.concatenate([np.arange(b.cu[i] + done[i], b.cu[i] + done[i] + n)
                               for i, n in enumerate(take)])
        at = torch.from_numpy(rows).to(DEV)
        done = [n + m for n, m in zip(done, take)]
        cud = torch.tensor(cu, dtype=torch.int32, device=DEV)
        kv = torch.tensor(done, dtype=torch.int32, device=DEV)
        fa.paged_write(x.k_new[at], x.v_new[at], x.k, x.v, x.table, kv, cu_seqlens_q=cud, **x.sc)
        o, lse = fa.paged_attn(x.q[at], x.k, x.v, x.table, kv, cu_seqlens_q=cud,
                               max_q=max(take), causal=True, **x.sc)
        sync()
        check_attn(o, lse, tuple(r[rows] for r in whole))
    assert done == total
    k, v = fa.paged_read(x.k, x.v, x.table, kv, 301, **x.sc)
    last = torch.stack([x.q[b.cu[i + 1] - 1] for i in range(2)])[:, :, None]
    o, lse = fa.decode(last.contiguous(), k, v, seqlens_k=kv)
    sync()
    ends = [int(b.cu[1]) - 1, int(b.cu[2]) - 1]
    check_attn(o[:, :, 0], lse[:, :, 0], tuple(r[ends] for r in whole))


def test_workspace_is_checked():
    lib = fa.load()
    b = Batch([1, 1], [3000, 40], 16, 2, 64, G=2, seed=24)
    x = b.fill().on(DEV)
    o, lse = torch.empty_like(x.q), torch.empty((2, 4), device=DEV)
    P, Hkv, page, d = x.k.shape
    need = fa.fa_paged_workspace_size(4, 2, 64, 1, x.table.shape[1] * page)
    assert need > 0 and fa.fa_paged_workspace_size(4, 3, 64, 1, 100) == 0
    ws = torch.empty(need + 16, dtype=torch.uint8, device=DEV)
    for at, size, status in ((None, need, 4), (ws.data_ptr(), need - 1, 4),
                             (ws.data_ptr() + 8, need, 4), (ws.data_ptr(), need, 0)):
        assert lib.fa_paged_attn(x.q.data_ptr(), x.k.data_ptr(), x.v.data_ptr(), None, None,
                                 o.data_ptr(), lse.data_ptr(), 0, P, page, 4, Hkv, d,
                                 *x.k.stride()[:3], x.table.data_ptr(), x.table.stride(0),
                                 x.table.shape[1], x.kv.data_ptr(), x.cu.data_ptr(), 2, 2, 1,
                                 4 * d, 0.125, 1, -1, at, size,
                                 torch.cuda.current_stream().cuda_stream) == status
    sync()
    check_attn(o, lse, b.oracle(True))


def test_binding_refusals_on_the_gpu():
    b = Batch([1, 2], [20, 5], 16, 2, 64, True, G=2, seed=23)
    x = b.fill().on(DEV)
    base = dict(q=x.q, k_pages=x.k, v_pages=x.v, page_table=x.table, kv_lens=x.kv,
                cu_seqlens_q=x.cu, max_q=2, **x.sc)
    fa.paged_attn(**base)
    fa.paged_attn(**dict(base, k_pages=x.k.view(torch.float8_e4m3fn),
                         v_pages=x.v.view(torch.float8_e4m3fn)))
    sync()
    for bad in (dict(q=x.q.float()), dict(q=x.q[:, :, :32]), dict(q=x.q[0]), dict(k_scale=None),
                dict(q=x.q.transpose(0, 1).contiguous().transpose(0, 1)),
                dict(v_scale=x.sc["v_scale"][:, :, :8]), dict(v_scale=x.sc["v_scale"].int()),
                dict(kv_lens=x.kv.long()), dict(kv_lens=x.kv[:1]), dict(kv_lens=x.kv.cpu()),
                dict(page_table=x.table.long()), dict(page_table=x.table[0]),
                dict(page_table=x.table.t().contiguous().t()), dict(cu_seqlens_q=x.cu[:2]),
                dict(cu_seqlens_q=x.cu.cpu()), dict(cu_seqlens_q=None, max_q=1),
                dict(q=x.q.cpu()), dict(out=(x.q[:2], torch.empty((3, 4), device=DEV))),
                dict(out=(torch.empty_like(x.q), torch.empty((3, 4), device=DEV).half()))):
        with pytest.raises(ValueError):
            fa.paged_attn(**dict(base, **bad))
    for bad in (dict(q=x.q[:, :3]), dict(scale=0.0), dict(window_left=-3), dict(max_q=0)):
        with pytest.raises((fa.FAError, ValueError)):
            fa.paged_attn(**dict(base, **bad))
    sync()


# ------------------------------------------------------------------ more shapes and values

@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq,G,Hkv,kv,page", [
    ([5, 8, 1], 4, 2, [1000, 8, 300], 32),     # 17 to 32 rows per K/V head
    ([1, 1], 17, 2, [700, 129], 48),
    ([2, 3], 10, 1, [260, 2], 16),
    ([1, 1, 1], 32, 1, [4000, 15, 16], 128),
    ([8, 1, 4], 4, 1, [3000, 1, 200], 64),     # 32 rows, cut between CTAs
])
def test_up_to_32_rows(nq, G, Hkv, kv, page, d, e4m3):
    run(Batch(nq, kv, page, Hkv, d, e4m3, G=G, seed=sum(kv) + G))


@pytest.mark.parametrize("d,e4m3", [(64, False), (64, True), (128, False), (128, True)])
def test_chunks_of_many_query_tiles(d, e4m3):
    # more query tiles than CTAs: whole tiles in rounds, then runs that are cut
    run(Batch([1300], [1500], 64, 8, d, e4m3, G=2, seed=31))
    run(Batch([700, 1, 0, 333], [705, 2000, 40, 333], 16, 4, d, e4m3, G=3, seed=32), True, 200)


@pytest.mark.parametrize("e4m3", [False, True])
def test_fewer_query_tiles_than_ctas(e4m3):
    # one or two heads' query tiles over a long cache: every tile is cut, each CTA's run ends
    # inside the next
    run(Batch([200], [8111], 128, 2, 64, e4m3, G=4, seed=33))
    run(Batch([64, 40], [3000, 9000], 16, 1, 128, e4m3, G=8, seed=34), False)


@pytest.mark.parametrize("seed", range(24))
def test_random_batches(seed):
    g = np.random.RandomState(1000 + seed)
    B = int(g.choice([1, 2, 5, 30]))
    top = int(g.choice([40, 300, 1500]))
    kv = [int(n) for n in g.randint(0, top + 1, B)]
    most = int(g.choice([1, 3, 9, 70]))
    nq = [int(min(g.randint(0, most + 1), n + 2)) for n in kv]
    nq[int(g.randint(B))] = most
    b = Batch(nq, kv, int(g.choice([16, 32, 80, 256])), int(g.choice([1, 2, 3])),
              int(g.choice([64, 128])), bool(g.randint(2)), G=int(g.choice([1, 2, 5, 8])),
              seed=seed, layout=str(g.choice(["head", "row", "pair"])),
              extra_rows=int(g.randint(3)), table_pad=int(g.randint(3)))
    run(b, bool(g.randint(2)), int(g.choice([-1, -1, 0, 17, 130])))


def test_batches_without_new_tokens():
    b = Batch([0, 0, 0], [40, 0, 7], 16, 2, 64, G=2, seed=35, extra_rows=9)
    x = b.fill().on(DEV)
    before = x.k.clone()
    for n in (1, 8, 100):   # each of the kernels
        out = (torch.full_like(x.q, 5.0), torch.full(x.q.shape[:2], 5.0, device=DEV))
        attn(b, x, causal=True, max_q=n, out=out)
        assert all((t == 5).all() for t in out)
    fa.paged_write(x.k_new, x.v_new, x.k, x.v, x.table, x.kv, cu_seqlens_q=x.cu)
    sync()
    assert torch.equal(x.k, before)


@pytest.mark.parametrize("nq", [[1, 1], [4, 6], [60, 33]])
@pytest.mark.parametrize("d", [64, 128])
def test_quantised_rows_of_very_different_magnitude(nq, d):
    # scales of neighbouring keys differ by up to 2^45; an absolute error of 2^-25 of the
    # largest scale 2^E per key is what the tile conversion may add, and 2^-25 times 448 of it
    # what the rounding of P to f16 may
    g = torch.Generator().manual_seed(d)
    b = Batch(nq, [700, 300], 16, 2, d, True, G=4, seed=36)
    for i in range(2):
        n = b.rows["k"][i].shape[0]
        e = torch.randint(-24, 1, (n, 2, 1), generator=g)
        b.rows["k"][i] = (b.rows["k"][i].float() * torch.exp2(e.float())).to(torch.bfloat16)
        e = torch.randint(-40, 6, (n, 2, 1), generator=g)
        b.rows["v"][i] = (b.rows["v"][i].float() * torch.exp2(e.float())).to(torch.bfloat16)
    x = b.fill().on(DEV)
    o, lse = attn(b, x, causal=True, max_q=max(nq))
    sync()
    o_ref, lse_ref, o_abs = b.oracle(True)
    top = 2.0 ** max(int(s.max()) - 127 for s in [b.scale["v"][b.scale["v"] != 133]])
    tol = 1.05 * 2.0 ** -8 * (o_abs + np.abs(o_ref)) + 700 * 449 * 2.0 ** -25 * top
    assert np.all(np.abs(o.double().cpu().numpy() - o_ref) <= tol)
    assert np.abs(lse.double().cpu().numpy() - lse_ref).max() <= 2e-4


@pytest.mark.parametrize("nq", [[1, 1], [60, 33]])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("q_exp,k_exp,v_exp", [(20, -20, 0), (-60, 0, 0), (0, 0, -30), (-15, 12, 4),
                                               (0, -40, 0)])
def test_magnitudes_of_queries_keys_and_values(q_exp, k_exp, v_exp, nq, e4m3):
    b = Batch(nq, [300, 170], 16, 2, 128, e4m3, G=2, seed=37)
    by = lambda t, e: (t.float() * 2.0 ** e).to(torch.bfloat16)
    b.q = by(b.q, q_exp)
    for n, e in (("k", k_exp), ("v", v_exp)):
        b.rows[n] = [by(t, e) for t in b.rows[n]]
    run(b)


@pytest.mark.parametrize("nq", [[1, 1], [60, 33]])
def test_rows_that_hold_a_nan(nq):
    # a NaN among a quantised sequence's keys or values reaches that sequence's rows alone
    for n in "kv":
        b = Batch(nq, [300, 170], 16, 1, 64, True, G=2, seed=38)
        b.rows[n][0][5, 0, 3] = float("nan")
        x = b.fill().on(DEV)
        o, lse = attn(b, x, causal=True, max_q=max(nq))
        sync()
        assert torch.isnan(o[:nq[0]]).all()
        b.rows[n][0][5, 0, 3] = 1.0
        ref = b.oracle(True)
        check_attn(o[nq[0]:], lse[nq[0]:], tuple(r[nq[0]:] for r in ref))


@pytest.mark.parametrize("d,e4m3", [(64, False), (128, False), (64, True), (128, True)])
def test_stalled_chunk_times_out_and_the_next_call_is_right(d, e4m3):
    b = Batch([90, 3], [700, 300], 16, 2, d, e4m3, G=2, seed=39)
    x = b.fill().on(DEV)
    sync()
    fa.fa_set_wait_timeout_ns(200_000_000)
    try:
        fa.fa_test_inject_stall(1)
        attn(b, x, causal=True, max_q=90)
        assert reported() == fa.FA_ERR_TIMEOUT
    finally:
        fa.fa_test_inject_stall(0)
        fa.fa_set_wait_timeout_ns(4_000_000_000)
    o, lse = attn(b, x, causal=True, max_q=90)
    sync()
    check_attn(o, lse, b.oracle(True))


@pytest.mark.parametrize("kv", [[700] * 17, [700] * 16 + [840], [700] * 16 + [900], [700] * 15,
                                [700] * 16 + [0], [700] * 19, [700] * 20])
def test_about_one_head_per_cta(kv):
    # the choice between a head per CTA and heads cut into equal runs, on both sides
    run(Batch([1] * len(kv), kv, 32, 8, 128, G=2, seed=41, table_pad=2))
    run(Batch([3] * len(kv), kv, 32, 8, 128, G=4, seed=42, table_pad=2), True, 600)


@pytest.mark.parametrize("nq", [1, 640])
def test_many_small_weights_beside_a_large_one(nq):
    # one key with a score of 18 above the other 65535, whose values are 1 and its own 0 (but one): O =
    # w / (1 + w) with w = 65535 e^-18, about 2^-10. Each weight may be off by 2^-32 of the
    # largest (and P and O by bf16's half step, as elsewhere).
    n, page, G = 65536, 256, 32
    k = torch.zeros(n, 1, 64)
    k[0] = 2.25
    v = torch.ones(n, 1, 64)
    v[0, 0, 1:] = 0.0   # (the row's scale is that of the others)
    c = fa.paged_cache(n // page, page, 1, 64, e4m3=True, device=DEV)
    table = torch.arange(n // page, dtype=torch.int32, device=DEV).reshape(1, -1)
    kv = torch.tensor([n], dtype=torch.int32, device=DEV)
    fa.paged_write(k.to(torch.bfloat16).to(DEV), v.to(torch.bfloat16).to(DEV), page_table=table,
                   kv_lens=kv, **c)
    q = torch.ones(nq, G, 64, dtype=torch.bfloat16, device=DEV)
    o, lse = fa.paged_attn(q, page_table=table, kv_lens=kv, max_q=nq, causal=False, **c)
    sync()
    w = (n - 1) * np.exp(-18.0)
    ref = w / (1 + w)
    assert (o[..., 1:].double() - ref).abs().max().item() <= 1.05 * 2.0 ** -7 * ref + n * 2.0 ** -32
    assert (lse.double() - 18 - np.log1p(w)).abs().max().item() <= 2e-4


@pytest.mark.parametrize("order", ["first", "last", "between", "two"])
def test_chunks_among_many_single_tokens(order):
    # units of more than 32 sequences lie between those of a chunk
    g = np.random.RandomState(len(order))
    one = [1] * 150
    nq = {"first": [300] + one, "last": one + [300], "between": one[:70] + [150, 0, 0] + one[70:],
          "two": [130] + one[:90] + [200] + one[:3]}[order]
    kv = [int(n) + int(g.randint(1, 200)) for n in nq]
    run(Batch(nq, kv, 16, 2, 64, G=4, seed=43, extra_rows=2))
    run(Batch(nq, kv, 32, 1, 128, True, G=8, seed=44), True, 60)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("nq", [[5, 2], [60, 40]])
def test_windows_wider_than_any_sequence(nq, causal):
    # more new tokens than positions too: some stand at negative ones
    b = Batch(nq, [3, 40], 16, 2, 64, G=2, seed=45)
    x = b.fill().on(DEV)
    ref = b.oracle(causal)
    for wl in (48, 2 ** 31 - 1, 2 ** 32):
        o, lse = attn(b, x, causal=causal, window_left=wl, max_q=max(nq))
        sync()
        check_attn(o, lse, ref)


def test_batches_without_sequences_or_pages_are_refused():
    c = fa.paged_cache(2, 16, 1, 64, device=DEV)
    for B, width in ((0, 3), (2, 0)):
        with pytest.raises(ValueError):
            fa.paged_attn(torch.zeros(B, 1, 64, dtype=torch.bfloat16, device=DEV),
                          page_table=torch.zeros(B, width, dtype=torch.int32, device=DEV),
                          kv_lens=torch.zeros(B, dtype=torch.int32, device=DEV), **c)


def test_output_in_place_of_q_is_refused():
    b = Batch([1, 2], [20, 5], 16, 2, 64, G=2, seed=46)
    x = b.fill().on(DEV)
    with pytest.raises(ValueError):
        attn(b, x, causal=True, max_q=2, out=(x.q, torch.empty(x.q.shape[:2], device=DEV)))


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_captured_chunk_is_replayed_with_other_lengths_and_offsets(e4m3):
    # one capture for 64 packed rows of up to 60 per sequence; rows and lengths move between
    # the sequences, some get none
    pool = Batch([64, 64, 64], [900, 700, 500], 16, 2, 64, e4m3, G=2, seed=47)
    x = pool.fill().on(DEV)
    q = x.q[:64].clone()
    kv, cu = x.kv.clone(), torch.tensor([0, 30, 60, 64], dtype=torch.int32, device=DEV)
    out = (torch.empty_like(q), torch.empty(q.shape[:2], device=DEV))

    def call():
        fa.paged_attn(q, x.k, x.v, x.table, kv, cu, max_q=60, causal=True, out=out, **x.sc)
    call()
    sync()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for nq, lens in (([30, 30, 4], [900, 700, 500]), ([0, 60, 4], [900, 61, 5]),
                     ([1, 2, 60], [640, 128, 127]), ([7, 0, 0], [7, 0, 300])):
        c = Batch(nq, lens, 16, 2, 64, e4m3, G=2, seed=47)
        c.q = pool.q[:64]
        for n in "kv":
            c.rows[n] = [r[:L] for r, L in zip(pool.rows[n], lens)]
        kv.copy_(torch.tensor(lens, dtype=torch.int32))
        cu.copy_(torch.tensor(np.concatenate([[0], np.cumsum(nq)]), dtype=torch.int32))
        g.replay()
        sync()
        check_attn(*out, c.oracle(True), rows=sum(nq))


@pytest.mark.parametrize("d", [64, 128])
def test_every_finite_magnitude_as_a_rows_largest(d):
    # exponent and codes are exact: compared with the oracle's bit by bit
    g = torch.Generator().manual_seed(d)
    top = torch.arange(0x7F80, dtype=torch.int32)  # bf16 bits
    n = top.numel()
    bits = torch.minimum((torch.rand(n, d, generator=g) * (top[:, None] + 1)).to(torch.int32),
                         top[:, None])
    bits += torch.randint(0, 2, (n, d), generator=g).to(torch.int32) * -32768
    bits[torch.arange(n), torch.randint(0, d, (n,), generator=g)] = top
    x = bits.to(torch.int16).view(torch.bfloat16).reshape(n, 1, d)
    P = -(-n // 256)
    c = fa.paged_cache(P, 256, 1, d, e4m3=True, device=DEV)
    fa.paged_write(x.to(DEV), x.to(DEV), kv_lens=torch.tensor([n], dtype=torch.int32, device=DEV),
                   page_table=torch.arange(P, dtype=torch.int32, device=DEV).reshape(1, P), **c)
    sync()
    codes, scale = oracle.quantize_rows(x.double().numpy())
    for name in "kv":
        got = c[name + "_pages"].cpu().numpy().reshape(P * 256, 1, d)[:n]
        assert np.array_equal(got, codes)
        assert np.array_equal(c[name + "_scale"].cpu().numpy().reshape(-1, 1)[:n], scale)
