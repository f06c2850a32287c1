"""Attention with keys of another length and a learned bias by relative position (fwd, bwd and
decode with k of another length, q_offset and rel_bias) against the definition in 64 bits."""
import math

import pytest
import torch

import oracle
import io_aware_exact_07_gb300 as fa
from _cross import bucket, keep_bits, plain, table_grad, within

gpu = pytest.mark.gpu
LSE_TOL = 5e-4  # 128 products of at most 2^7 in all, scaled by 1/8: 128 * 2^-23 * 2^7 / 8 = 2.4e-4,
                # and as much again for the bias, the exponents and the logarithm


def draw(B, H, Hkv, Nq, Nk, d, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)
    return (r(B, H, Nq, d), r(B, Hkv, Nk, d), r(B, Hkv, Nk, d), r(B, H, Nq, d))


def check(B, H, Hkv, Nq, Nk, d, causal=False, q_offset=0, window=(-1, -1), lens=None, p=0.0,
          rule=None, clip=None, table_type=torch.float32, seed=0, junk=None, table=None):
    """One forward and backward pass; rule: (num_buckets, max_distance, both) or clip: (left,
    right), a table row per distance; junk: what the padding of k and v holds."""
    q, k, v, do = draw(B, H, Hkv, Nq, Nk, d, seed)
    if junk is not None:
        for b, n in enumerate(lens):
            k[b, :, n:] = junk
            v[b, :, n:] = junk
    buckets = rel = bias = None
    if rule is not None:
        buckets = fa.rel_buckets(*rule)
        row = lambda x: bucket(rule, x)
        rows = rule[0]
    elif clip is not None:
        m = torch.arange(sum(clip) + 1, dtype=torch.int32, device="cuda")
        buckets = fa.RelBuckets(m, clip[0], sum(clip) + 1)
        row = lambda x: max(-clip[0], min(x, clip[1])) + clip[0]
        rows = sum(clip) + 1
    if buckets is not None:
        if table is None:
            g = torch.Generator().manual_seed(seed + 1)
            table = torch.randn((rows, H), generator=g).mul(2).to(table_type)
        rel = fa.rel_bias(table.cuda(), buckets)
        far = Nq + Nk + abs(q_offset)
        of = torch.tensor([row(x) for x in range(-far, far + 1)])
        bias = lambda h, x: table[:, h].double()[of[x + far]]
    lens_dev = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    kw = dict(causal=causal, q_offset=q_offset, window=window, seqlens_k=lens_dev, dropout_p=p,
              seed=(5 << 32) + 3, offset=7, rel_bias=rel)
    dev = [x.cuda() for x in (q, k, v, do)]
    o, lse = fa.fwd(*dev[:3], **kw)
    grads = fa.bwd(*dev[:3], o, dev[3], lse, **kw)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_OK
    keep = keep_bits(B, H, Nq, Nk, p, (5 << 32) + 3, 7) if p > 0 else None
    want, tol = plain(q, k, v, do, causal=causal, q_offset=q_offset, window=window, lens=lens,
                      bias=bias, keep=keep, p8=oracle.p8(p))
    none = want["lse"].isinf()
    got_lse = lse.cpu().double()
    assert torch.equal(got_lse[none], want["lse"][none])
    assert (got_lse - want["lse"])[~none].abs().max().item() <= LSE_TOL if (~none).any() else True
    within("o", o, want["o"], tol["o"])
    for n, x in zip(("dq", "dk", "dv"), grads):
        within(n, x, want[n], tol[n])
    assert o.cpu()[none].eq(0).all() and grads[0].cpu()[none].eq(0).all()
    if rel is not None:
        pos = torch.arange(Nq).expand(B, Nq) + q_offset
        dt, bound = table_grad(want, tol, row, rows, pos)
        got = grads[3].cpu().double()
        assert got.shape == dt.shape
        over = (got - dt).abs() - bound
        assert over.max() <= 0, (over.max(), (got - dt).abs().max())
    return (o, lse) + tuple(grads)


# ---------------------------------------------------------------- keys of another length

@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,Nk", [(1, 1), (1, 130), (130, 1), (33, 100), (128, 256), (300, 129),
                                   (257, 640)])
def test_lengths(Nq, Nk, d):
    check(1, 2, 2, Nq, Nk, d, seed=Nq + Nk)


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_offset", [-140, -1, 0, 1, 127, 128, 200, 500])
def test_causal_with_an_offset(q_offset, d):
    check(1, 2, 1, 200, 400, d, causal=True, q_offset=q_offset, seed=q_offset + 200)


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window", [(0, 0), (100, -1), (-1, 30), (130, 5), (2 ** 31 - 1, 2 ** 30)])
def test_windows_with_an_offset(window, d):
    check(1, 1, 1, 150, 420, d, q_offset=177, window=window, seed=3)


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("junk", [None, math.nan, math.inf])
def test_padding_of_any_content(d, junk):
    check(4, 4, 2, 70, 300, d, lens=[0, 1, 200, 300], junk=junk, seed=4)


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_padding_with_causal_rows_that_see_nothing(d):
    check(3, 2, 2, 200, 260, d, causal=True, q_offset=-60, lens=[5, 128, 259], junk=math.nan, seed=5)


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_grouped_heads_and_dropout(d):
    check(2, 6, 2, 140, 200, d, p=0.2, lens=[77, 200], seed=6)


# few key tiles, whose query tiles are shared among CTAs: of one and several query heads, with masks
# that leave some tiles and CTAs nothing
@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", [
    dict(B=1, H=2, Hkv=2, Nq=2500, Nk=95), dict(B=2, H=6, Hkv=2, Nq=900, Nk=200, lens=[0, 150]),
    dict(B=1, H=4, Hkv=1, Nq=1300, Nk=300, causal=True, q_offset=-700),
    dict(B=1, H=1, Hkv=1, Nq=5000, Nk=260, window=(100, 60), q_offset=-400),
    dict(B=2, H=2, Hkv=2, Nq=1700, Nk=130, p=0.2, lens=[130, 40]),
    dict(B=2, H=4, Hkv=4, Nq=1500, Nk=150, lens=[129, 3], rule=(8, 100, True), junk=math.nan),
    dict(B=1, H=3, Hkv=1, Nq=1100, Nk=270, causal=True, q_offset=20, rule=(32, 128, False)),
    dict(B=1, H=1, Hkv=1, Nq=8200, Nk=1)])
def test_few_key_tiles_and_many_queries(case, d):
    check(d=d, seed=60, **case)


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", [dict(Nk=5), dict(Nk=128, rule=(8, 16, True)), dict(Nk=2, p=0.3),
                                  dict(Nk=300, lens=[3, 300, 0], rule=(8, 16, True)),
                                  dict(Nk=300, causal=True, q_offset=-40),
                                  dict(Nk=900, window=(20, 10), q_offset=300)])
def test_few_keys_lose_nothing_to_the_rounding_of_o(case, d):
    """Rows that see one key tile: dQ and dK are off by what dS and they themselves are rounded,
    2^-8 of each at most, not by what the rounded O would cost D."""
    case = dict(case)
    Nk, p, lens = case.pop("Nk"), case.pop("p", 0.0), case.pop("lens", [300] * 3)
    rule, window = case.pop("rule", None), case.get("window", (-1, -1))
    q, k, v, do = draw(3, 2, 2, 150, Nk, d, seed=50)
    lens = [min(n, Nk) for n in lens]
    kw = dict(case, seqlens_k=torch.tensor(lens, dtype=torch.int32, device="cuda"), dropout_p=p,
              seed=3)
    bias = None
    if rule is not None:
        table = torch.randn((rule[0], 2), generator=torch.Generator().manual_seed(1))
        kw["rel_bias"] = fa.rel_bias(table.cuda(), fa.rel_buckets(*rule))
        of = torch.tensor([bucket(rule, x) for x in range(-600, 601)])
        bias = lambda h, x: table[:, h].double()[of[x + 600]]
    dev = [x.cuda() for x in (q, k, v, do)]
    o, lse = fa.fwd(*dev[:3], **kw)
    grads = fa.bwd(*dev[:3], o, dev[3], lse, **kw)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_OK
    keep = keep_bits(3, 2, 150, Nk, p, 3, 0) if p > 0 else None
    want, tol = plain(q, k, v, do, lens=lens, bias=bias, keep=keep, p8=oracle.p8(p),
                      exact_d=True, window=window, causal=case.get("causal", False),
                      q_offset=case.get("q_offset", 0))
    one = torch.zeros(3, 150, dtype=torch.bool)  # rows whose tile of queries sees one key tile
    for b in range(3):
        for t0 in range(0, 150, 128):
            pos = t0 + case.get("q_offset", 0)
            see = range(-(-lens[b] // 128))
            if case.get("causal"):
                see = [j for j in see if 128 * j <= pos + 127]
            if window[0] >= 0:
                see = [j for j in see if 128 * j + 127 >= pos - window[0] and
                       128 * j <= pos + 127 + window[1]]
            one[b, t0:t0 + 128] = len(see) == 1
    for b in range(3):
        if one[b].any():
            within("dq", grads[0][b][:, one[b].cuda()], want["dq"][b][:, one[b]],
                   tol["dq"][b][:, one[b]])
        if one[b].all():
            within("dk", grads[1][b], want["dk"][b], tol["dk"][b])
    assert one.any()


@gpu
def test_more_units_than_multiprocessors():
    check(40, 4, 4, 140, 260, 64, lens=[7 * i % 261 for i in range(40)], seed=7)


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_equal_lengths_are_the_usual_calls(d):
    # keys that the causal mask hides: the plain kernels' results, bit by bit, but for what comes
    # from a D of the scores instead of the rounded O (rows that see one key tile)
    q, k, v, do = (x.cuda() for x in draw(2, 2, 2, 300, 300, d, 8))
    o, lse = fa.fwd(q, k, v, causal=True)
    out = (o, lse) + fa.bwd(q, k, v, o, do, lse, causal=True)
    pad = torch.zeros((2, 2, 60, d), dtype=torch.bfloat16, device="cuda")
    kk, vv = torch.cat((k, pad), 2).contiguous(), torch.cat((v, pad), 2).contiguous()
    o2, lse2 = fa.fwd(q, kk, vv, causal=True)
    dq, dk, dv = fa.bwd(q, kk, vv, o2, do, lse2, causal=True)
    assert dk[:, :, 300:].eq(0).all() and dv[:, :, 300:].eq(0).all()
    assert torch.equal(out[0], o2) and torch.equal(out[1], lse2)
    assert torch.equal(out[2][:, :, 128:], dq[:, :, 128:])
    assert torch.equal(out[4], dv[:, :, :300])
    # the first row's weight is 1 whatever its score: no gradient, where the rounded O leaves some
    assert dq[:, :, 0].abs().max() < 1e-6 < out[2][:, :, 0].abs().max() + 1e-6


# ---------------------------------------------------------------- bias by relative position

RULES = [(32, 128, True), (32, 128, False), (8, 20, True), (16, 500, False)]


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rule", RULES)
def test_bias_and_its_gradient(rule, d):
    check(2, 2, 2, 300, 300, d, rule=rule, seed=10)


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rule", RULES[:2])
def test_bias_with_a_causal_mask_and_padding(rule, d):
    check(3, 4, 2, 260, 260, d, rule=rule, causal=True, lens=[0, 130, 255], junk=math.nan, seed=11)


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_offset", [-300, -1, 0, 77, 128, 400])
def test_bias_with_an_offset(q_offset, d):
    check(1, 2, 2, 140, 420, d, rule=(8, 30, True), q_offset=q_offset, seed=12)


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("clip", [(0, 0), (1, 0), (0, 3), (200, 100), (700, 700)])
def test_a_row_per_distance(clip, d):
    check(1, 2, 2, 260, 300, d, clip=clip, table_type=torch.bfloat16, seed=13)


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_far_tiles_on_both_sides(d):
    check(2, 2, 1, 700, 800, d, rule=(8, 16, True), lens=[800, 500], seed=14)


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_bias_with_dropout_and_window(d):
    check(2, 2, 2, 200, 200, d, rule=(16, 60, True), p=0.25, window=(90, 40), lens=[200, 100],
          seed=15)


@gpu
@pytest.mark.parametrize("Nq,Nk", [(1, 1), (1, 2), (2, 1), (129, 1), (1, 400)])
def test_bias_at_the_smallest_sizes(Nq, Nk):
    check(3, 2, 2, Nq, Nk, 64, rule=(8, 16, True), seed=16)


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_a_bucket_of_minus_infinity_hides_its_keys(d):
    table = torch.randn((8, 2), generator=torch.Generator().manual_seed(17))
    table[0] = -math.inf   # the query's own position
    table[3, 1] = -math.inf  # everything far to the left, for one head
    table[7, 0] = -math.inf
    check(1, 2, 2, 400, 400, d, rule=(8, 16, True), table=table, seed=17)


@gpu
def test_units_of_many_heads_and_batches():
    check(9, 20, 20, 130, 140, 64, rule=(8, 16, False), lens=[140, 1, 0, 60, 128, 129, 30, 90, 7],
          seed=18)


@gpu
def test_frozen_bias_and_repeated_calls():
    q, k, v, do = (x.cuda() for x in draw(1, 2, 2, 300, 300, 64, 19))
    rel = fa.rel_bias(torch.randn((8, 2), device="cuda"), fa.rel_buckets(8, 16))
    o, lse = fa.fwd(q, k, v, rel_bias=rel)
    a = fa.bwd(q, k, v, o, do, lse, rel_bias=rel)
    b = fa.bwd(q, k, v, o, do, lse, rel_bias=rel)
    c = fa.bwd(q, k, v, o, do, lse, rel_bias=rel, rel_grad=False)
    assert len(a) == 4 and len(c) == 3
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert all(torch.equal(x, y) for x, y in zip(a, c))


@gpu
def test_gradient_of_the_table_against_differences():
    q, k, v, do = draw(1, 2, 2, 150, 150, 64, 20)
    rule = (8, 30, True)
    table = torch.randn((8, 2), generator=torch.Generator().manual_seed(2)).double()
    b = fa.rel_buckets(*rule)
    rel = fa.rel_bias(table.float().cuda(), b)
    dev = [x.cuda() for x in (q, k, v, do)]
    o, lse = fa.fwd(*dev[:3], rel_bias=rel)
    dt = fa.bwd(*dev[:3], o, dev[3], lse, rel_bias=rel)[3].cpu().double()
    of = torch.tensor([bucket(rule, x) for x in range(-150, 151)])

    def loss(t):
        out, _ = plain(q, k, v, bias=lambda h, x: t[:, h][of[x + 150]])
        return (out["o"] * do.double()).sum()
    step = 1e-4  # the differences' own error is about step^2 times a third derivative
    for n, h in ((0, 0), (1, 1), (3, 0), (5, 1), (7, 0)):
        up, down = table.float().double().clone(), table.float().double().clone()
        up[n, h] += step
        down[n, h] -= step
        slope = (loss(up) - loss(down)) / (2 * step)
        assert abs(slope - dt[n, h]) <= 2e-3 * max(1.0, dt.abs().max().item())


# ---------------------------------------------------------------- steps over a cache

def check_step(B, H, Hkv, Nq, Nk, d, lens=None, rule=(32, 128, False), causal=True, window=-1,
               num_ctas=0, junk=None, seed=0, table_type=torch.float32):
    q, k, v, _ = draw(B, H, Hkv, Nq, Nk, d, seed)
    if junk is not None:
        for b, n in enumerate(lens):
            k[b, :, n:] = junk
            v[b, :, n:] = junk
    table = torch.randn((rule[0], H), generator=torch.Generator().manual_seed(seed)).mul(2)
    table = table.to(table_type)
    rel = fa.rel_bias(table.cuda(), fa.rel_buckets(*rule))
    lens_dev = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = fa.decode(q.cuda(), k.cuda(), v.cuda(), causal=causal, seqlens_k=lens_dev,
                       num_ctas=num_ctas, window_left=window, rel_bias=rel)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_OK
    of = torch.tensor([bucket(rule, x) for x in range(-Nk, Nk + Nq + 1)])
    starts = [(Nk if lens is None else n) - Nq for n in lens or [Nk] * B]
    want, tol = plain(q, k, v, causal=causal, window=(window, -1), lens=lens, starts=starts,
                      bias=lambda h, x: table[:, h].double()[of[x + Nk]])
    none = want["lse"].isinf()
    got = lse.cpu().double()
    assert torch.equal(got[none], want["lse"][none])
    if (~none).any():
        assert (got - want["lse"])[~none].abs().max() <= LSE_TOL
    within("o", o, want["o"], tol["o"])
    return o, lse


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,G", [(1, 1), (1, 4), (3, 4), (5, 4), (24, 1), (5, 5), (33, 3), (128, 1)])
def test_step(Nq, G, d):
    check_step(3, 2 * G, 2, Nq, 700, d, lens=[700, 300, 129], junk=math.nan, seed=21)


@gpu
@pytest.mark.parametrize("Nq", [3, 20])
@pytest.mark.parametrize("num_ctas", [1, 7, 50, 1000])
@pytest.mark.parametrize("rule", [(32, 128, True), (8, 20, False), (64, 1000, True)])
def test_step_however_it_is_split(rule, num_ctas, Nq):
    check_step(2, 4, 2, Nq, 1000, 64, lens=[1000, 555], rule=rule, num_ctas=num_ctas,
               causal=num_ctas != 7, seed=22, table_type=torch.bfloat16)


@gpu
@pytest.mark.parametrize("Nq", [1, 30])
def test_step_of_many_ragged_sequences(Nq):
    # more batch rows than threads plan with at once, none without a length among them
    lens = [(37 * i) % 301 for i in range(600)]
    check_step(600, 1, 1, Nq, 300, 64, lens=lens, seed=24)
    check_step(70, 2, 2, Nq, 900, 128, lens=[(113 * i) % 901 for i in range(70)], seed=25)


@gpu
@pytest.mark.parametrize("Nq", [2, 40])
@pytest.mark.parametrize("d", [64, 128])
def test_step_with_a_window_and_the_shortest_caches(d, Nq):
    check_step(5, 2, 2, Nq, 300, d, lens=[0, 1, 2, 128, 300], junk=math.inf, window=100, seed=23)
    check_step(5, 2, 2, Nq, 700, d, lens=[0, 1, 2, 640, 700], junk=math.nan, window=100, seed=26)


# ---------------------------------------------------------------- the map of distances

@pytest.mark.parametrize("num_buckets", [4, 8, 32, 64])
@pytest.mark.parametrize("far", [33, 128, 300, 2000])
@pytest.mark.parametrize("both", [False, True])
def test_buckets_by_the_rule(num_buckets, far, both):
    if far <= (num_buckets // 2 if both else num_buckets) // 2:
        return
    m, left = fa.fa_rel_buckets(num_buckets, far, both)
    m = m.tolist()
    last = len(m) - 1 - left
    assert m == [bucket((num_buckets, far, both), x) for x in range(-left, last + 1)]
    # what lies beyond has the ends' buckets, and the ends are where these begin
    assert m[0] == bucket((num_buckets, far, both), -10 * far) != m[1]
    assert m[-1] == bucket((num_buckets, far, both), 10 * far)


def test_buckets_at_exact_powers():
    # 16 buckets of both sides: 4 exact ones, then 4 up to 64 = 4 * 2^4: they begin at 4, 8, 16, 32
    m, left = fa.fa_rel_buckets(16, 64, True)
    assert left == 32 and m.tolist()[left::-1].index(5) == 8
    assert [m.tolist()[left - n] for n in (3, 4, 7, 8, 15, 16, 31, 32)] == [3, 4, 4, 5, 5, 6, 6, 7]


def test_buckets_refused():
    for args in ((2, 128, True), (1, 128, False), (33, 128, True), (32, 8, True), (32, 16, False),
                 (2000, 30000, False), (32, 40000, True)):
        with pytest.raises(fa.FAError):
            fa.fa_rel_buckets(*args)


# ---------------------------------------------------------------- refusals

def test_c_entry_points_refuse_on_the_host():
    import ctypes
    lib = fa.load()
    a = ctypes.c_void_p(1 << 20)
    off = ctypes.c_void_p((1 << 20) + 8)
    none = None

    def fwd(q=a, k=a, v=a, o=a, lse=a, B=1, H=4, Hkv=2, Nq=5, Nk=9, d=64, scale=0.125, off=0,
            wl=-1, wr=-1, p=0.0, lines=none, left=3, right=3):
        return lib.fa_fwd_cross(q, k, v, o, lse, B, H, Hkv, Nq, Nk, d, scale, 0, off, wl, wr, p, 0,
                                0, None, lines, left, right, None)
    bad = fa.FA_ERR_INVALID_ARG
    for kw in (dict(q=none), dict(k=off), dict(o=none), dict(lse=ctypes.c_void_p(2)), dict(B=0),
               dict(Hkv=3), dict(Hkv=0), dict(Nq=0), dict(Nk=0), dict(scale=0.0), dict(p=1.0),
               dict(wl=-2), dict(wr=-5), dict(off=(1 << 28) + 1), dict(off=-(1 << 28) - 1),
               dict(Nk=(1 << 28) + 1), dict(B=1 << 10, Nk=1 << 21), dict(lines=a, left=-1),
               dict(lines=ctypes.c_void_p(6)), dict(lines=a, right=1 << 17)):
        assert fwd(**kw) == bad, kw
    assert fwd(d=96) == fa.FA_ERR_UNSUPPORTED
    assert fwd(lines=a, left=40000, right=40000) == fa.FA_ERR_UNSUPPORTED

    def bwd(dq=a, ws=a, wsb=1 << 30, lines=a, map=a, nb=8, dt=a, H=4, Nq=5):
        return lib.fa_bwd_cross(a, a, a, a, a, a, dq, a, a, 1, H, 2, Nq, 9, 64, 0.125, 0, 0, -1, -1,
                                0.0, 0, 0, None, lines, 3, 3, map, nb, dt, ws, wsb, None)
    assert bwd(dq=off) == bad and bwd(map=none) == bad and bwd(lines=none) == bad
    assert bwd(nb=0) == bad and bwd(dt=ctypes.c_void_p(3)) == bad and bwd(Nq=-1) == bad
    assert bwd(nb=1 << 17) == fa.FA_ERR_UNSUPPORTED
    need = fa.fa_bwd_cross_workspace_size(1, 4, 5, 9, 64, False, 0, True, 3, 3)
    assert bwd(ws=none) == bwd(wsb=need - 1) == bwd(ws=off) == fa.FA_ERR_WORKSPACE
    # no table gradient: D, 20 floats, and a list of up to 4 key tiles with their number
    assert fa.fa_bwd_cross_workspace_size(1, 4, 5, 9, 64) == 512 < need
    assert fa.fa_bwd_cross_workspace_size(1, 4, 0, 9, 64) == 0
    assert fa.fa_bwd_cross_workspace_size(1, 4, 5, 9, 64, False, 0, True, -1, 3) == 0

    def lines(table=a, kind=0, map=a, left=3, right=3, nb=8, H=4, out=a):
        return lib.fa_rel_bias(table, kind, map, left, right, nb, H, out, None)
    for kw in (dict(table=none), dict(map=none), dict(out=none), dict(left=-1), dict(nb=0),
               dict(H=0), dict(table=ctypes.c_void_p((1 << 20) + 2))):
        assert lines(**kw) == bad, kw
    assert lines(kind=2) == lines(H=70000) == lines(nb=70000) == fa.FA_ERR_UNSUPPORTED
    assert fa.fa_rel_line_length(-1, 0) == fa.fa_rel_line_length(40000, 40000) == 0

    def step(lines=a, left=3, Nk=9, Nq=1, d=64):
        return lib.fa_decode_rel(a, a, a, a, a, 1, 4, 2, Nq, Nk, d, 0.125, 1, -1, None, lines, left,
                                 3, 4, None, 0, None)
    assert step(lines=none) == step(left=-2) == step(Nk=(1 << 28) + 1) == bad
    assert step(Nq=65) == step(d=32) == fa.FA_ERR_UNSUPPORTED
    assert step() == fa.FA_ERR_WORKSPACE  # a number of CTAs: heads may be cut
    # 4 CTAs, a header and two pieces of 8 rows each: 4 x 16 bytes, 64 floats, 64 x 64 floats
    assert fa.fa_decode_rel_workspace_size(1, 4, 2, 1, 9, 64, 4) == 256 + 256 + 16384
    # tiles of 128 rows: 2 heads and 2 CTAs of 26 rows, 104 x 64 and 104 floats, 2 pieces' numbers
    assert fa.fa_decode_rel_workspace_size(1, 4, 2, 13, 9, 64, 4) == 104 * 256 + 512 + 256
    assert fa.fa_decode_rel_workspace_size(1, 4, 2, 5, 9, 128, 4) == 40 * 512 + 256 + 256
    assert fa.fa_decode_rel_workspace_size(1, 4, 2, 65, 9, 64, 4) == 0
    for left, right in ((0, 0), (3, 0), (5, 6), (1000, 1001)):
        assert fa._line_length(left, right) == fa.fa_rel_line_length(left, right)
    # the block forms refuse integers beyond their parameters' range
    assert lib.fa_fwd_cross_block(None, None) == bad
    block = fa._FWD_CROSS_BLOCK(*[1 << 20] * 5, 1, 4, 2, 5, 1 << 33, 64, 0.125, 0, 0, -1, -1, 0.0, 0, 0,
                                0, 0, 0, 0)
    assert lib.fa_fwd_cross_block(block, None) == bad


def test_binding_refuses_on_the_cpu():
    # shapes, types and devices are refused before anything runs
    x = torch.zeros((1, 2, 8, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.fwd(x, x[:, :, :4].contiguous(), x)
    b = fa.RelBuckets(torch.zeros(5, dtype=torch.int32), 2, 4)
    with pytest.raises(ValueError):
        fa.rel_bias(torch.zeros((4, 2)), b)


@gpu
def test_binding_refuses():
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device="cuda")
    q, k = z(2, 4, 40, 64), z(2, 2, 100, 64)
    o, lse = fa.fwd(q, k, k)
    b = fa.rel_buckets(8, 16)
    rel = fa.rel_bias(z(8, 4, t=torch.float32), b)
    for call in (lambda: fa.fwd(q, k, z(2, 2, 99, 64)), lambda: fa.fwd(q, z(2, 3, 100, 64), k),
                 lambda: fa.fwd(q, z(1, 2, 100, 64), z(1, 2, 100, 64)),
                 lambda: fa.fwd(q, z(2, 2, 100, 128), z(2, 2, 100, 128)),
                 lambda: fa.fwd(q, k, k, block_mask=z(1, 1, t=torch.uint8)),
                 lambda: fa.fwd(q, k, k, seqlens_k=z(3, t=torch.int32)),
                 lambda: fa.fwd(q, k, k, seqlens_k=z(2, t=torch.int64)),
                 lambda: fa.fwd(q, k, k, seqlens_k=torch.zeros(2, dtype=torch.int32)),
                 lambda: fa.fwd(z(2, 2, 40, 64), k, k, rel_bias=rel),  # lines of 4 heads
                 lambda: fa.bwd(q, k, k, z(2, 4, 41, 64), q, lse),
                 lambda: fa.bwd(q, k, k, o, q, lse.double()),
                 lambda: fa.bwd(q, k, k, o, q, lse[:, :, :39]),
                 lambda: fa.decode(q[:, :, :1].contiguous(), k, k, rel_bias=fa.rel_bias(
                     z(8, 2, t=torch.float32), b)),
                 lambda: fa.rel_bias(z(7, 4, t=torch.float32), b),
                 lambda: fa.rel_bias(z(8, 4, t=torch.float16), b),
                 lambda: fa.rel_bias(z(4, 8, t=torch.float32).T, b),
                 lambda: fa.rel_bias(z(8, 4, t=torch.float32), b._replace(left=99)),
                 lambda: fa.rel_bias(z(8, 4, t=torch.float32), b._replace(map=b.map.long()))):
        with pytest.raises(ValueError):
            call()
    small = z(16, t=torch.uint8)
    for call in (lambda: fa.bwd(q, k, k, o, q, lse, workspace=small),
                 lambda: fa.fwd(q, k, k, window=(-2, -1)), lambda: fa.fwd(q, k, k, dropout_p=1.0),
                 lambda: fa.fwd(q, k, k, scale=-1.0), lambda: fa.fwd(q, k, k, q_offset=1 << 29)):
        with pytest.raises(fa.FAError):
            call()
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_OK


@gpu
def test_a_map_with_rows_that_the_table_lacks():
    m = torch.tensor([0, 5, 1, -1, 2], dtype=torch.int32, device="cuda")
    table = torch.full((3, 1), 2.0, device="cuda")
    rel = fa.rel_bias(table, fa.RelBuckets(m, 2, 3))
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_ERR_INVALID_ARG
    line = rel.lines[0, 256:261].cpu()
    assert line[[1, 3]].eq(0).all() and (line[[0, 2, 4]] - 2 * math.log2(math.e)).abs().max() < 1e-6


# ---------------------------------------------------------------- graphs, streams, a whole layer

@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_captured_and_replayed(d):
    """Forward, backward and a step in one graph, replayed with other values and lengths."""
    rule = (32, 128, False)
    b = fa.rel_buckets(*rule)
    q, k, v, do = (x.cuda() for x in draw(2, 4, 2, 200, 300, d, 30))
    table = torch.randn((32, 4), device="cuda")
    lens = torch.tensor([300, 100], dtype=torch.int32, device="cuda")
    q1 = q[:, :, :1].contiguous()

    def run():
        rel = fa.rel_bias(table, b)
        o, lse = fa.fwd(q, k, v, causal=True, q_offset=100, seqlens_k=lens, rel_bias=rel)
        g = fa.bwd(q, k, v, o, do, lse, causal=True, q_offset=100, seqlens_k=lens, rel_bias=rel)
        return (o, lse) + g + fa.decode(q1, k, v, causal=True, seqlens_k=lens, rel_bias=rel)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for seed, n in ((31, [300, 100]), (32, [17, 290]), (33, [0, 128])):
        for x, y in zip((q, k, v, do), draw(2, 4, 2, 200, 300, d, seed)):
            x.copy_(y)
        q1.copy_(q[:, :, :1])
        table.copy_(torch.randn((32, 4), generator=torch.Generator().manual_seed(seed)))
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        graph.replay()
        got = [x.clone() for x in out]
        assert all(torch.equal(x, y) for x, y in zip(got, run()))
    assert fa.fa_device_status() == fa.FA_OK


@gpu
@pytest.mark.parametrize("as_handle", [False, True])
def test_on_another_stream(as_handle):
    q, k, v, do = (x.cuda() for x in draw(2, 4, 2, 200, 300, 64, 34))
    b = fa.rel_buckets(32, 128)
    table = torch.randn((32, 4), device="cuda")
    q1 = q[:, :, :1].contiguous()

    def run(**kw):
        rel = fa.rel_bias(table, b, **kw)
        o, lse = fa.fwd(q, k, v, rel_bias=rel, **kw)
        g = fa.bwd(q, k, v, o, do, lse, rel_bias=rel, **kw)
        return (rel.lines, o, lse) + g + fa.decode(q1, k, v, rel_bias=rel, num_ctas=40, **kw)
    want = run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda.empty_cache()
    for _ in range(2):
        # memory of every size is given back while writes to it wait behind a long kernel
        torch.cuda._sleep(200_000_000)
        late = [torch.empty(n, dtype=torch.uint8, device="cuda").fill_(77)
                for n in (512, 4096, 65536, 1 << 18, 1 << 20, 1 << 21) for _ in range(6)]
        del late
        got = run(stream=side.cuda_stream if as_handle else side)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert fa.fa_device_status() == fa.FA_OK


@gpu
def test_two_streams_at_once():
    """Two calls that overlap, each with its own workspace, give what they give alone."""
    a = [x.cuda() for x in draw(4, 8, 8, 600, 600, 64, 35)]
    c = [x.cuda() for x in draw(2, 8, 8, 500, 900, 128, 36)]
    rel = fa.rel_bias(torch.randn((32, 8), device="cuda"), fa.rel_buckets(32, 128))

    def run(x, **kw):
        o, lse = fa.fwd(*x[:3], rel_bias=rel, **kw)
        return (o, lse) + fa.bwd(*x[:3], o, x[3], lse, rel_bias=rel, **kw)
    want = run(a), run(c)
    torch.cuda.synchronize()
    s = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        got = run(a, stream=s[0]), run(c, stream=s[1])
        torch.cuda.synchronize()
        for x, y in zip(want, got):
            assert all(torch.equal(m, n) for m, n in zip(x, y))
    assert fa.fa_device_status() == fa.FA_OK


@gpu
def test_an_encoder_and_a_decoder_layer_train():
    """Self attention of an encoder with bias, causal self attention of a decoder with bias and
    cross attention between them: gradients of the chained calls against those of the definition
    in 64 bits, tokens of the decoder's next step against its forward pass."""
    B, H, Ns, Nt, d = 2, 2, 150, 90, 64
    g = torch.Generator().manual_seed(40)
    src, tgt, do = (torch.randn((B, H, n, d), generator=g).to(torch.bfloat16).cuda()
                    for n in (Ns, Nt, Nt))
    te, td = (torch.randn((32, H), generator=g).cuda() for _ in range(2))
    lens = torch.tensor([150, 40], dtype=torch.int32, device="cuda")
    enc, dec = fa.rel_buckets(32, 128, True), fa.rel_buckets(32, 128, False)
    re, rd = fa.rel_bias(te, enc), fa.rel_bias(td, dec)
    es, el = fa.fwd(src, src, src, seqlens_k=lens, rel_bias=re)
    ds, dl = fa.fwd(tgt, tgt, tgt, causal=True, rel_bias=rd)
    cs, cl = fa.fwd(ds, es, es, seqlens_k=lens)
    dq, dk, dv = fa.bwd(ds, es, es, cs, do, cl, seqlens_k=lens)
    ge = fa.bwd(src, src, src, es, (dk + dv), el, seqlens_k=lens, rel_bias=re)
    gd = fa.bwd(tgt, tgt, tgt, ds, dq, dl, causal=True, rel_bias=rd)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_OK

    leaf = lambda x: x.double().cpu().requires_grad_()
    s64, t64, te64, td64 = leaf(src), leaf(tgt), leaf(te), leaf(td)

    def attn(q, k, mask=None, bias=None):
        z = q @ k.transpose(2, 3) / math.sqrt(d)
        z = z if bias is None else z + bias
        z = z if mask is None else z.masked_fill(~mask, -math.inf)
        return torch.softmax(z, -1) @ k

    def lookup(t, n, both):
        row = torch.tensor([[bucket((32, 128, both), j - i) for j in range(n)] for i in range(n)])
        return t[row].permute(2, 0, 1)[None]
    pad = (torch.arange(Ns)[None] < lens.cpu()[:, None])[:, None, None]
    e = attn(s64, s64, pad, lookup(te64, Ns, True))
    t = attn(t64, t64, torch.ones(Nt, Nt).tril().bool(), lookup(td64, Nt, False))
    c = attn(t, e, pad)
    (c * do.double().cpu()).sum().backward()
    # every stage rounds its inputs and results to bf16 (2^-8 each); a handful of such stages
    rel_err = lambda x, y: ((x.double().cpu() - y).norm() / y.norm()).item()
    assert rel_err(cs, c.detach()) <= 4 * 2.0 ** -8
    assert rel_err(ge[0].float() + ge[1].float() + ge[2].float(), s64.grad) <= 8 * 2.0 ** -8
    assert rel_err(gd[0].float() + gd[1].float() + gd[2].float(), t64.grad) <= 8 * 2.0 ** -8
    assert rel_err(ge[3], te64.grad) <= 8 * 2.0 ** -8
    assert rel_err(gd[3], td64.grad) <= 8 * 2.0 ** -8
    # the last token alone: a step over the cache of the others, then cross attention
    last = tgt[:, :, -1:].contiguous()
    d1, _ = fa.decode(last, tgt, tgt, causal=True, rel_bias=rd)
    c1, _ = fa.decode(d1, es, es, seqlens_k=lens)
    assert rel_err(d1, t.detach()[:, :, -1:]) <= 2 * 2.0 ** -8
    assert rel_err(c1, c.detach()[:, :, -1:]) <= 4 * 2.0 ** -8
