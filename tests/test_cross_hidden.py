"""Tables of biases that hide keys: entries of -inf and entries so low that they count as that, in the
forward and backward pass and in steps by both of their kernels; and entries out of range."""
import math

import pytest
import torch

import io_aware_exact_07_gb300 as fa
from _cross import F64, bucket, plain, within
from test_cross import LSE_TOL, check, draw

pytestmark = pytest.mark.gpu

RULE = (8, 40, True)


def table_of(H, hide, value=-math.inf):
    """Biases of 8 buckets: 0 to 3 left of the query (0 its own position, 3 all that is far), 4 to 7
    right of it."""
    t = torch.randn((8, H), generator=torch.Generator().manual_seed(H)).mul(2)
    if hide == "far":
        t[3], t[7, 0] = value, value
    elif hide == "near":
        t[:3] = value
    elif hide == "head":
        t[:, 1] = value
    elif hide == "own":  # the first query of a causal call sees nothing else
        t[0] = value
    return t


HIDE = ["far", "near", "head", "own"]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hide", HIDE)
@pytest.mark.parametrize("case", [
    dict(B=1, H=2, Hkv=2, Nq=400, Nk=400), dict(B=1, H=4, Hkv=2, Nq=150, Nk=300, causal=True),
    dict(B=2, H=2, Hkv=1, Nq=300, Nk=100, lens=[100, 3], q_offset=-60),
    dict(B=1, H=2, Hkv=2, Nq=1500, Nk=130, q_offset=-300)])
def test_forward_and_backward(case, hide, d):
    table = table_of(case["H"], hide)
    out = check(d=d, rule=RULE, table=table, seed=80, **case)
    o, lse, dq = (x.cpu() for x in out[:3])
    if hide == "head":  # rows without a key, by the bias alone
        assert lse[:, 1].eq(-math.inf).all() and o[:, 1].eq(0).all() and dq[:, 1].eq(0).all()


# 1 and 24 query rows per K/V head: the step kernel and that of 128-row tiles, with heads in one piece
# and cut, so that some pieces have no visible key
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hide", HIDE)
@pytest.mark.parametrize("num_ctas", [0, 7, 60])
@pytest.mark.parametrize("Nq,G", [(1, 1), (4, 2), (12, 2)])
def test_step(Nq, G, num_ctas, hide, d):
    B, Hkv, Nk, lens = 3, 2, 900, [900, 140, 30]
    H = Hkv * G
    q, k, v, _ = draw(B, H, Hkv, Nq, Nk, d, 81)
    table = table_of(H, hide)
    rel = fa.rel_bias(table.cuda(), fa.rel_buckets(*RULE))
    o, lse = fa.decode(q.cuda(), k.cuda(), v.cuda(), causal=True, num_ctas=num_ctas, rel_bias=rel,
                       seqlens_k=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_OK
    of = torch.tensor([bucket(RULE, x) for x in range(-Nk, Nk + 1)])
    want, tol = plain(q, k, v, causal=True, lens=lens, starts=[n - Nq for n in lens],
                      bias=lambda h, x: table[:, h].double()[of[x + Nk]])
    none = want["lse"].isinf()
    got = lse.cpu().double()
    assert torch.equal(got[none], want["lse"][none]) and o.cpu()[none].eq(0).all()
    if (~none).any():
        assert (got - want["lse"])[~none].abs().max() <= LSE_TOL
    within("o", o, want["o"], tol["o"])
    assert none.any() == (hide == "head")


# What a type's lowest value or a large negative number hides is hidden: fp32 scores and lse could not
# tell keys apart that all have such a bias.
LOW = [-2.0 ** 15, -65504.0, -1e9, torch.finfo(torch.bfloat16).min, torch.finfo(torch.float32).min]


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("hide", HIDE)
def test_low_entries_hide_as_minus_infinity_does(hide, kind):
    q, k, v, do = (x.cuda() for x in draw(2, 4, 2, 200, 260, 64, 82))
    b = fa.rel_buckets(*RULE)

    def run(value):
        t = table_of(4, hide, value).to(kind)
        rel = fa.rel_bias(t.cuda(), b)
        o, lse = fa.fwd(q, k, v, rel_bias=rel)
        out = (o, lse) + fa.bwd(q, k, v, o, do, lse, rel_bias=rel)
        for rows in (1, 20):
            out += fa.decode(q[:, :, :rows].contiguous(), k, v, causal=True, rel_bias=rel)
        return out
    want = run(-math.inf)
    for value in LOW:
        if kind is torch.bfloat16 and value == torch.finfo(torch.float32).min:
            continue  # rounds to -inf
        got = run(value)
        assert all(torch.equal(x, y) for x, y in zip(got, want)), value
    assert all(x.isfinite().all() for i, x in enumerate(want) if i not in (1, 7, 9))
    assert fa.fa_device_status() == fa.FA_OK


def test_a_bias_of_minus_ten_thousand_on_every_key_takes_no_part():
    """Scores near -1e4, which fp32 holds to half a step of 2^-11 in log2 units (and lse in natural
    ones): in the forward a score has its line's and its own, and so has the sum of weights, 4 2^-11 ln 2
    of a weight, less than 2^-9; in the backward lse comes to it with its own half step before and after
    its change of units, 1 + 1.44 + 1 of 2^-11: less than 2^-8 in all."""
    q, k, v, do = draw(1, 2, 2, 200, 260, 64, 83)
    table = table_of(2, "none") - 1e4
    b = fa.rel_buckets(*RULE)
    rel = fa.rel_bias(table.cuda(), b)
    dev = [x.cuda() for x in (q, k, v, do)]
    o, lse = fa.fwd(*dev[:3], rel_bias=rel)
    grads = fa.bwd(*dev[:3], o, dev[3], lse, rel_bias=rel)
    of = torch.tensor([bucket(RULE, x) for x in range(-300, 301)])
    want, tol = plain(q, k, v, do, bias=lambda h, x: table[:, h].double()[of[x + 300]])
    assert (lse.cpu().double() - want["lse"]).abs().max() <= 2 * 2.0 ** -10
    kd, qd, vd, gd = (x.to(F64).abs() for x in (k, q, v, do))
    p = torch.softmax(q.to(F64) @ k.to(F64).transpose(2, 3) / 8 +
                      table.double()[of[torch.arange(260)[None] - torch.arange(200)[:, None] + 300]]
                      .permute(2, 0, 1), -1)
    off_o = 2.0 ** -9 * (p @ vd)
    within("o", o, want["o"], tol["o"] + off_o)
    within("dv", grads[2], want["dv"], tol["dv"] + 2.0 ** -8 * (p.transpose(2, 3) @ gd))
    # dS: a weight's error times what it multiplies, and D's from what O is off
    ds = 2.0 ** -8 * tol["ds"] + p * (gd * off_o).sum(-1, keepdim=True)
    within("dq", grads[0], want["dq"], tol["dq"] + ds @ kd / 8)
    within("dk", grads[1], want["dk"], tol["dk"] + ds.transpose(2, 3) @ qd / 8)


@pytest.mark.parametrize("value", [2.0 ** 15 + 1, 1e9, math.inf])
def test_entries_above_the_range_are_reported(value):
    b = fa.rel_buckets(*RULE)
    t = torch.zeros((8, 2), device="cuda")
    t[3, 1] = 2.0 ** 15
    fa.rel_bias(t, b)
    torch.cuda.synchronize()
    assert fa.fa_device_status(clear=True) == fa.FA_OK
    t[3, 1] = value
    line = fa.rel_bias(t, b).lines
    torch.cuda.synchronize()
    assert fa.fa_device_status(clear=True) == fa.FA_ERR_INVALID_ARG
    assert line[1].max().item() == pytest.approx(2.0 ** 15 * math.log2(math.e), rel=2.0 ** -22)
